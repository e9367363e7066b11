"""Cases, plain forms and 64-bit references of the operators of a speculative
decoding step over a 4-bit paged cache, and of the rotated append that serves
every pool.

  append  queries and keys rotated (one position axis or several), the keys and
          values stored in the paged pool: bf16, E4M3 under the blocks' scales,
          or 4-bit codes (these are read back as values)
  decode  attention of one query token per sequence over the 4-bit pool
  multi   attention of several causal query tokens per sequence over it
  verify  drafted tokens against the target's probabilities, from given
          random numbers

``own`` False computes them with elementary torch operations in 32 bits
(verification's sums in 64); ``own`` True calls the library.  ``exact`` restates
each in 64 bits.

A 4-bit pool is uint8 [num_blocks, kv_heads, block * dim * 9 / 8]: per (block,
head) the codes of K and of V ([block, dim / 2] bytes each), then the (scale,
min) bf16 pairs of K and of V ([block, dim / 64, 2] each).  A code c stands for
min + scale * c; element e of a row is nibble e % 8 (the low one of a byte
first) of 32-bit word (e % 64 / 8) * (dim / 64) + e / 64 of its codes.
"""
import math

import numpy as np
import torch

own = False

POOL_DTYPE = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
MAX_POSITION = 16384


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # A decode step of four short sequences on a 4-bit pool: call latency.
        dict(name="append 4x1 int4", op="append", batch=4, heads=8, kv_heads=2, dim=64, block=16,
             dtype="int4", lo=1, hi=200, new=1, rotary=64, interleaved=False, axes=1),
        # One decode step's rows of 128 sequences of a 70B-like layer.
        dict(name="append 128x1 bf16", op="append", batch=128, heads=64, kv_heads=8, dim=128, block=32,
             dtype="bf16", lo=1024, hi=8192, new=1, rotary=128, interleaved=False, axes=1),
        # The rows of a speculative step: part of every head rotated, pairs side by side.
        dict(name="append 64x5 fp8", op="append", batch=64, heads=32, kv_heads=8, dim=128, block=16,
             dtype="fp8", lo=512, hi=4096, new=5, rotary=64, interleaved=True, axes=1),
        # Eight prompts with images: positions of time, height and width.
        dict(name="append 8x8k int4", op="append", batch=8, heads=32, kv_heads=8, dim=128, block=16,
             dtype="int4", lo=1024, hi=8192, new=0, rotary=128, interleaved=False, axes=3),
        # A tiny decode batch: launch latency.
        dict(name="decode tiny", op="decode", batch=4, heads=8, kv_heads=2, dim=64, block=16, lo=1, hi=200),
        # An 8B-like layer's batch.
        dict(name="decode 64x4k", op="decode", batch=64, heads=32, kv_heads=8, dim=128, block=16, lo=512,
             hi=4096),
        # Long contexts, few sequences.
        dict(name="decode 8x131k", op="decode", batch=8, heads=32, kv_heads=8, dim=128, block=16, lo=32768,
             hi=131072),
        # A 70B-like layer's batch.
        dict(name="decode 128x8k", op="decode", batch=128, heads=64, kv_heads=8, dim=128, block=32, lo=1024,
             hi=8192),
        # Speculative verification: five query tokens per sequence.
        dict(name="multi 64x5", op="multi", batch=64, heads=32, kv_heads=8, dim=128, block=16, lo=512, hi=4096,
             queries=5),
        # Whole prompts of four requests.
        dict(name="multi 4x4k", op="multi", batch=4, heads=32, kv_heads=8, dim=128, block=16, lo=1024, hi=4096,
             queries=0),
        # One request, four drafts, a small vocabulary.
        dict(name="verify 1x4 bf16", op="verify", batch=1, drafts=4, vocab=32000, dtype="bf16", draft="probs"),
        # A batch of 64 requests with five drafts each.
        dict(name="verify 64x5 fp32", op="verify", batch=64, drafts=5, vocab=128256, dtype="fp32", draft="probs"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 5e14


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        c = _draw(rng)
        if _cost(c) <= most and (c["op"] == "verify" or _plain_bytes(c) < 4e10):
            return c


def _plain_bytes(c):
    """What the plain form holds of padded keys, values and scores."""
    L = _lengths(c)
    if c["op"] == "append":
        return 40 * int(_new_counts(c, L).sum()) * (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
    n = int(_new_counts(c, L).max())
    return c["batch"] * (int(L.max()) + 32) * (24 * c["kv_heads"] * c["dim"] + 12 * c["heads"] * n)


def _draw(rng):
    op = rng.choice(("append", "decode", "multi", "verify"))
    if op == "verify":
        return dict(op=op, batch=_log_int(rng, 1, 256), drafts=rng.randint(0, 16), vocab=_log_int(rng, 100, 262144),
                    dtype=rng.choice(("fp32", "bf16", "fp16")), draft=rng.choice(("probs", "probs", "none")))
    c = dict(op=op, batch=_log_int(rng, 1, 128), kv_heads=rng.choice((1, 2, 4, 8)), dim=rng.choice((64, 128)),
             block=rng.choice((16, 32)))
    c["heads"] = c["kv_heads"] * rng.randint(1, 8)
    hi = _log_int(rng, 1, 131072 if op == "decode" else 8192)
    c.update(lo=max(1, int(hi * rng.uniform(0.05, 1.0))), hi=hi)
    if op == "multi":
        c.update(queries=rng.choice((0, rng.randint(2, 16), _log_int(rng, 1, 1024))))
    if op == "append":
        c.update(dtype=rng.choice(("bf16", "fp8", "int4")), new=rng.choice((0, 1, _log_int(rng, 1, 512))),
                 rotary=rng.choice((c["dim"], c["dim"], c["dim"] // 2, 16 * rng.randint(1, c["dim"] // 16))),
                 interleaved=rng.random() < 0.3, axes=rng.choice((1, 1, 2, 3)))
    return c


def _lengths(case):
    """The batch's lengths, from the case alone (a seed only permutes them)."""
    r = np.random.RandomState([case["batch"], case["lo"], case["hi"]])
    return r.randint(case["lo"], case["hi"] + 1, case["batch"]).astype(np.int64)


def _new_counts(case, L):
    """New (query) tokens of each sequence: a given number of last ones, or all."""
    n = case.get("new", case.get("queries", 1))
    return L if n == 0 else np.minimum(L, n)


def _sections(case):
    """Frequencies of each axis: about as many for each, the first (time) fewest."""
    half, axes = case["rotary"] // 2, case["axes"]
    part = (half + axes - 1) // axes
    return [half - part * (axes - 1)] + [part] * (axes - 1)


def work(case):
    op, B = case["op"], case["batch"]
    if op == "verify":
        e = 4 if case["dtype"] == "fp32" else 2
        rows = 1 if case["draft"] == "none" or case["drafts"] == 0 else 2
        return {"bytes": B * (rows * case["vocab"] * e + 16 * (case["drafts"] + 1) + 8), "flops": 0}
    L = _lengths(case)
    n = _new_counts(case, L)
    T, H, hq, d = int(n.sum()), case["kv_heads"], case["heads"], case["dim"]
    if op == "append":
        stored = {"bf16": 2, "fp8": 1, "int4": 9 / 16}[case["dtype"]]
        again = stored + 2 if case["dtype"] == "int4" else 0           # read back as bf16
        return {"bytes": int(T * d * (4 * hq + 2 * H * (2 + stored + again)) + 4 * T * (1 + case["axes"])),
                "flops": 0}
    pairs = int((n * L - n * (n - 1) // 2).sum())
    blocks = int(((L + case["block"] - 1) // case["block"]).sum())
    return {"bytes": int(L.sum()) * H * d * 9 // 8 + 4 * blocks + 4 * T * hq * d, "flops": 4 * pairs * hq * d}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _tables(case, L, g):
    """int32 tables of randomly placed blocks (padding -1) and the pool size."""
    bs, B = case["block"], case["batch"]
    nb = (L + bs - 1) // bs
    width, need = int(nb.max()), int(nb.sum())
    total = int(need * 1.1) + 1
    perm = torch.randperm(total, device="cuda", generator=g, dtype=torch.int32)
    counts = torch.from_numpy(nb).cuda()
    first = torch.cumsum(counts, 0) - counts
    j = torch.arange(width, device="cuda")
    at = first[:, None] + j
    return torch.where(j < counts[:, None], perm[at.clamp(max=need - 1)], -1).to(torch.int32).contiguous(), total


def _pool4(case, blocks, g):
    """A 4-bit pool of rows as an append leaves them: codes about the middle of
    their range, scales that vary from group to group, offsets off centre."""
    bs, H, d = case["block"], case["kv_heads"], case["dim"]
    pool = torch.empty((blocks, H, bs * d * 9 // 8), dtype=torch.uint8, device="cuda")
    codes = torch.randint(0, 256, (2, blocks, H, bs * d), dtype=torch.uint8, device="cuda", generator=g)
    # the mean of two throws, high and low nibble alike: a triangle over 0..15
    mean = ((codes[0] & 15) + (codes[1] & 15) + 1) // 2 + (((codes[0] >> 4) + (codes[1] >> 4) + 1) // 2 << 4)
    pool[:, :, :bs * d] = mean
    scale = 0.3 * (0.5 + torch.rand((blocks, H, bs * d // 32), device="cuda", generator=g))
    low = -scale * (7.0 + torch.rand(scale.shape, device="cuda", generator=g))
    pool[:, :, bs * d:] = torch.stack((scale, low), dim=-1).to(torch.bfloat16).flatten(2).view(torch.uint8)
    return pool


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] == "verify":
        return _prepare_verify(case, g)
    L = np.random.RandomState(int(seed) % (1 << 31)).permutation(_lengths(case))
    B, H, hq, d = case["batch"], case["kv_heads"], case["heads"], case["dim"]
    n = _new_counts(case, L)
    s = dict(case=case, L=L, n=n, T=int(n.sum()), max_n=int(n.max()), max_len=int(L.max()), scale=d ** -0.5,
             seq_lens=torch.from_numpy(L.astype(np.int32)).cuda(),
             query_start=torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda())
    s["tables"], total = _tables(case, L, g)
    if case["op"] != "append":
        s["kv_cache"] = _pool4(case, total, g)
        s["q"] = (2 * torch.randn((s["T"], hq, d), device="cuda", generator=g)).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["workspace"] = torch.empty(128 << 20, dtype=torch.uint8, device="cuda")
        return s
    dtype = case["dtype"]
    if dtype == "int4":
        s["kv_cache"] = torch.zeros((total, H, case["block"] * d * 9 // 8), dtype=torch.uint8, device="cuda")
        s["k_out"] = torch.empty((s["T"], H, d), dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
    else:
        shape = (total, case["block"], H, d)
        s["k_cache"], s["v_cache"] = (torch.zeros(shape, dtype=POOL_DTYPE[dtype], device="cuda") for _ in "kv")
        s["k_scale"] = s["v_scale"] = None
        if dtype == "fp8":
            s["k_scale"], s["v_scale"] = ((torch.rand((total, H), device="cuda", generator=g) + 0.5) / 112
                                          for _ in "kv")
    # the rows of one projection: q, k and v of a token side by side
    qkv = torch.randn((s["T"], hq + 2 * H, d), device="cuda", generator=g)
    qkv *= 0.5 + torch.rand((1, hq + 2 * H, d), device="cuda", generator=g)      # some channels are larger
    s["qkv"] = qkv.to(torch.bfloat16)
    s["q"], s["k"], s["v"] = s["qkv"].split((hq, H, H), dim=1)
    s["q_out"] = torch.empty((s["T"], hq, d), dtype=torch.bfloat16, device="cuda")
    # cosines and sines of every position, their angles in 64 bits
    half = case["rotary"] // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(MAX_POSITION, dtype=torch.float64, device="cuda")[:, None] * freq
    s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), dim=1).float()
    s["sections"], s["positions"] = None, None
    if case["axes"] > 1:
        s["sections"] = _sections(case)
        s["positions"] = torch.randint(0, MAX_POSITION, (case["axes"], s["T"]), dtype=torch.int32, device="cuda",
                                       generator=g)
    return s


def _prepare_verify(case, g):
    B, D, V = case["batch"], case["drafts"], case["vocab"]
    dtype = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[case["dtype"]]
    T = B * (D + 1)
    logits = 3 * torch.randn((T, V), device="cuda", generator=g)
    # the draft model's row i is near the target's, not the same
    near = logits.view(B, D + 1, V)[:, :D].reshape(B * D, V)
    draft = torch.softmax(near + torch.randn(near.shape, device="cuda", generator=g), dim=1)
    tokens = torch.randint(0, V, (B, D + 1), dtype=torch.int32, device="cuda", generator=g)
    if D:
        wait = torch.empty_like(draft).exponential_(generator=g)
        tokens[:, 1:] = (draft / wait).argmax(dim=1).view(B, D).to(torch.int32)
    return dict(case=case, T=T, tokens=tokens.view(-1), target=torch.softmax(logits, dim=1).to(dtype),
                draft=draft.to(dtype) if case["draft"] == "probs" and D else None,
                uniform=torch.rand(T, device="cuda", generator=g),
                query_start=torch.arange(0, T + 1, D + 1, dtype=torch.int32, device="cuda"),
                seq_lens=torch.randint(D + 1, 4096, (B,), dtype=torch.int32, device="cuda", generator=g),
                out_tokens=torch.empty(T, dtype=torch.int32, device="cuda"),
                accepted=torch.empty(B, dtype=torch.int32, device="cuda"),
                new_lens=torch.empty(B, dtype=torch.int32, device="cuda"))


# --------------------------------------------------------------------------
# Plain forms (32 bits)
# --------------------------------------------------------------------------

def _values4(records, bs, d):
    """fp32 K and V rows [..., block, dim] of 4-bit records [..., bytes]."""
    at, out = 0, []
    for _ in "kv":
        b = records[..., at:at + bs * d // 2].unflatten(-1, (bs, 8, d // 64, 4))
        at += bs * d // 2
        c = torch.stack((b & 15, b >> 4), dim=-1).flatten(-2)          # [..., bs, word, group, nibble]
        out.append(c.transpose(-3, -2).float())
    for i in range(2):
        par = records[..., at:at + bs * d // 16].contiguous().view(torch.bfloat16).float()
        at += bs * d // 16
        par = par.unflatten(-1, (bs, d // 64, 2))
        out[i] = (out[i] * par[..., 0, None, None] + par[..., 1, None, None]).flatten(-3)
    return out


def _plain_attention(s):
    c = s["case"]
    B, H, d, bs = c["batch"], c["kv_heads"], c["dim"], c["block"]
    K, V = _values4(s["kv_cache"][s["tables"].clamp(min=0).long()], bs, d)   # [B, MB, H, bs, d]
    K, V = (x.transpose(2, 3).flatten(1, 2) for x in (K, V))                # [B, tokens, H, d]
    t = torch.arange(K.shape[1], device=K.device)
    i = torch.arange(s["max_n"], device=K.device)
    qs = s["query_start"].long()
    n = (qs[1:] - qs[:-1])[:, None]
    rows = (qs[:-1, None] + i).clamp(max=s["T"] - 1)                        # [B, max_n]
    q = s["q"][rows].float().view(B, -1, H, c["heads"] // H, d)
    S = torch.einsum("bnhgd,bthd->bhgnt", q, K).mul_(s["scale"])
    pos = s["seq_lens"].long()[:, None] - n + i                             # [B, max_n]
    S.masked_fill_((t > pos[:, :, None])[:, None, None], -math.inf)
    V.masked_fill_((t >= s["seq_lens"][:, None])[:, :, None, None], 0.0)
    S.sub_(S.amax(dim=-1, keepdim=True)).exp_()
    S.div_(S.sum(dim=-1, keepdim=True))
    o = torch.einsum("bhgnt,bthd->bnhgd", S, V).flatten(2, 3).to(torch.bfloat16)
    s["out"][rows[i < n]] = o[i < n]
    return s["out"]


def _rotated(x, s):
    """bf16 rows [T, heads, dim] rotated in fp32 (each product and sum rounded once)."""
    c = s["case"]
    R, half = c["rotary"], c["rotary"] // 2
    if s["positions"] is None:
        pos = s["pos"][None].expand(half, -1)
    else:
        axis = torch.repeat_interleave(torch.arange(c["axes"], device=x.device),
                                       torch.tensor(s["sections"], device=x.device))
        pos = s["positions"].long()[axis]                              # [half, T]
    j = torch.arange(half, device=x.device)[:, None]
    cos, sin = s["cos_sin"][pos, j].T[:, None], s["cos_sin"][pos, j + half].T[:, None]
    y = x.clone()
    first, second = (slice(0, R, 2), slice(1, R, 2)) if c["interleaved"] else (slice(0, half), slice(half, R))
    a, b = x[:, :, first].float(), x[:, :, second].float()
    y[:, :, first] = (a * cos - b * sin).to(torch.bfloat16)
    y[:, :, second] = (b * cos + a * sin).to(torch.bfloat16)
    return y


def _coded4(x):
    """4-bit codes [T, H, word, group, nibble] and (scale, min) [T, H, group] of bf16 rows."""
    x = torch.nan_to_num(x.float(), nan=0.0).clamp(-2.0 ** 126, 2.0 ** 126) + 0.0
    x = x.unflatten(-1, (-1, 64))
    lo, hi = x.amin(dim=-1), x.amax(dim=-1)
    step = (hi - lo) * np.float32(1 / 15)
    # up to the next bf16 number, so that fifteen steps reach the largest value
    step = ((step.view(torch.int32) + 0xFFFF) & -65536).view(torch.float32).clamp(min=2.0 ** -126)
    c = torch.round((x - lo[..., None]) * (torch.ones_like(step) / step)[..., None]).clamp(0, 15)
    return c.to(torch.uint8).unflatten(-1, (8, 8)).transpose(-3, -2), step, lo


def _plain_append(s):
    c = s["case"]
    bs, d, dtype = c["block"], c["dim"], c["dtype"]
    qs = s["query_start"].long()
    n = qs[1:] - qs[:-1]
    b = torch.repeat_interleave(torch.arange(c["batch"], device=qs.device), n, output_size=s["T"])
    s["pos"] = torch.arange(s["T"], device=qs.device) - qs[b] + (s["seq_lens"].long() - n)[b]
    s["q_out"].copy_(_rotated(s["q"], s))
    k, v = _rotated(s["k"], s), s["v"]
    blk, row = s["tables"].long()[b, s["pos"] // bs], s["pos"] % bs
    if dtype == "bf16":
        s["k_cache"][blk, row], s["v_cache"][blk, row] = k, v
        return s["q_out"], s["k_cache"], s["v_cache"]
    if dtype == "fp8":
        for x, cache, scale in ((k, s["k_cache"], s["k_scale"]), (v, s["v_cache"], s["v_scale"])):
            y = (x.float() / scale[blk][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            cache.view(torch.uint8)[blk, row] = y.view(torch.uint8)
        return s["q_out"], s["k_cache"], s["v_cache"]
    H = c["kv_heads"]
    codes = s["kv_cache"][:, :, :bs * d].unflatten(-1, (2, bs, d // 2))
    params = s["kv_cache"][:, :, bs * d:].unflatten(-1, (2, bs, d // 16))
    heads = torch.arange(H, device=qs.device)
    for i, x, out in ((0, k, s["k_out"]), (1, v, s["v_out"])):
        y, step, lo = _coded4(x)
        to = (blk[:, None], heads, i, row[:, None])
        codes[to] = (y[..., 0::2] + 16 * y[..., 1::2]).flatten(-3)
        pair = torch.stack((step, lo), dim=-1).to(torch.bfloat16)
        params[to] = pair.flatten(-2).view(torch.uint8)
    # the rows read back
    k, v = _values4(s["kv_cache"][blk], bs, d)                         # [T, H, bs, d]
    at = (torch.arange(s["T"], device=qs.device)[:, None], heads, row[:, None])
    s["k_out"].copy_(k[at])
    s["v_out"].copy_(v[at])
    return s["q_out"], s["k_out"], s["v_out"]


def _plain_verify(s):
    p, q, u = s["target"], s["draft"], s["uniform"]
    D1 = s["case"]["drafts"] + 1
    B, V = s["case"]["batch"], s["case"]["vocab"]
    x = s["tokens"].view(B, D1)[:, 1:].long()                          # the drafts
    px = p.view(B, D1, V)[:, :-1].gather(2, x[..., None])[..., 0].double()
    uu = u.view(B, D1).double()
    qx = 1.0 if q is None else q.view(B, D1 - 1, V).gather(2, x[..., None])[..., 0].double()
    a = (uu[:, :-1] * qx < px).long().cumprod(dim=1).sum(dim=1)        # accepted
    at = torch.arange(B, device=a.device)
    row = p.view(B, D1, V)[at, a].float()
    if D1 > 1:
        last = a.clamp(max=D1 - 2)
        if q is None:
            less = row.scatter(1, x[at, last][:, None], 0.0)
        else:
            less = (row - q.view(B, D1 - 1, V)[at, last].float()).clamp(min=0.0)
        refused = (a < D1 - 1)[:, None] & (less.sum(dim=1) > 0)[:, None]
        row = torch.where(refused, less, row)
    total = row.double().cumsum(dim=1)
    z = (total <= (uu[:, -1] * total[:, -1])[:, None]).sum(dim=1).clamp(max=V - 1)
    i = torch.arange(D1, device=a.device)
    drafts = torch.cat((x, x.new_zeros((B, 1))), dim=1)
    out = torch.where(i < a[:, None], drafts, torch.where(i == a[:, None], z[:, None], -1))
    s["out_tokens"].copy_(out.view(-1))
    s["accepted"].copy_(a)
    s["new_lens"].copy_(s["seq_lens"] - D1 + 1 + a)
    return s["out_tokens"], s["accepted"], s["new_lens"]


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"append": _plain_append, "decode": _plain_attention, "multi": _plain_attention,
                "verify": _plain_verify}[op](s)
    import paged_kv_cache_97_gb300 as pkv
    c = s["case"]
    if op == "decode":
        pkv.paged_attention_decode_q4(s["out"], s["q"], s["kv_cache"], s["tables"], s["seq_lens"], c["block"],
                                      s["max_len"], s["scale"], s["workspace"])
        return s["out"]
    if op == "multi":
        pkv.paged_attention_multi_q4(s["out"], s["q"], s["kv_cache"], s["tables"], s["seq_lens"],
                                     s["query_start"], c["block"], s["max_len"], s["max_n"], s["scale"],
                                     s["workspace"])
        return s["out"]
    if op == "verify":
        pkv.verify_drafts(s["out_tokens"], s["accepted"], s["tokens"], s["target"], s["draft"], s["uniform"],
                          s["query_start"], seq_lens=s["seq_lens"], new_lens=s["new_lens"])
        return s["out_tokens"], s["accepted"], s["new_lens"]
    how = dict(positions=s["positions"], sections=s["sections"], interleaved=c["interleaved"],
               query_start=s["query_start"], max_query_len=s["max_n"])
    if c["dtype"] == "int4":
        pkv.append_rotary_q4(s["q_out"], s["q"], s["k"], s["v"], s["kv_cache"], s["cos_sin"], s["tables"],
                             s["seq_lens"], c["block"], **how)
        pkv.read_q4(s["k_out"], s["v_out"], s["kv_cache"], s["tables"], s["seq_lens"], c["block"],
                    query_start=s["query_start"], max_query_len=s["max_n"])
        return s["q_out"], s["k_out"], s["v_out"]
    pkv.append_rotary(s["q_out"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["cos_sin"], s["tables"],
                      s["seq_lens"], k_scale=s["k_scale"], v_scale=s["v_scale"], **how)
    return s["q_out"], s["k_cache"], s["v_cache"]


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def _cached64(s, b, head):
    """Sequence b's K and V rows of one head, [L, dim] in 64 bits each."""
    c = s["case"]
    bs, d, L = c["block"], c["dim"], int(s["L"][b])
    rec = s["kv_cache"][s["tables"][b, :(L + bs - 1) // bs].long(), head]
    e = torch.arange(d, device=rec.device)
    byte = (e % 64 // 8 * (d // 64) + e // 64) * 4 + e % 8 // 2
    rows = []
    for i in range(2):
        codes = rec[:, i * bs * d // 2:(i + 1) * bs * d // 2].view(-1, bs, d // 2)[:, :, byte]
        codes = torch.where(e % 2 == 1, codes >> 4, codes & 15).double()
        par = rec[:, bs * d + i * bs * d // 16:bs * d + (i + 1) * bs * d // 16].contiguous()
        par = par.view(torch.bfloat16).view(-1, bs, d // 64, 2).double()[:, :, e // 64]
        rows.append((par[..., 1] + par[..., 0] * codes).view(-1, d)[:L])
    return rows


def _exact_attention(s, case):
    G = case["heads"] // case["kv_heads"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    start = np.concatenate([[0], np.cumsum(s["n"])])
    for b in range(case["batch"]):
        L, n = int(s["L"][b]), int(s["n"][b])
        for h in range(case["kv_heads"]):
            K, V = _cached64(s, b, h)
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                rows = slice(int(start[b]) + i, int(start[b]) + i + m)
                q = s["q"][rows, h * G:(h + 1) * G].double()
                S = torch.einsum("ngd,td->ngt", q, K) * s["scale"]
                pos = L - n + i + torch.arange(m, device="cuda")
                S.masked_fill_((torch.arange(L, device="cuda") > pos[:, None])[:, None], -math.inf)
                out[rows, h * G:(h + 1) * G] = torch.softmax(S, dim=-1) @ V
    return out


def _exact_append(s, case):
    """The rotation in 64 bits.  A stored key or value is a decision on the
    rotated bf16 row, so the coded pools' contents have no such value."""
    T, bs, half = s["T"], case["block"], case["rotary"] // 2
    start = np.concatenate([[0], np.cumsum(s["n"])])
    b = np.repeat(np.arange(case["batch"]), s["n"])
    pos = np.arange(T) - start[b] + (s["L"] - s["n"])[b]
    at = np.tile(pos[:, None], (1, half))
    if case["axes"] > 1:
        given, j0 = s["positions"].cpu().numpy(), 0
        for axis, size in enumerate(s["sections"]):
            at[:, j0:j0 + size] = given[axis][:, None]
            j0 += size
    freq = torch.arange(half, device="cuda")
    where = torch.from_numpy(at).cuda()
    cos, sin = (s["cos_sin"][where, freq + o].double()[:, None] for o in (0, half))

    def turned(x):
        y = x.double()
        pair = y[..., :2 * half].unflatten(-1, (half, 2) if case["interleaved"] else (2, half))
        p, r = (pair[..., 0], pair[..., 1]) if case["interleaved"] else (pair[..., 0, :], pair[..., 1, :])
        z = torch.stack((p * cos - r * sin, r * cos + p * sin), dim=-1 if case["interleaved"] else -2)
        return torch.cat((z.flatten(-2), y[..., 2 * half:]), dim=-1)

    q = turned(s["q"])
    if case["dtype"] != "bf16":
        return q, None, None
    to = (s["tables"].long()[torch.from_numpy(b).cuda(), torch.from_numpy(pos // bs).cuda()],
          torch.from_numpy(pos % bs).cuda())
    k, v = s["k_cache"].double(), s["v_cache"].double()
    k[to], v[to] = turned(s["k"]), s["v"].double()
    return q, k, v


def _exact_verify(s, case):
    D1, V = case["drafts"] + 1, case["vocab"]
    tokens, u = s["tokens"].cpu().numpy(), s["uniform"].double().cpu().numpy()
    out = np.full(s["T"], -1, np.int32)
    accepted = np.zeros(case["batch"], np.int32)
    for b in range(case["batch"]):
        r0, a = b * D1, 0

        def row(x, i):
            return x[i].float().double().cpu().numpy()

        while a < D1 - 1:
            x = tokens[r0 + a + 1]
            q = 1.0 if s["draft"] is None else float(s["draft"][r0 - b + a, x])
            if not u[r0 + a] * q < float(s["target"][r0 + a, x]):
                break
            out[r0 + a] = x
            a += 1
        w = row(s["target"], r0 + a)
        if a < D1 - 1:
            less = w.copy()
            if s["draft"] is None:
                less[tokens[r0 + a + 1]] = 0
            else:
                # the difference is a 32-bit number
                less = np.maximum((w - row(s["draft"], r0 - b + a)).astype(np.float32), 0).astype(np.float64)
            w = less if less.sum() > 0 else w
        total = np.cumsum(w)
        out[r0 + a] = min(int(np.searchsorted(total, u[r0 + D1 - 1] * total[-1], side="right")), V - 1)
        accepted[b] = a
    lens = s["seq_lens"].cpu().numpy() - D1 + 1 + accepted
    return [torch.from_numpy(x.astype(np.int32)) for x in (out, accepted, lens)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(s, case)
    if case["op"] == "append":
        return _exact_append(s, case)
    return None if work(case)["flops"] > 2e12 else _exact_attention(s, case)
