"""Cases, plain forms and 64-bit references of the cache operators that work
beside the paged decode attention.

Six operators over the paged pool ([num_blocks, block_size, kv_heads, dim]):

  weights  decode attention that also accumulates the attention weight each
           cached token receives (what an eviction rule ranks tokens by)
  prompt   the same weights for several causal queries per sequence
  select   the tokens each (sequence, KV head) keeps: the most recent ones and
           the heaviest of the others
  evict    the kept rows packed into the sequence's first blocks
  append   new tokens into an 8-bit pool whose (block, head) scales follow
           the data
  diff     differential attention for one query token per sequence

``own`` False computes them with elementary torch operations in 32 bits;
``own`` True calls the library.  ``exact`` restates each in 64 bits.
"""
import math

import numpy as np
import torch

own = False

CODE_MAX = {"int8": 127.0, "fp8": 448.0}
POOL_DTYPE = {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.float8_e4m3fn}
ELEM = {"bf16": 2, "int8": 1, "fp8": 1}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # A tiny decode batch: launch latency.
        dict(name="weights tiny", op="weights", batch=4, heads=8, kv_heads=2, dim=64, block=16,
             dtype="bf16", lo=1, hi=200),
        # One layer of a 70B-like model serving 128 sequences from an INT8 cache.
        dict(name="weights 128x8k int8", op="weights", batch=128, heads=64, kv_heads=8, dim=128,
             block=32, dtype="int8", lo=1024, hi=8192),
        # Speculative verification: five query tokens per sequence.
        dict(name="prompt verify 64x5", op="prompt", batch=64, heads=32, kv_heads=8, dim=128,
             block=16, dtype="bf16", lo=512, hi=4096, queries=5),
        # Whole prompts of four requests.
        dict(name="prompt 4x4k", op="prompt", batch=4, heads=32, kv_heads=8, dim=128, block=16,
             dtype="bf16", lo=1024, hi=4096, queries=0),
        # An 8B-like layer's batch brought back to 1024 tokens per head.
        dict(name="select 64x4k", op="select", batch=64, kv_heads=8, lo=512, hi=4096, budget=1024,
             recent=256),
        # Long contexts brought back to 4096 tokens per head.
        dict(name="select 8x131k", op="select", batch=8, kv_heads=8, lo=32768, hi=131072,
             budget=4096, recent=1024),
        # The rows of the first selection packed in place.
        dict(name="evict 64x1k bf16", op="evict", batch=64, kv_heads=8, dim=128, block=16,
             dtype="bf16", lo=512, hi=4096, budget=1024, recent=256, fresh=False),
        # An E4M3 cache packed into fresh blocks (the old ones are shared).
        dict(name="evict 128x2k fp8", op="evict", batch=128, kv_heads=8, dim=128, block=32,
             dtype="fp8", lo=1024, hi=8192, budget=2048, recent=512, fresh=True),
        # One decode step's append of 128 sequences.
        dict(name="append 128x1 fp8", op="append", batch=128, kv_heads=8, dim=128, block=32,
             dtype="fp8", lo=1024, hi=8192, new=1),
        # The prompts of eight requests.
        dict(name="append 8x8k fp8", op="append", batch=8, kv_heads=8, dim=128, block=16,
             dtype="fp8", lo=1024, hi=8192, new=0),
        # Differential attention: a tiny batch, and an 8B-like layer's batch.
        dict(name="diff tiny", op="diff", batch=4, heads=4, kv_heads=1, dim=64, block=16,
             dtype="bf16", lo=1, hi=200),
        dict(name="diff 64x4k", op="diff", batch=64, heads=16, kv_heads=4, dim=128, block=16,
             dtype="bf16", lo=512, hi=4096),
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
        if _cost(c) <= most:
            return c


def _draw(rng):
    op = rng.choice(("weights", "prompt", "select", "evict", "append", "diff"))
    c = dict(op=op, batch=_log_int(rng, 1, 128), kv_heads=rng.choice((1, 2, 4, 8)))
    hi = _log_int(rng, 64 if op == "select" else 1,
                  131072 if op in ("weights", "select", "diff") else 8192)
    lo = max(1, int(hi * rng.uniform(0.05, 1.0)))
    c.update(lo=lo, hi=hi)
    if op == "select":
        # the longest sequence has tokens to lose
        budget = _log_int(rng, 1, min(int(_lengths(c).max()) * 3 // 4 + 1, 8192))
        c.update(budget=budget, recent=rng.randint(0, budget // 2))
        return c
    c.update(dim=rng.choice((64, 128)), block=rng.choice((16, 32)),
             dtype=rng.choice(("int8", "fp8") if op == "append" else ("bf16", "int8", "fp8")))
    if op == "weights" or op == "prompt":
        c.update(heads=c["kv_heads"] * rng.randint(1, 8))
    if op == "prompt":
        c.update(queries=rng.choice((0, _log_int(rng, 1, 512))))
    if op == "diff":
        c.update(heads=c["kv_heads"] * rng.randint(1, 4))
    if op == "append":
        c.update(new=rng.choice((0, 1, _log_int(rng, 1, 512))))
    if op == "evict":
        budget = _log_int(rng, 1, hi)
        c.update(budget=budget, recent=rng.randint(0, budget), fresh=rng.random() < 0.5)
    return c


def _lengths(case):
    """The batch's lengths, from the case alone (a seed only permutes them)."""
    r = np.random.RandomState([case["batch"], case["lo"], case["hi"]])
    return r.randint(case["lo"], case["hi"] + 1, case["batch"]).astype(np.int64)


def _new_counts(case, L, key):
    """New (query) tokens of each sequence: the last `key` tokens, or all."""
    return L if case[key] == 0 else np.minimum(L, case[key])


def work(case):
    L = _lengths(case)
    op, B, H = case["op"], case["batch"], case["kv_heads"]
    tokens = int(L.sum())
    if op == "select":
        return {"bytes": 4 * H * (tokens + B * case["budget"]) + 8 * B, "flops": 0}
    d, e, bs = case["dim"], ELEM[case["dtype"]], case["block"]
    blocks = int(((L + bs - 1) // bs).sum())
    scales = 0 if e == 2 else 4 * blocks * H                # per tensor
    if op == "weights":
        hq = case["heads"]
        return {"bytes": 2 * tokens * H * d * e + 2 * scales + 4 * blocks + 2 * 4 * H * tokens
                + 4 * B * hq * d, "flops": 4 * tokens * hq * d}
    if op == "prompt":
        hq = case["heads"]
        n = _new_counts(case, L, "queries")
        pairs = int((n * L - n * (n - 1) // 2).sum())
        return {"bytes": tokens * H * d * e + scales + 4 * blocks + 4 * H * (2 * tokens - int(n.sum()))
                + 2 * int(n.sum()) * hq * d, "flops": 2 * pairs * hq * d}
    if op == "evict":
        keep = int(np.minimum(L, case["budget"]).sum())
        kb = int(((np.minimum(L, case["budget"]) + bs - 1) // bs).sum())
        return {"bytes": 4 * keep * H * d * e + (0 if e == 2 else 4 * 4 * kb * H)
                + 12 * keep * H + 4 * blocks, "flops": 0}
    if op == "append":
        n = _new_counts(case, L, "new")
        touched = int(((L + bs - 1) // bs - (L - n) // bs).sum())
        return {"bytes": 2 * int(n.sum()) * H * d * 3 + 4 * 4 * touched * H + 4 * touched, "flops": 0}
    hq = case["heads"]
    return {"bytes": 4 * tokens * H * d * e + 4 * scales + 4 * blocks + 8 * B * hq * d,
            "flops": 12 * tokens * hq * d}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _codes(shape, dtype, g):
    x = torch.randn(shape, device="cuda", generator=g)
    if dtype == "bf16":
        return x.to(torch.bfloat16)
    if dtype == "int8":
        return (x * 32).round().clamp(-127, 127).to(torch.int8)
    return (x * 112).clamp(-448, 448).to(torch.float8_e4m3fn)


def _pool(s, case, heads, total_blocks, g):
    """K and V pools with scales, and a table of randomly placed blocks."""
    dtype = case["dtype"]
    shape = (total_blocks, case["block"], heads, case["dim"])
    s["k_cache"], s["v_cache"] = _codes(shape, dtype, g), _codes(shape, dtype, g)
    s["k_scale"] = s["v_scale"] = None
    if dtype != "bf16":
        unit = 1 / 32 if dtype == "int8" else 1 / 112
        for name in ("k_scale", "v_scale"):
            s[name] = (torch.rand((total_blocks, heads), device="cuda", generator=g) + 0.5) * unit


def _tables(case, L, g, extra=0):
    """int32 tables of randomly placed blocks (padding -1), the pool size, and
    `extra` further blocks per sequence as a second table."""
    bs, B = case["block"], case["batch"]
    nb = (L + bs - 1) // bs
    width = int(nb.max())
    need = int(nb.sum())
    total = int((need + extra * B) * 1.1) + 1
    perm = torch.randperm(total, device="cuda", generator=g, dtype=torch.int32)
    counts = torch.from_numpy(nb).cuda()
    first = torch.cumsum(counts, 0) - counts
    j = torch.arange(width, device="cuda")
    at = first[:, None] + j
    table = torch.where(j < counts[:, None], perm[at.clamp(max=need - 1)], -1).to(torch.int32)
    other = perm[need:need + extra * B].view(B, extra).contiguous() if extra else None
    return table.contiguous(), total, other


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    L = np.random.RandomState(int(seed) % (1 << 31)).permutation(_lengths(case))
    op, B, H = case["op"], case["batch"], case["kv_heads"]
    s = dict(case=case, L=L, max_len=int(L.max()),
             seq_lens=torch.from_numpy(L.astype(np.int32)).cuda())
    if op == "select":
        # accumulated softmax weights: a few heavy tokens, many light ones,
        # some whose weight underflowed to zero
        w = torch.randn((B, H, s["max_len"]), device="cuda", generator=g)
        z = torch.rand((B, H, s["max_len"]), device="cuda", generator=g)
        s["weights"] = torch.where(z < 0.03, 0.0, torch.exp(2.5 * w))
        s["keep_idx"] = torch.empty((B, H, case["budget"]), dtype=torch.int32, device="cuda")
        s["keep_len"] = torch.empty(B, dtype=torch.int32, device="cuda")
        return s
    d = case["dim"]
    heads = 2 * H if op == "diff" else H
    extra = 0
    if op == "evict" and case["fresh"]:
        extra = (min(case["budget"], s["max_len"]) + case["block"] - 1) // case["block"]
    s["tables"], total, s["dst_tables"] = _tables(case, L, g, extra)
    _pool(s, case, heads, total, g)
    s["scale"] = d ** -0.5
    width = s["tables"].shape[1] * case["block"]
    if op in ("weights", "prompt", "evict"):
        # about what one earlier step of as many queries left
        size = case.get("heads", H) / H * max(case.get("queries", 1), 1) / float(L.mean())
        s["weights"] = size * torch.exp(torch.randn((B, H, width), device="cuda", generator=g))
    if op == "weights" or op == "diff":
        rows = case["heads"] * (2 if op == "diff" else 1)
        s["q"] = (2 * torch.randn((B, rows, d), device="cuda", generator=g)).to(torch.bfloat16)
        s["out"] = torch.empty((B, case["heads"], d * rows // case["heads"]), dtype=torch.bfloat16,
                               device="cuda")
        s["workspace"] = torch.empty(B * rows * (s["max_len"] + 1024) * 8, dtype=torch.uint8,
                                     device="cuda")
    if op == "diff":
        s["lam"] = 0.2 + 0.6 * torch.rand(case["heads"], device="cuda", generator=g)
        s["norm_weight"] = 0.2 * (1 + 0.1 * torch.randn(2 * d, device="cuda", generator=g))
    if op in ("prompt", "append"):
        n = _new_counts(case, L, "queries" if op == "prompt" else "new")
        s["n"], s["max_n"], s["T"] = n, int(n.max()), int(n.sum())
        s["query_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
    if op == "prompt":
        s["q"] = (2 * torch.randn((s["T"], case["heads"], d), device="cuda", generator=g)).to(torch.bfloat16)
        s["workspace"] = torch.empty(s["T"] * case["heads"] * 8 * (s["max_len"] // 256 + 2) + 4096,
                                     dtype=torch.uint8, device="cuda")
    if op == "append":
        size = 0.5 + torch.rand((s["T"], H, 1), device="cuda", generator=g)
        s["k"] = (size * torch.randn((s["T"], H, d), device="cuda", generator=g)).to(torch.bfloat16)
        s["v"] = (size * torch.randn((s["T"], H, d), device="cuda", generator=g)).to(torch.bfloat16)
    if op == "evict":
        # what a selection leaves: the last tokens and random others
        t = torch.arange(s["max_len"], device="cuda")
        Ld = s["seq_lens"][:, None, None]
        rank = torch.rand((B, H, s["max_len"]), device="cuda", generator=g)
        rank = torch.where(t >= Ld - case["recent"], 2.0, rank)
        rank = torch.where(t >= Ld, -1.0, rank)
        k = min(case["budget"], s["max_len"])
        s["keep_len"] = s["seq_lens"].clamp(max=k).to(torch.int32)
        idx = torch.topk(rank, k, dim=2).indices
        idx = torch.where(torch.arange(k, device="cuda") < s["keep_len"][:, None, None], idx,
                          1 << 30).sort(dim=2).values
        s["keep_idx"] = torch.where(idx < (1 << 30), idx, -1).to(torch.int32).contiguous()
    return s


# --------------------------------------------------------------------------
# Plain forms (32 bits)
# --------------------------------------------------------------------------

def _gathered(s, name, heads):
    """Every sequence's cached rows as fp32 [B, tokens, heads, dim] (padding
    blocks read block 0)."""
    t = s["tables"].clamp(min=0).long()
    x = s[name + "_cache"][t].float()                                  # [B, MB, bs, H, d]
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][t][:, :, None, :, None]
    B, MB, bs, H, d = x.shape
    return x.view(B, MB * bs, H, d)


def _softmax(scores):
    e = torch.exp(scores - scores.amax(dim=-1, keepdim=True))
    return e / e.sum(dim=-1, keepdim=True)


def _plain_weights(s):
    c = s["case"]
    B, H, d = c["batch"], c["kv_heads"], c["dim"]
    K, V = _gathered(s, "k", H), _gathered(s, "v", H)
    t = torch.arange(K.shape[1], device=K.device)
    q = s["q"].float().view(B, H, -1, d)
    S = torch.einsum("bhgd,bthd->bhgt", q, K) * s["scale"]
    L = s["seq_lens"][:, None, None]
    p = _softmax(S.masked_fill(t >= L[:, :, :, None], -math.inf))
    s["out"].copy_(torch.einsum("bhgt,bthd->bhgd", p, V).view(B, -1, d))
    w = p.sum(dim=2)
    old = s["weights"]
    s["weights"].copy_(torch.where(t < L - 1, old + w, torch.where(t == L - 1, w, old)))
    return s["out"], s["weights"]


def _plain_prompt(s):
    c = s["case"]
    B, H, d = c["batch"], c["kv_heads"], c["dim"]
    K = _gathered(s, "k", H)
    t = torch.arange(K.shape[1], device=K.device)
    i = torch.arange(s["max_n"], device=K.device)
    qs = s["query_start"].long()
    n = (qs[1:] - qs[:-1])[:, None]
    rows = (qs[:-1, None] + i).clamp(max=s["T"] - 1)                   # [B, max_n]
    q = s["q"][rows].float().view(B, -1, H, c["heads"] // H, d)
    S = torch.einsum("bnhgd,bthd->bhgnt", q, K).mul_(s["scale"])
    L = s["seq_lens"].long()[:, None]
    pos = L - n + i                                                    # [B, max_n]
    S.masked_fill_((t > pos[:, :, None])[:, None, None], -math.inf)
    S.sub_(S.amax(dim=-1, keepdim=True)).exp_()
    S.div_(S.sum(dim=-1, keepdim=True))
    S.masked_fill_((i >= n)[:, None, None, :, None], 0.0)
    w = S.sum(dim=(2, 3))
    L, n = L[:, :, None], n[:, :, None]
    old = s["weights"]
    s["weights"].copy_(torch.where(t >= L, old, torch.where(t < L - n, old + w, w)))
    return s["weights"]


def _plain_select(s):
    c, w = s["case"], s["weights"]
    W, budget = w.shape[2], c["budget"]
    t = torch.arange(W, device=w.device, dtype=torch.int32)
    L = s["seq_lens"][:, None, None]
    key = torch.where(torch.isnan(w), -math.inf, w)
    # a stable descending order of the candidates; the recent tokens first,
    # what is past the end last
    key = torch.where(t >= L - c["recent"], math.inf, key)
    order = torch.sort(torch.where(t >= L, -math.inf, key), dim=2, descending=True, stable=True).indices
    rank = torch.empty_like(order)
    rank.scatter_(2, order, torch.arange(W, device=w.device).expand_as(order).contiguous())
    kept = (t < L) & (rank < budget)
    k = min(budget, W)
    idx = torch.where(kept, t, W).sort(dim=2).values[:, :, :k]
    s["keep_idx"].fill_(-1)
    s["keep_idx"][:, :, :k] = torch.where(idx < W, idx, -1)
    s["keep_len"].copy_(s["seq_lens"].clamp(max=budget))
    return s["keep_idx"], s["keep_len"]


def _quantised(x, scale, dtype):
    """Codes of fp32 x under scale (broadcast; 0 reads as 1), as fp32 values."""
    y = x / torch.where(scale == 0, 1.0, scale)
    if dtype == "int8":
        return y.round().clamp(-127, 127)
    return y.clamp(-448, 448).to(torch.float8_e4m3fn).float()


def _scale_of(amax, dtype):
    return amax / torch.full_like(amax, CODE_MAX[dtype])


def _plain_evict(s):
    c = s["case"]
    B, H, bs, dtype = c["batch"], c["kv_heads"], c["block"], c["dtype"]
    dev = s["keep_idx"].device
    k = s["keep_idx"].shape[2]
    J = (k + bs - 1) // bs
    last = (s["keep_len"].long() - 1)[:, None]
    # rows past the last kept one repeat it (the same value to the same place)
    j = torch.minimum(torch.arange(J * bs, device=dev)[None], last)    # [B, J * bs]
    src = torch.gather(s["keep_idx"].long(), 2, j[:, None].expand(B, H, J * bs))
    tab, dst = s["tables"].long(), (s["dst_tables"] if c["fresh"] else s["tables"]).long()
    b = torch.arange(B, device=dev)[:, None, None]
    h = torch.arange(H, device=dev)[None, :, None]
    sblk = tab[b, src // bs]                                           # [B, H, J * bs]
    jb = (j // bs)[:, None].expand(B, H, J * bs)
    dblk = dst[b, jb]
    moved_w = s["weights"][b, h, src]
    stay = ((src == j[:, None]) & (sblk == dblk)).view(B, H, J, bs).all(dim=3)
    outs = []
    for name in ("k", "v"):
        cache, scale = s[name + "_cache"], s[name + "_scale"]
        rows = cache.view(torch.uint8)[sblk, src % bs, h] if dtype == "fp8" else cache[sblk, src % bs, h]
        if dtype != "bf16":
            codes = rows.view(torch.float8_e4m3fn) if dtype == "fp8" else rows
            x = codes.float() * scale[sblk, h][..., None]
            amax = x.abs().view(B, H, J, -1).amax(dim=3)
            new = torch.where(stay, scale[dblk.view(B, H, J, bs)[..., 0], h], _scale_of(amax, dtype))
            new = torch.gather(new, 2, jb)                             # the row's own block's
            y = _quantised(x, new[..., None], dtype)
            y = torch.where(torch.gather(stay, 2, jb)[..., None], codes.float(), y).to(cache.dtype)
            rows = y.view(torch.uint8) if dtype == "fp8" else y
            scale[dblk, h] = new
        (cache.view(torch.uint8) if dtype == "fp8" else cache)[dblk, j[:, None] % bs, h] = rows
        outs += [cache] if scale is None else [cache, scale]
    s["weights"][b, h, j[:, None]] = moved_w
    return outs + [s["weights"]]


def _plain_append(s):
    c = s["case"]
    B, bs, dtype = c["batch"], c["block"], c["dtype"]
    dev = s["seq_lens"].device
    qs, L = s["query_start"].long(), s["seq_lens"].long()
    n = qs[1:] - qs[:-1]
    first = L - n                                                      # first new position
    J = (s["max_n"] + bs - 2) // bs + 1
    # the touched logical blocks; further ones repeat the last
    lb = torch.minimum((first // bs)[:, None] + torch.arange(J, device=dev), ((L - 1) // bs)[:, None])
    pos = lb[:, :, None] * bs + torch.arange(bs, device=dev)           # [B, J, bs]
    is_new = (pos >= first[:, None, None]) & (pos < L[:, None, None])
    is_old = pos < first[:, None, None]
    row = (qs[:-1, None, None] + pos - first[:, None, None]).clamp(0, s["T"] - 1)
    blk = s["tables"].long()[torch.arange(B, device=dev)[:, None], lb]  # [B, J]
    opened = is_new[:, :, 0, None]                                     # row 0 is new
    outs = []
    for name in ("k", "v"):
        cache, scale = s[name + "_cache"], s[name + "_scale"]
        raw = cache.view(torch.uint8)[blk].view(cache.dtype)           # [B, J, bs, H, d]
        x = s[name][row].float()
        amax = torch.where(is_new[..., None, None], x.abs(), 0.0).amax(dim=(2, 4))
        old = scale[blk]                                               # [B, J, H]
        new = torch.maximum(torch.where(opened, 0.0, old), _scale_of(amax, dtype))
        grown = (new > old)[:, :, None, :, None] & is_old[..., None, None]
        sc, so = new[:, :, None, :, None], old[:, :, None, :, None]
        codes = raw.float()
        y = torch.where(grown, _quantised(codes * so, sc, dtype), codes)
        y = torch.where(is_new[..., None, None], _quantised(x, sc, dtype), y).to(cache.dtype)
        cache.view(torch.uint8)[blk] = y.view(torch.uint8)
        scale[blk] = new
        outs += [cache, scale]
    return outs


def _plain_diff(s):
    c = s["case"]
    B, H, d = c["batch"], c["kv_heads"], c["dim"]
    K, V = _gathered(s, "k", 2 * H), _gathered(s, "v", 2 * H)
    T = K.shape[1]
    t = torch.arange(T, device=K.device)
    q = s["q"].float().view(B, H, -1, 2, d)
    S = torch.einsum("bhgmd,bthmd->bhgmt", q, K.view(B, T, H, 2, d)) * s["scale"]
    p = _softmax(S.masked_fill(t >= s["seq_lens"][:, None, None, None, None], -math.inf))
    a = torch.einsum("bhgmt,bthd->bhgmd", p, V.view(B, T, H, 2 * d))
    y = a[..., 0, :] - s["lam"].view(1, H, -1, 1) * a[..., 1, :]
    y = y / torch.sqrt((y * y).mean(dim=-1, keepdim=True) + 1e-5) * s["norm_weight"]
    s["out"].copy_(y.reshape(B, -1, 2 * d))
    return s["out"]


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"weights": _plain_weights, "prompt": _plain_prompt, "select": _plain_select,
                "evict": _plain_evict, "append": _plain_append, "diff": _plain_diff}[op](s)
    import paged_kv_cache_97_gb300 as pkv
    if op == "weights":
        pkv.paged_attention_decode_weights(
            s["out"], s["weights"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["seq_lens"],
            s["max_len"], s["scale"], s["workspace"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["out"], s["weights"]
    if op == "prompt":
        pkv.attention_weights(s["weights"], s["q"], s["k_cache"], s["tables"], s["seq_lens"],
                              s["query_start"], s["max_len"], s["max_n"], s["scale"],
                              s["workspace"], k_scale=s["k_scale"])
        return s["weights"]
    if op == "select":
        pkv.select_tokens(s["keep_idx"], s["keep_len"], s["weights"], s["seq_lens"], s["max_len"],
                          s["case"]["recent"])
        return s["keep_idx"], s["keep_len"]
    if op == "evict":
        pkv.evict_tokens(s["k_cache"], s["v_cache"], s["tables"], s["seq_lens"], s["keep_idx"],
                         s["keep_len"], dst_block_tables=s["dst_tables"], weights=s["weights"],
                         k_scale=s["k_scale"], v_scale=s["v_scale"])
        if s["k_scale"] is None:
            return [s["k_cache"], s["v_cache"], s["weights"]]
        return [s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"], s["weights"]]
    if op == "append":
        pkv.append_scaled(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                          s["tables"], s["seq_lens"], s["query_start"], s["max_n"])
        return [s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"]]
    pkv.paged_diff_attention_decode(
        s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["seq_lens"], s["max_len"],
        s["scale"], s["lam"], norm_weight=s["norm_weight"], eps=1e-5, workspace=s["workspace"],
        k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s["out"]


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def _seq64(s, name, b, head):
    """Sequence b's cached rows of one pool head, [L, dim] in 64 bits."""
    L, bs = int(s["L"][b]), s["case"]["block"]
    ids = s["tables"][b, :(L + bs - 1) // bs].long()
    x = s[name + "_cache"][ids, :, head].double()
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][ids, head].double()[:, None, None]
    return x.reshape(-1, x.shape[-1])[:L]


def _round64(x, scale, dtype):
    """The stored code values of 64-bit x: the quotient by the scale (0 reads
    as 1) is a 32-bit number, then the nearest code, ties to even."""
    y = (x / torch.where(scale == 0, torch.ones_like(scale), scale)).float().double()
    if dtype == "int8":
        return torch.round(y).clamp(-127, 127)
    # spacing 2^(e - 4) of |y| in [2^(e-1), 2^e), no finer than the subnormals' 2^-9
    power = torch.tensor([2.0 ** e for e in range(-9, 6)], dtype=torch.float64, device=y.device)
    step = power[(torch.frexp(y).exponent.long().clamp(-5, 9) + 5)]
    return (torch.round(y / step) * step).clamp(-448, 448)


def _exact_attention(s, case):
    B, H, op = case["batch"], case["kv_heads"], case["op"]
    G = case["heads"] // H
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if op == "weights" else None
    for b in range(B):
        L = int(s["L"][b])
        for h in range(H):
            q = s["q"][b].double()
            if op == "weights":
                S = q[h * G:(h + 1) * G] @ _seq64(s, "k", b, h).T * s["scale"]
                p = torch.softmax(S, dim=-1)
                out[b, h * G:(h + 1) * G] = p @ _seq64(s, "v", b, h)
                weights[b, h, L - 1] = 0
                weights[b, h, :L] += p.sum(dim=0)
                continue
            q = q[2 * h * G:2 * (h + 1) * G].view(G, 2, -1)
            V = torch.cat([_seq64(s, "v", b, 2 * h), _seq64(s, "v", b, 2 * h + 1)], dim=1)
            a1, a2 = (torch.softmax(q[:, m] @ _seq64(s, "k", b, 2 * h + m).T * s["scale"], dim=-1) @ V
                      for m in (0, 1))
            y = a1 - s["lam"][h * G:(h + 1) * G, None].double() * a2
            out[b, h * G:(h + 1) * G] = (y * torch.rsqrt((y ** 2).mean(dim=-1, keepdim=True) + 1e-5)
                                         * s["norm_weight"].double())
    return (out, weights) if op == "weights" else out


def _exact_prompt(s, case):
    H = case["kv_heads"]
    G = case["heads"] // H
    weights = s["weights"].double()
    start = np.concatenate([[0], np.cumsum(s["n"])])
    for b in range(case["batch"]):
        L, n = int(s["L"][b]), int(s["n"][b])
        for h in range(H):
            K = _seq64(s, "k", b, h)
            acc = torch.zeros(L, dtype=torch.float64, device="cuda")
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                q = s["q"][start[b] + i:start[b] + i + m, h * G:(h + 1) * G].double()
                S = torch.einsum("ngd,td->gnt", q, K) * s["scale"]
                pos = L - n + i + torch.arange(m, device="cuda")
                S.masked_fill_(torch.arange(L, device="cuda") > pos[:, None], -math.inf)
                acc += torch.softmax(S, dim=-1).sum(dim=(0, 1))
            weights[b, h, L - n:L] = 0
            weights[b, h, :L] += acc
    return weights


def _exact_select(s, case):
    budget, recent = case["budget"], case["recent"]
    idx = np.full(tuple(s["keep_idx"].shape), -1, np.int32)
    w = s["weights"].double().cpu().numpy()
    for b in range(case["batch"]):
        L = int(s["L"][b])
        for h in range(case["kv_heads"]):
            if L <= budget:
                keep = np.arange(L)
            else:
                heavy = np.argsort(-w[b, h, :L - recent], kind="stable")[:budget - recent]
                keep = np.sort(np.concatenate([heavy, np.arange(L - recent, L)]))
            idx[b, h, :len(keep)] = keep
    return torch.from_numpy(idx), torch.from_numpy(np.minimum(s["L"], budget).astype(np.int32))


def _exact_evict(s, case):
    bs, H, dtype = case["block"], case["kv_heads"], case["dtype"]
    pools = {n: s[n + "_cache"].double() for n in ("k", "v")}
    scales = {n: None if s[n + "_scale"] is None else s[n + "_scale"].double() for n in ("k", "v")}
    weights = s["weights"].double()
    dst = s["dst_tables"] if case["fresh"] else s["tables"]
    heads = torch.arange(H, device="cuda")[:, None]
    for b in range(case["batch"]):
        m = int(s["keep_len"][b])
        src = s["keep_idx"][b, :, :m].long()                           # [H, m]
        sb, db = s["tables"][b].long()[src // bs], dst[b, torch.arange(m, device="cuda") // bs].long()
        weights[b, :, :m] = s["weights"][b].double().gather(1, src)
        for n in ("k", "v"):
            rows = s[n + "_cache"].view(torch.uint8 if dtype == "fp8" else s[n + "_cache"].dtype)
            x = rows[sb, src % bs, heads].view(s[n + "_cache"].dtype).double()
            to = (db.expand(H, m), (torch.arange(m, device="cuda") % bs).expand(H, m), heads)
            if dtype == "bf16":
                pools[n][to] = x
                continue
            value = (x * s[n + "_scale"][sb, heads].double()[..., None]).float().double()
            for j in range(0, m, bs):
                part = slice(j, min(j + bs, m))
                block = db[j]
                same = (src[:, part] == torch.arange(part.start, part.stop, device="cuda")).all(dim=1)
                same &= s["tables"][b, j // bs] == block
                new = (value[:, part].abs().amax(dim=(1, 2)) / CODE_MAX[dtype]).float().double()
                new = torch.where(same, s[n + "_scale"][block].double(), new)
                scales[n][block] = new
                y = _round64(value[:, part], new[:, None, None], dtype)
                x[:, part] = torch.where(same[:, None, None], x[:, part], y)
            pools[n][to] = x
    if dtype == "bf16":
        return [pools["k"], pools["v"], weights]
    if dtype == "int8":
        pools = {n: p.to(torch.int8) for n, p in pools.items()}
    return [pools["k"], scales["k"], pools["v"], scales["v"], weights]


def _exact_append(s, case):
    bs, dtype = case["block"], case["dtype"]
    outs = []
    start = np.concatenate([[0], np.cumsum(s["n"])])
    for n in ("k", "v"):
        pool, scale = s[n + "_cache"].double(), s[n + "_scale"].double()
        for b in range(case["batch"]):
            L, m = int(s["L"][b]), int(s["n"][b])
            x = s[n][int(start[b]):int(start[b]) + m].double()
            for j in range((L - m) // bs, (L + bs - 1) // bs):
                block = int(s["tables"][b, j])
                r0, r1 = max(L - m - j * bs, 0), min(L - j * bs, bs)
                rows = x[j * bs + r0 - (L - m):j * bs + r1 - (L - m)]
                before = scale[block].clone()
                new = (rows.abs().amax(dim=(0, 2)) / CODE_MAX[dtype]).float().double()
                if r0 > 0:
                    new = torch.maximum(new, before)
                    value = (pool[block, :r0] * before[:, None]).float().double()
                    again = _round64(value, new[:, None], dtype)
                    pool[block, :r0] = torch.where((new > before)[:, None], again, pool[block, :r0])
                pool[block, r0:r1] = _round64(rows, new[:, None], dtype)
                scale[block] = new
        outs += [pool.to(torch.int8) if dtype == "int8" else pool, scale]
    return outs


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prompt" and work(case)["flops"] > 4e12:
        return None
    if op in ("weights", "diff"):
        return _exact_attention(s, case)
    return {"prompt": _exact_prompt, "select": _exact_select, "evict": _exact_evict,
            "append": _exact_append}[op](s, case)
