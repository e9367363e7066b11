"""The rotated append, the 4-bit pool and the verification of drafts at the
borders of their forms: clusters that start apart, more rounds than have sums of
their own, constant rows of large values, queries of far smaller magnitude,
8-bit codes of awkward values and scales, captured steps and streams.  References
and tolerances are those of test_gpu_q4."""
import math

import pytest
import torch

import q4_reference as ref
from test_gpu_q4 import (Step, check, check_verify, clean_status, decode, flags_of, multi, pkv, poison, run_verify,
                         same_bits, starts, verify_case, within)  # noqa: F401

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------
# Verification of drafts
# --------------------------------------------------------------------------

def test_verify_clusters_start_apart(pkv):
    """Clusters of eight CTAs that find the GPU full, beside another stream's and one
    after the other, so that a cluster's CTAs begin at different times: rows so
    short that a CTA has its sum at once."""
    cases = [verify_case([1] * 60, 16384, torch.bfloat16, 40 + i) for i in range(2)]
    want = [ref.verify(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    dev = [[x.cuda() for x in c] for c in cases]
    outs = [[torch.full((60,), 77, dtype=torch.int32, device="cuda") for _ in range(30)] for _ in cases]
    acc = [torch.empty(60, dtype=torch.int32, device="cuda") for _ in cases]
    torch.cuda.synchronize()
    for r in range(30):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                pkv.verify_drafts(outs[i][r], acc[i], *dev[i])
    torch.cuda.synchronize()
    for i in range(2):
        lo, hi = (torch.tensor([z[k] for _, z in want[i]]) for k in range(2))
        for out in outs[i]:
            assert ((lo <= out.cpu()) & (out.cpu() <= hi)).all()
            assert same_bits(out, outs[i][0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,V,shift", [(320, 151665, 0), (310, 300001, 0), (200, 300001, 0), (310, 150016, 1)])
def test_verify_more_rounds_than_sums(pkv, dtype, B, V, shift):
    """Rows read one element a load by few warps: a warp takes more rounds than it
    keeps sums of.  The weight lies in the last elements of a warp's part, of
    the row, and everywhere; a row's base may be off 16 bytes."""
    g = torch.Generator().manual_seed(V + B)
    u = torch.rand(B, generator=g)
    warps = 8 if B > 304 else 16
    per = -(-(-(-V // warps)) // 32) * 32
    want = torch.empty(B, 2, dtype=torch.long)
    flat = torch.zeros(B * V + 8, dtype=dtype, device="cuda")
    p = flat[shift:shift + B * V].view(B, V)
    for b in range(B):
        kind, warp = b % 4, b // 4 % warps
        end = min((warp + 1) * per, V)
        if kind == 0:                               # the warp's last elements
            at, size = end - 40, 40
        elif kind == 1:                             # the last of all
            at, size = V - 3, 3
        elif kind == 2:                             # around the 64th round and after
            at, size = min(warp * per + 64 * 256 - 5, V - 600), 600
        else:
            at, size = 0, V
        w = torch.rand(size, generator=g).to(dtype)
        p[b, at:at + size] = w.cuda()
        total = w.double().cumsum(0).numpy()
        off = size * 2.0 ** -45 + 2.0 ** -50
        goal = float(u[b]) * total[-1]
        for k, s in enumerate((-off, off)):
            want[b, k] = at + min(int(total.searchsorted(goal + s, side="right")), size - 1)
    tokens = torch.zeros(B, dtype=torch.int32, device="cuda")
    out, acc = (torch.full((B,), 77777777, dtype=torch.int32, device="cuda") for _ in "oa")
    pkv.verify_drafts(out, acc, tokens, p, None, u.cuda(), starts([1] * B).cuda(), max_query_len=1)
    got = out.cpu().long()
    assert (got < V).all()
    assert ((want[:, 0] <= got) & (got <= want[:, 1])).all()
    assert (acc == 0).all()


# --------------------------------------------------------------------------
# Attention over the 4-bit pool
# --------------------------------------------------------------------------

def appended(pkv, k, v, block):
    """A 4-bit pool that holds rows k, v [L, H, d] of one sequence: (pool, tables, lengths, reference rows)."""
    L, H, d = k.shape
    nb = (L + block - 1) // block
    kv = torch.full((nb, H, ref.record_bytes(block, d)), 0xFF, dtype=torch.uint8, device="cuda")
    bt = torch.arange(nb, dtype=torch.int32, device="cuda")[None].contiguous()
    sl = torch.tensor([L], dtype=torch.int32, device="cuda")
    pkv.append_rotary_q4(None, None, k.cuda(), v.cuda(), kv, None, bt, sl, block,
                         query_start=torch.tensor([0, L], dtype=torch.int32, device="cuda"), max_query_len=L)
    return kv, bt, sl, ref.rows_of(kv.cpu(), block, d, L)


@pytest.mark.parametrize("block,dim", [(16, 64), (32, 128)])
@pytest.mark.parametrize("n,room", [(1, 0), (3, 0), (40, 0), (40, 1)])
@pytest.mark.parametrize("size", [2.0 ** 97, -2.0 ** 110, 2.0 ** 122, -2.0 ** 125])
@pytest.mark.parametrize("rest", [0.0, 1.0])
def test_constant_rows_of_large_values(pkv, block, dim, n, room, size, rest):
    """V's rows of one value each (the least scale, the value as minimum) that come
    after ordinary ones: a weight times the minimum stays within fp32."""
    L, H, G = 500, 2, 4                             # (four steps a warp)
    g = torch.Generator().manual_seed(n)
    k, v = (torch.randn((L, H, dim), generator=g).to(torch.bfloat16) for _ in "kv")
    v = (v.float() * rest).to(torch.bfloat16)
    v[250:] = size
    v[260:350] = 0.0
    q = torch.randn((n, H * G, dim), generator=g).to(torch.bfloat16)
    kv, bt, sl, rows = appended(pkv, k, v, block)
    want, tol = ref.attention(rows, q, dim ** -0.5, torch.arange(L - n, L), wide=room > 0)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    if n == 1:
        pkv.paged_attention_decode_q4(out, q.cuda(), kv, bt, sl, block, L, dim ** -0.5,
                                      poison(pkv.q4_workspace_bytes(H * G, H, dim)))
    else:
        size = (pkv.q4_long_workspace_bytes(1, n, n, L, H * G, H, dim) if room else
                pkv.q4_workspace_bytes(H * G, H, dim, n))
        pkv.paged_attention_multi_q4(out, q.cuda(), kv, bt, sl, starts([n]).cuda(), block, L, n, dim ** -0.5,
                                     poison(size))
    within(out, want, tol)


@pytest.mark.parametrize("n", [1, 5])
def test_queries_exact_down_to_their_bound(pkv, n):
    """Elements of q of 2^-27 of the largest (which is the least of its octave) that
    meet keys of 2^27 enter exactly, high nibbles as well: tokens whose keys lie in the
    odd elements and ones whose keys lie in the even ones have nearly equal scores, and
    the odd elements' last bit is 2^-7 of theirs."""
    L, d = n + 5, 128
    k = torch.zeros((L, 1, d))
    k[::2, :, 65::2], k[1::2, :, 64::2] = 3 * 2.0 ** 27, 3 * 2.0 ** 27
    v = torch.randn((L, 1, d), generator=torch.Generator().manual_seed(50))
    kv, bt, sl, rows = appended(pkv, k.to(torch.bfloat16), v.to(torch.bfloat16), 16)
    q = torch.zeros((n, 4, d), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    q[..., 64:] = 2.0 ** -27 * (1 + 2.0 ** -7)
    want, tol = ref.attention(rows, q, 1.0, torch.arange(L - n, L))
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = poison(pkv.q4_workspace_bytes(4, 1, d, n))
    if n == 1:
        pkv.paged_attention_decode_q4(out, q.cuda(), kv, bt, sl, 16, L, 1.0, ws)
    else:
        pkv.paged_attention_multi_q4(out, q.cuda(), kv, bt, sl, starts([n]).cuda(), 16, L, n, 1.0, ws)
    within(out, want, tol)


@pytest.mark.parametrize("n,room", [(1, None), (3, None), (40, -1)])
@pytest.mark.parametrize("size", [2.0 ** -122, 2.0 ** -100, 2.0 ** 118, 2.0 ** 125, 1.5 * 2.0 ** 127])
def test_queries_of_any_magnitude(pkv, n, room, size):
    """Queries down to the smallest and up to the largest bf16 numbers, with keys and a
    factor to match."""
    pool = ref.Pool4([300], 2, 64, 16, seed=51, kscale=lambda s, g: 2.0 ** (-60 if size > 1 else 60))
    q = (pool.randn(n, 8, 64).float().clamp(-1.9, 1.9) * (size / 4)).to(torch.bfloat16)
    q[..., 0] = size
    scale = 2.0 ** (60 if size > 1 else -60) / size
    got = decode(pkv, pool, q, scale) if n == 1 else multi(pkv, pool, q, [n], scale, room=room)
    check(got, pool, q, [n], scale, wide=True)


# --------------------------------------------------------------------------
# Appends
# --------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
def test_append_rotary_8_bit_borders(pkv, kind, dim):
    """Values and scales at the borders of the 8-bit codes: what reshape_and_cache
    stores, bit for bit."""
    g = torch.Generator().manual_seed(60)
    special = [0.0, -0.0, math.nan, -math.nan, math.inf, -math.inf, 3.3e38, -3.3e38, 1e-40, -1e-40, 448.0, 464.0, 465.0,
               127.0, 127.5, -128.0, 2.0 ** 40, -2.0 ** 40, 2.0 ** 41, 2.0 ** -9, 2.0 ** -10, 0.5, 1.5, 2.5, 17.0, -33.0]
    scales = [0.0, 1.0, 1e-45, 1e-38, 2.0 ** -81, 2.0 ** -80, 2.0 ** -40, 1 / 40, 3.0, 2.0 ** 40, 2.0 ** 80, 2.0 ** 81,
              3e38, math.inf, math.nan, -1.0, -0.0]
    H, n = 2, 3 * len(scales)
    x = torch.randn((2, n * 16, H, dim), generator=g)
    x *= torch.exp2(torch.randint(-45, 46, x.shape[:-1] + (1,), generator=g).float())
    x[:, ::4] = torch.tensor(special)[torch.randint(0, len(special), x[:, ::4].shape, generator=g)]
    s = torch.tensor(scales).repeat(3)[:, None].expand(n, H).contiguous()
    x[:, 1::4] = torch.randn(x[:, 1::4].shape, generator=g) * 40 * s.nan_to_num(1.0, 1.0).abs().clamp(1e-38, 1e36).repeat_interleave(16, 0)[None, 1::4, :, None]
    k, v = x.to(torch.bfloat16)
    dt = torch.int8 if kind == "int8" else torch.float8_e4m3fn
    caches = [torch.zeros((n, 16, H, dim), dtype=dt, device="cuda") for _ in range(4)]
    ks, vs = s.cuda(), s.flip(0).contiguous().cuda()
    bt = torch.arange(n, dtype=torch.int32, device="cuda").view(3, -1).contiguous()
    sl = torch.full((3,), n * 16 // 3, dtype=torch.int32, device="cuda")
    pkv.append_rotary(None, None, k.contiguous().cuda(), v.contiguous().cuda(), caches[0], caches[1], None, bt, sl,
                      query_start=starts([n * 16 // 3] * 3).cuda(), max_query_len=n * 16 // 3, k_scale=ks, v_scale=vs)
    slots = torch.arange(n * 16, device="cuda")
    pkv.reshape_and_cache(k.contiguous().cuda(), v.contiguous().cuda(), caches[2], caches[3], slots, ks, vs)
    for i in range(2):
        a, b = (c.cpu().view(torch.uint8) for c in (caches[i], caches[i + 2]))
        off = (a != b).nonzero()
        assert len(off) == 0, f"{len(off)} codes differ, first at {off[0].tolist()}"


def test_append_refuses_other_things(pkv):
    """What is no tensor, or has too few dimensions, is named, as everywhere."""
    bt, sl = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((2, 2), (2,)))
    kv = torch.zeros((4, 2, ref.record_bytes(16, 64)), dtype=torch.uint8, device="cuda")
    pool = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 8, 64), dtype=torch.bfloat16, device="cuda")
    rows = q[:, :2].contiguous()
    for name, at in (("q_out", 0), ("q", 1), ("k", 2), ("v", 3)):
        for bad, error in ((None, (TypeError, ValueError)), (3, TypeError), ("x", TypeError),
                           (torch.zeros(128, dtype=torch.bfloat16, device="cuda"), ValueError),
                           (torch.zeros((2, 2, 64), device="cuda"), TypeError), (rows.cpu(), ValueError)):
            args = [q.clone(), q, rows, rows]
            args[at] = bad
            with pytest.raises(error, match=name):
                pkv.append_rotary(*args, pool, pool.clone(), None, bt, sl)
            with pytest.raises(error, match=name):
                pkv.append_rotary_q4(*args, kv, None, bt, sl, 16)


# --------------------------------------------------------------------------
# Graphs and streams
# --------------------------------------------------------------------------

def test_long_queries_on_streams_and_in_graphs(pkv):
    """Plan, images, prompts and short queries: on two streams at once (a workspace
    each), and two captured calls that share one workspace, replayed in turn."""
    L, n = [700, 40, 900, 300], [600, 1, 200, 33]
    pool = ref.Pool4(L, 2, 128, 16, seed=70)
    dev = kv, bt, sl = pool.on()
    q = pool.randn(sum(n), 8, 128)
    first = multi(pkv, pool, q, n, 0.1, dev=dev, room=-1)
    check(first, pool, q, n, 0.1, wide=True)
    other_n = [1, 40, 128, 300]
    second = multi(pkv, pool, q[:sum(other_n)], other_n, 0.1, dev=dev, room=-1)
    qd, size = q.cuda(), pkv.q4_long_workspace_bytes(4, sum(n), 600, 900, 8, 2, 128)

    def call(out, m, ws):
        T = sum(m)
        pkv.paged_attention_multi_q4(out[:T], qd[:T], kv, bt, sl, qs[tuple(m)], 16, 900, 600, 0.1, ws)
    qs = {tuple(m): starts(m).cuda() for m in (n, other_n)}
    outs, wss = [torch.empty_like(qd) for _ in range(2)], [poison(size) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for out, ws, st in zip(outs, wss, streams):
            with torch.cuda.stream(st):
                call(out, n, ws)
    torch.cuda.synchronize()
    assert all(same_bits(o, first) for o in outs)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, out, m in zip(graphs, outs, (n, other_n)):
        with torch.cuda.graph(g):
            call(out, m, wss[0])
    for _ in range(4):
        for g, out, m, want in zip(graphs, outs, (n, other_n), (first, second)):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert same_bits(out[:sum(m)], want)


def test_a_captured_step(pkv):
    """Append, attention, read back and verification captured as one step, replayed on
    new inputs in the same buffers; the eager calls give the same bits."""
    B, n, hq, hkv, d, bs, V = 5, 4, 8, 2, 128, 16, 32000
    T = B * n
    kv = torch.zeros((40, hkv, ref.record_bytes(bs, d)), dtype=torch.uint8, device="cuda")
    bt = torch.randperm(40, generator=torch.Generator().manual_seed(1))[:B * 8].view(B, 8).to(torch.int32).cuda()
    cs, qs = ref.table(200, d).cuda(), starts([n] * B).cuda()
    sl = torch.tensor([4, 17, 64, 100, 128], dtype=torch.int32, device="cuda")
    x = torch.zeros((T, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    tokens, p, r, u, _ = [y.cuda() for y in verify_case([n] * B, V, torch.bfloat16, 80)]
    ws = poison(pkv.q4_workspace_bytes(hq, hkv, d, n))

    def step(kv, new):
        q, out = (torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda") for _ in "qo")
        rows = [torch.empty((T, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        got, acc = (torch.empty(m, dtype=torch.int32, device="cuda") for m in (T, B))
        pkv.append_rotary_q4(q, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], kv, cs, bt, sl, bs, query_start=qs,
                             max_query_len=n)
        pkv.paged_attention_multi_q4(out, q, kv, bt, sl, qs, bs, 128, n, d ** -0.5, ws)
        pkv.read_q4(*rows, kv, bt, sl, bs, query_start=qs, max_query_len=n)
        pkv.verify_drafts(got, acc, tokens, p, r, u, qs, max_query_len=n, seq_lens=sl, new_lens=new)
        return q, out, *rows, got, acc, new
    step(kv, torch.empty_like(sl))                  # (first use outside of a capture)
    kept = kv.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    new = torch.empty_like(sl)
    with torch.cuda.graph(g):
        captured = step(kv, new)
    for seed in range(4):
        gen = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(x.shape, generator=gen))
        u.copy_(torch.rand(T, generator=gen))
        eager = [y.clone() for y in step(kept, torch.empty_like(sl))]
        for y in captured:
            y.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert same_bits(kv, kept) and all(same_bits(a, b) for a, b in zip(captured, eager))


def test_verify_draft_probabilities_of_no_draft(pkv):
    """draft_probs of no row (every sequence has its last token alone): a sequence
    that has a draft all the same, or no token, is a bad one."""
    p = torch.full((2, 64), 1 / 64, device="cuda")
    tokens = torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    none, u = p[:0], torch.tensor([0.5, 0.25], device="cuda")
    out, acc = (torch.full((2,), 77, dtype=torch.int32, device="cuda") for _ in "oa")
    pkv.verify_drafts(out, acc, tokens, p, none, u, starts([1, 1]).cuda())
    assert out.tolist() == [32, 16] and acc.tolist() == [0, 0]
    pkv.verify_drafts(out, acc, tokens, p, none, u, starts([2, 0]).cuda())
    assert flags_of(pkv) == pkv.FLAG_BAD_SEQ_LEN
    assert out.tolist() == [-1, -1] and acc.tolist() == [0, 0]


@pytest.mark.parametrize("dim,heads,group,L,n", [(128, 1, 4, [9000, 300], [200, 64]), (64, 1, 2, [5000], [1500]),
                                                 (128, 2, 8, [4097, 33, 2500], [16, 1, 130])])
def test_long_queries_over_long_contexts(pkv, dim, heads, group, L, n):
    pool = ref.Pool4(L, heads, dim, 16, seed=71)
    q = pool.randn(sum(n), heads * group, dim, scale=2.0)
    check(multi(pkv, pool, q, n, dim ** -0.5, room=-1), pool, q, n, dim ** -0.5, wide=True)
