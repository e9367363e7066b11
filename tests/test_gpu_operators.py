"""GPU parity of the operators around the paged decode attention against
their 64-bit references: attention weights, token selection, eviction,
self-scaling append and differential attention.  Whole numbers, codes, scales
and moved rows are compared exactly; the tolerances of the others are the
reference's own bounds (operator_reference.softmax_bound)."""
import numpy as np
import pytest
import torch

import operator_reference as ref

pytestmark = pytest.mark.gpu

POOLS = [("bf16", 16, 64), ("bf16", 32, 128), ("int8", 16, 128), ("int8", 32, 64), ("fp8", 16, 64),
         ("fp8", 32, 128), ("bf16", 16, 128), ("int8", 32, 128), ("fp8", 16, 128)]


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_97_gb300 as pkv
    pkv.load()
    return pkv


@pytest.fixture(autouse=True)
def clean_status(pkv):
    """Every test starts and (unless it reads the flags itself) ends with a
    clear status word."""
    pkv.get_status()
    yield
    st, flags = pkv.get_status()
    assert flags == 0, f"status word 0x{flags:x}"


def same_bits(got, want):
    a, b = got.cpu().contiguous(), want.contiguous()
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def within(got, want, tol):
    off = (got.cpu().double() - want).abs()
    assert torch.isfinite(off).all()
    worst = (off / (tol + 1e-300)).max().item()
    assert (off <= tol).all(), f"{worst:.2f} of the bound"


def workspace(n):
    # poisoned: what a call does not write it must not read
    return torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")


def decode_weights(pkv, pool, q, weights, scale, max_len=None, ws=None):
    k, v, sc, bt, sl = pool.on()
    max_len = max_len or max(max(pool.L), 1)
    B, hq, d = q.shape
    if ws is None:
        ws = workspace(pkv.weights_workspace_bytes(B, hq, d, max_len, pool.block))
    out = torch.full((B, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    w = weights.cuda()
    pkv.paged_attention_decode_weights(out, w, q.cuda(), k, v, bt, sl, max_len, scale, ws, **sc)
    return out, w


# --------------------------------------------------------------------------
# Decode attention with weights
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,block,dim", POOLS)
@pytest.mark.parametrize("group", [1, 3, 4, 8])
def test_decode_weights(pkv, dtype, block, dim, group):
    L = [1, 2, block - 1, block, block + 1, 100, 257]
    pool = ref.Pool(L, 2, dim, block, dtype, seed=group)
    q = pool.randn(len(L), 2 * group, dim, scale=2.0)
    weights = torch.rand((len(L), 2, 301), generator=pool.g) * group / 50
    out, w = decode_weights(pkv, pool, q, weights, dim ** -0.5)
    want, tol, ww, wtol = ref.decode_weights(pool, q, weights, dim ** -0.5)
    within(out, want, tol)
    within(w, ww, wtol)
    for b, n in enumerate(L):
        assert same_bits(w[b, :, n:], weights[b, :, n:])


@pytest.mark.parametrize("dtype,L", [("bf16", [1500, 700, 256, 255]), ("int8", [2049, 513]),
                                     ("fp8", [1025, 3])])
def test_decode_weights_partitions(pkv, dtype, L):
    """Sequences of several partitions beside ones that fit one."""
    pool = ref.Pool(L, 1, 128, 16, dtype, seed=5, width=160)
    q = pool.randn(len(L), 4, 128, scale=2.0)
    weights = torch.full((len(L), 1, max(L)), float("nan"))
    for b, n in enumerate(L):
        weights[b, :, :n - 1] = torch.rand(n - 1, generator=pool.g)   # the last entry is not read
    out, w = decode_weights(pkv, pool, q, weights, 128 ** -0.5)
    want, tol, ww, wtol = ref.decode_weights(pool, q, torch.nan_to_num(weights), 128 ** -0.5)
    within(out, want, tol)
    for b, n in enumerate(L):
        within(w[b, :, :n], ww[b, :, :n], wtol[b, :, :n])
        assert torch.isnan(w[b, :, n:]).all()


def test_decode_weights_output_is_the_decode_attention(pkv):
    """The same output bits as paged_attention_decode on a bf16 pool, and
    weights that sum to the group size."""
    L = [700, 33, 256]
    pool = ref.Pool(L, 2, 128, 16, "bf16", seed=7)
    q = pool.randn(3, 8, 128, scale=2.0)
    out, w = decode_weights(pkv, pool, q, torch.zeros(3, 2, 700), 128 ** -0.5)
    k, v, sc, bt, sl = pool.on()
    plain = torch.empty_like(out)
    pkv.paged_attention_decode(plain, q.cuda(), k, v, bt, sl, 700, 128 ** -0.5,
                               workspace(pkv.workspace_bytes(3, 8, 128, 700, 16)))
    assert same_bits(out, plain.cpu())
    total = w.double().sum(dim=2).cpu()
    assert (total - 4).abs().max() <= 4 * 2.0 ** -17       # 700 weights, each with a relative error of 2^-18


@pytest.mark.parametrize("dtype", ["bf16", "int8", "fp8"])
def test_decode_weights_add_up_small_ones(pkv, dtype):
    """Weights of 2^-24.1 from each of eight heads, on entries of 1: none alone
    changes the entry, their sum 2^-21.1 does.  (One rounding of the sum, 2^-24
    of the entry, is within the bound's 2^-22.)"""
    pool = ref.Pool([600, 40], 1, 64, 16, dtype, seed=1)
    ref.raw(pool.k)[:] = 0
    one = {"bf16": 0x3F80, "int8": 1, "fp8": 0x38}[dtype]
    for b in (0, 1):
        k = pool.k.view(torch.int16) if dtype == "bf16" else ref.raw(pool.k)
        k[pool.tables[b, 0].item(), 3, 0, 0] = one
    if dtype != "bf16":
        pool.k_scale[:] = 1.0
    q = torch.zeros((2, 8, 64), dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    weights = torch.ones((2, 1, 600))
    scale = 24.1 * 0.6931471805599453
    out, w = decode_weights(pkv, pool, q, weights, scale)
    want, tol, ww, wtol = ref.decode_weights(pool, q, weights, scale)
    assert abs(ww[0, 0, 100].item() - 1 - 2.0 ** -21.1) < 2.0 ** -24
    within(w[0], ww[0], wtol[0])
    within(w[1, :, :40], ww[1, :, :40], wtol[1, :, :40])


def test_decode_weights_shared_blocks(pkv):
    """Sequences that share physical blocks keep weights of their own."""
    pool = ref.Pool([64, 64, 64], 2, 64, 16, "bf16", seed=3)
    pool.tables[1] = pool.tables[0]
    pool.tables[2, :2] = pool.tables[0, :2]
    q = pool.randn(3, 4, 64, scale=2.0)
    weights = torch.rand((3, 2, 64), generator=pool.g)
    out, w = decode_weights(pkv, pool, q, weights, 0.125)
    want, tol, ww, wtol = ref.decode_weights(pool, q, weights, 0.125)
    within(out, want, tol)
    within(w, ww, wtol)


def test_decode_weights_bad_sequences(pkv):
    """A bad length or block zeroes the sequence's rows and leaves its
    weights; the others are served."""
    L = [40, 0, 50, 300, 60]
    pool = ref.Pool(L, 1, 64, 16, "bf16", seed=4, width=19)
    pool.tables[2, 1] = pool.num_blocks
    q = pool.randn(5, 2, 64, scale=2.0)
    weights = torch.rand((5, 1, 310), generator=pool.g)
    pool.seq_lens[4] = 19 * 16 + 1                          # past the table
    out, w = decode_weights(pkv, pool, q, weights, 0.125, max_len=310)
    st, flags = pkv.get_status()
    assert flags == pkv.FLAG_BAD_SEQ_LEN | pkv.FLAG_BAD_BLOCK
    good = ref.Pool(L, 1, 64, 16, "bf16", seed=4, width=19)
    for b in (1, 2, 4):
        assert (out[b] == 0).all() and same_bits(w[b], weights[b])
    for b in (0, 3):
        one = slice(b, b + 1)
        sub = good
        K, V = sub.rows("k", b, 0), sub.rows("v", b, 0)
        p, rel = ref.softmax_bound(q[b].double(), K, 0.125)
        tol = 2.0 ** -8 * (p @ V).abs() + (2.0 ** -8 + rel) * 1.01 * (p @ V.abs())
        within(out[one], (p @ V)[None], tol[None])
        assert not same_bits(w[b, :, :L[b]], weights[b, :, :L[b]])


def test_decode_weights_graph_and_stream(pkv):
    """A captured step replays on new inputs, and a step runs on a side stream."""
    L = [300, 17]
    pool = ref.Pool(L, 2, 128, 16, "bf16", seed=8)
    q = pool.randn(2, 8, 128, scale=2.0)
    weights = torch.rand((2, 2, 300), generator=pool.g)
    k, v, sc, bt, sl = pool.on()
    ws = workspace(pkv.weights_workspace_bytes(2, 8, 128, 300, 16))
    out = torch.empty((2, 8, 128), dtype=torch.bfloat16, device="cuda")
    w, qd = weights.cuda(), torch.zeros_like(q, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pkv.paged_attention_decode_weights(out, w, qd, k, v, bt, sl, 300, 128 ** -0.5, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkv.paged_attention_decode_weights(out, w, qd, k, v, bt, sl, 300, 128 ** -0.5, ws)
    qd.copy_(q)
    w.copy_(weights)
    graph.replay()
    torch.cuda.synchronize()
    want, tol, ww, wtol = ref.decode_weights(pool, q, weights, 128 ** -0.5)
    within(out, want, tol)
    within(w, ww, wtol)
    graph.replay()                                          # a second step adds the same again
    torch.cuda.synchronize()
    _, _, www, wtol2 = ref.decode_weights(pool, q, ww.float(), 128 ** -0.5)
    within(w, www, wtol + wtol2 + 2.0 ** -23 * ww.abs())


# --------------------------------------------------------------------------
# Weights of several query tokens
# --------------------------------------------------------------------------

def prompt_weights(pkv, pool, q, counts, weights, scale, accumulate=True, max_len=None, max_n=None):
    k, v, sc, bt, sl = pool.on()
    qs = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    max_len, max_n = max_len or max(pool.L), max_n or max(counts)
    ws = workspace(pkv.attention_weights_workspace_bytes(q.shape[0], q.shape[1], max_len))
    w = weights.cuda()
    pkv.attention_weights(w, q.cuda(), k, bt, sl, qs, max_len, max_n, scale, ws, accumulate=accumulate,
                          k_scale=sc["k_scale"])
    return w


@pytest.mark.parametrize("dtype,block,dim", POOLS)
@pytest.mark.parametrize("group", [1, 5, 8])
def test_prompt_weights(pkv, dtype, block, dim, group):
    L = [1, 90, 33, 130, 64, 7]
    counts = [1, 5, 33, 17, 0, 7]                            # whole prompts, chunks, one token, none
    pool = ref.Pool(L, 2, dim, block, dtype, seed=group)
    q = pool.randn(sum(counts), 2 * group, dim, scale=2.0)
    weights = torch.rand((len(L), 2, 150), generator=pool.g) * group / 50
    w = prompt_weights(pkv, pool, q, counts, weights, dim ** -0.5)
    want, tol = ref.prompt_weights(pool, q, counts, weights, dim ** -0.5)
    within(w, want, tol)
    for b, n in enumerate(L):
        assert same_bits(w[b, :, n:], weights[b, :, n:])
    assert same_bits(w[4], weights[4])


@pytest.mark.parametrize("dtype,L,counts", [("bf16", [1400, 600], [3, 20]), ("fp8", [700], [1]),
                                            ("int8", [300, 520], [300, 65])])
@pytest.mark.parametrize("accumulate", [True, False])
def test_prompt_weights_long(pkv, dtype, L, counts, accumulate):
    """Keys split over CTAs, several row tiles, and the stored form (whose
    earlier entries may hold anything)."""
    pool = ref.Pool(L, 1, 64, 16, dtype, seed=2, width=100)
    q = pool.randn(sum(counts), 4, 64, scale=2.0)
    weights = torch.rand((len(L), 1, 1500), generator=pool.g) if accumulate else \
        torch.full((len(L), 1, 1500), float("nan"))
    w = prompt_weights(pkv, pool, q, counts, weights, 0.125, accumulate)
    want, tol = ref.prompt_weights(pool, q, counts, torch.nan_to_num(weights), 0.125, accumulate)
    for b, n in enumerate(L):
        within(w[b, :, :n], want[b, :, :n], tol[b, :, :n])
        assert same_bits(w[b, :, n:], weights[b, :, n:])


@pytest.mark.parametrize("dtype,block,dim", POOLS)
@pytest.mark.parametrize("group,n,L", [(3, 130, [130, 300]), (7, 40, [290, 41]), (1, 200, [456, 200]),
                                       (4, 96, [700, 97]), (16, 9, [140, 10])])
def test_prompt_weights_row_tiles(pkv, dtype, block, dim, group, n, L):
    """Several 128-row tiles, heads that do not divide them, keys split over
    CTAs, chunks that end inside a tile; a sequence of one query beside them."""
    pool = ref.Pool(L + [50], 1, dim, block, dtype, seed=group)
    counts = [n, n, 1]
    q = pool.randn(sum(counts), group, dim, scale=2.0)
    weights = torch.rand((3, 1, max(L) + 5), generator=pool.g) * group * n / 300
    w = prompt_weights(pkv, pool, q, counts, weights, dim ** -0.5)
    want, tol = ref.prompt_weights(pool, q, counts, weights, dim ** -0.5)
    within(w, want, tol)
    for b, m in enumerate(pool.L):
        assert same_bits(w[b, :, m:], weights[b, :, m:])


@pytest.mark.parametrize("dtype", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("scale", [0.125, 3.0, -0.125])
def test_prompt_weights_steep_scores(pkv, dtype, scale):
    """Scores whose exponentials pass fp32's range many times over against the
    first keys' (the running reference has to move), and a negative scale."""
    pool = ref.Pool([260], 1, 64, 16, dtype, seed=11)
    q = pool.randn(100, 2, 64, scale=2.0)
    for j in range(16):                                       # the first keys are small
        ref.raw(pool.k)[pool.tables[0, 0].item(), j] = 0
    weights = torch.zeros((1, 1, 260))
    w = prompt_weights(pkv, pool, q, [100], weights, scale)
    want, tol = ref.prompt_weights(pool, q, [100], weights, scale)
    within(w, want, tol)


@pytest.mark.parametrize("dtype", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("scale", [0.125, 3.0, -0.125, 0.0])
@pytest.mark.parametrize("n,group", [(5, 2), (16, 2), (3, 1), (1, 32)])
@pytest.mark.parametrize("accumulate", [True, False])
def test_prompt_weights_steep_scores_of_few_rows(pkv, dtype, scale, n, group, accumulate):
    """The one-pass kernel (at most 32 rows) under steep scores, negative ones
    and none, added to earlier weights and stored over anything."""
    L = [260, 1100, n]
    pool = ref.Pool(L, 1, 64, 16, dtype, seed=11)
    q = pool.randn(3 * n, group, 64, scale=2.0)
    for b in (0, 1):
        for j in range(16):                                   # the first keys are small
            ref.raw(pool.k)[pool.tables[b, 0].item(), j] = 0
    weights = torch.rand((3, 1, 1100), generator=pool.g) if accumulate else torch.full((3, 1, 1100), float("nan"))
    w = prompt_weights(pkv, pool, q, [n] * 3, weights, scale, accumulate)
    want, tol = ref.prompt_weights(pool, q, [n] * 3, torch.nan_to_num(weights), scale, accumulate)
    for b, m in enumerate(L):
        within(w[b, :, :m], want[b, :, :m], tol[b, :, :m])
        assert same_bits(w[b, :, m:], weights[b, :, m:])


@pytest.mark.parametrize("dtype,block,dim", POOLS)
@pytest.mark.parametrize("group,counts", [(11, [2, 1, 0]), (24, [1, 1, 1]), (31, [1, 0, 1]), (130, [3, 1, 2]),
                                          (128, [2, 1, 1])])
def test_prompt_weights_large_groups(pkv, dtype, block, dim, group, counts):
    """Groups that leave rows of a tile unused, and ones past a row tile."""
    pool = ref.Pool([200, 70, 33], 1, dim, block, dtype, seed=group)
    q = pool.randn(sum(counts), group, dim, scale=2.0)
    weights = torch.rand((3, 1, 211), generator=pool.g) * group / 50
    w = prompt_weights(pkv, pool, q, counts, weights, dim ** -0.5)
    want, tol = ref.prompt_weights(pool, q, counts, weights, dim ** -0.5)
    within(w, want, tol)
    for b, m in enumerate(pool.L):
        assert same_bits(w[b, :, m:], weights[b, :, m:])


@pytest.mark.parametrize("dtype,n", [("bf16", 2), ("bf16", 5), ("bf16", 40), ("fp8", 5), ("int8", 12)])
def test_prompt_weights_of_a_long_context(pkv, dtype, n):
    """The last queries of contexts past what a cluster's TMEM holds."""
    pool = ref.Pool([20001, 8193, 50], 1, 64, 32, dtype, seed=n)
    q = pool.randn(3 * n, 4, 64, scale=2.0)
    weights = torch.rand((3, 1, 20100), generator=pool.g) / 1000
    w = prompt_weights(pkv, pool, q, [n] * 3, weights, 0.125)
    want, tol = ref.prompt_weights(pool, q, [n] * 3, weights, 0.125)
    within(w, want, tol)


def test_prompt_weights_of_one_token_are_the_decode_step(pkv):
    L = [300, 41]
    pool = ref.Pool(L, 2, 128, 32, "bf16", seed=9)
    q = pool.randn(2, 8, 128, scale=2.0)
    weights = torch.rand((2, 2, 300), generator=pool.g)
    _, a = decode_weights(pkv, pool, q, weights, 128 ** -0.5)
    b = prompt_weights(pkv, pool, q, [1, 1], weights, 128 ** -0.5)
    _, _, want, tol = ref.decode_weights(pool, q, weights, 128 ** -0.5)
    within(a, want, tol)
    within(b, want, tol)


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("bf16", 128), ("int8", 64), ("fp8", 128)])
def test_prompt_weights_many_units(pkv, dtype, dim):
    """More units of work (row tiles, key tiles) than CTAs fit the GPU several
    times over, ragged, some empty; bad sequences among them change nothing."""
    B, hkv, G = 48, 8, 2
    L = [(37 * b * b + 11 * b) % 690 + 1 for b in range(B)]
    counts = [min(n, (b * 29) % 83) for b, n in enumerate(L)]
    counts[5] = min(L[5], 82)
    good, pool = (ref.Pool(L, hkv, dim, 16, dtype, seed=21) for _ in range(2))
    q = pool.randn(sum(counts), hkv * G, dim, scale=2.0)
    weights = torch.rand((B, hkv, 700), generator=pool.g)
    block = next(b for b in range(20, B) if L[b] > 200 and counts[b] > 40)
    pool.tables[block, 3] = pool.k.shape[0]                   # outside the pool
    length = next(b for b in range(block + 1, B) if counts[b] > 40)
    pool.seq_lens[length] = 16 * pool.tables.shape[1] + 1     # past the table
    w = prompt_weights(pkv, pool, q, counts, weights, dim ** -0.5, max_len=700)
    assert pkv.get_status()[1] == pkv.FLAG_BAD_SEQ_LEN | pkv.FLAG_BAD_BLOCK
    want, tol = ref.prompt_weights(good, q, counts, weights, dim ** -0.5)
    for b, n in enumerate(L):
        if b in (block, length):
            assert same_bits(w[b], weights[b])
            continue
        within(w[b, :, :n], want[b, :, :n], tol[b, :, :n])
        assert same_bits(w[b, :, n:], weights[b, :, n:])


@pytest.mark.parametrize("dtype,block,dim", POOLS)
@pytest.mark.parametrize("n", [3, 4, 5, 10, 16])
def test_prompt_weights_few_rows_long_bound(pkv, dtype, block, dim, n):
    """12 to 64 rows where max_seq_len is past what a cluster's TMEM holds: the
    two-pass kernels, most key splits empty."""
    pool = ref.Pool([n + 3, 700, 260, 1], 2, dim, block, dtype, seed=n, width=9008 // block)
    counts = [n, n, 1, 1]
    q = pool.randn(sum(counts), 8, dim, scale=2.0)
    weights = torch.rand((4, 2, 9000), generator=pool.g) * n / 30
    w = prompt_weights(pkv, pool, q, counts, weights, dim ** -0.5, max_len=9000)
    want, tol = ref.prompt_weights(pool, q, counts, weights, dim ** -0.5)
    for b, m in enumerate(pool.L):
        within(w[b, :, :m], want[b, :, :m], tol[b, :, :m])
        assert same_bits(w[b, :, m:], weights[b, :, m:])


@pytest.mark.parametrize("dtype", ["bf16", "int8"])
def test_prompt_weights_repeat_bit_for_bit(pkv, dtype):
    """Which CTA takes which unit differs from call to call; the bits do not."""
    L = [(131 * b * b + 17 * b) % 1500 + 300 for b in range(24)]
    pool = ref.Pool([max(L)], 8, 64, 16, dtype, seed=3)       # one context that all sequences share
    k, v, sc, bt, sl = pool.on()
    bt = bt.expand(len(L), -1).contiguous()
    sl = torch.tensor(L, dtype=torch.int32, device="cuda")
    q = pool.randn(sum(L), 16, 64, scale=2.0).cuda()
    qs = torch.tensor(np.concatenate([[0], np.cumsum(L)]), dtype=torch.int32, device="cuda")
    ws = workspace(pkv.attention_weights_workspace_bytes(sum(L), 16, max(L)))
    first = None
    for _ in range(8):
        w = torch.zeros((len(L), 8, max(L)), device="cuda")
        pkv.attention_weights(w, q, k, bt, sl, qs, max(L), max(L), 0.125, ws, k_scale=sc["k_scale"])
        if first is None:
            first = w.cpu()
        assert same_bits(w.cpu(), first)
    # Every query row's weights add up to one: an exponential is off by 2^-22
    # and by its argument's rounding (|s - m'| < 2^7: 2^-18 by the product and
    # the sum), the sums of up to 2048 positive terms by 2^-13 at most.
    total = first.double().sum(dim=(1, 2))
    assert torch.allclose(total, torch.tensor(L).double() * 16, rtol=2.0 ** -12)


def test_prompt_weights_on_two_streams_and_in_a_graph(pkv):
    """Calls that overlap on two streams, each with a workspace of its own, and
    replays of a captured call give the bits of a call alone."""
    L, counts = [900, 640, 333], [200, 90, 100]
    pools = [ref.Pool(L, 4, 64, 16, "bf16", seed=s) for s in (1, 2)]
    args = []
    for pool in pools:
        k, v, sc, bt, sl = pool.on()
        q = pool.randn(sum(counts), 8, 64, scale=2.0).cuda()
        qs = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        ws = workspace(pkv.attention_weights_workspace_bytes(q.shape[0], 8, 900))
        args.append((q, k, bt, sl, qs, 900, max(counts), 0.125, ws))
    alone = []
    for a in args:
        w = torch.zeros((3, 4, 900), device="cuda")
        pkv.attention_weights(w, *a)
        alone.append(w.cpu())
    ws = [torch.zeros((3, 4, 900), device="cuda") for _ in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    for i in range(6):
        for st, w, a in zip(streams, ws, args):
            pkv.attention_weights(w, *a, accumulate=False, stream=st.cuda_stream)
    torch.cuda.synchronize()
    for w, want in zip(ws, alone):
        assert same_bits(w.cpu(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.attention_weights(ws[0], *args[0], accumulate=False, stream=torch.cuda.current_stream().cuda_stream)
    for _ in range(3):
        ws[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(ws[0].cpu(), alone[0])


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("L", [[250, 200, 240], [1000, 900, 1024]])
def test_prompt_weights_rows_start_without_statistics(pkv, dtype, L):
    """The rows of the workspace ([Hkv][tokens][group][key splits] pairs) that
    no unit of work completes say so (maximum -inf, sum -1), whatever was there
    before, so that the weights they would give are left out: here rows of a
    sequence with a bad length and rows that no sequence has, over the finite
    statistics of an earlier call."""
    H, G, counts, T = 1, 4, [40, 50, 60], 170
    pool = ref.Pool(L, H, 64, 16, dtype, seed=6)
    k, v, sc, bt, sl = pool.on()
    q = pool.randn(T, H * G, 64, scale=2.0)
    n = pkv.attention_weights_workspace_bytes(T, H * G, max(L))
    splits = n // (T * H * G * 8)
    assert splits == (1 if max(L) <= 256 else 4)              # of 256 tokens: few units, all of them are used
    ws = torch.full((n // 4,), 1.5, device="cuda")
    qs = torch.tensor([0, 40, 90, 150], dtype=torch.int32, device="cuda")
    sl[1] = 2000                                              # past the table
    weights = torch.rand((3, H, max(L)), generator=pool.g)
    w = weights.cuda()
    pkv.attention_weights(w, q.cuda(), k, bt, sl, qs, max(L), 60, 0.125, ws, k_scale=sc["k_scale"])
    assert pkv.get_status()[1] == pkv.FLAG_BAD_SEQ_LEN
    want, tol = ref.prompt_weights(pool, q, counts, weights, 0.125)
    for b in (0, 2):
        within(w[b, :, :L[b]], want[b, :, :L[b]], tol[b, :, :L[b]])
    assert same_bits(w[1], weights[1])
    rows = ws.view(H, T, G, splits, 2).cpu()
    none = torch.zeros(T, dtype=torch.bool)
    none[40:90] = none[150:] = True
    assert (rows[:, none, :, :, 0] == -float("inf")).all() and (rows[:, none, :, :, 1] == -1).all()
    assert torch.isfinite(rows[:, ~none, :, 0, 0]).all() and (rows[:, ~none, :, 0, 1] > 0).all()


def test_prompt_weights_bad_sequences(pkv):
    L = [40, 20, 50, 64, 64]
    counts = [4, 21, 5, 6, 6]                                # 21 > 20
    pool = ref.Pool(L, 1, 64, 16, "bf16", seed=4)
    pool.tables[2, 3] = -1
    pool.seq_lens[3] = 65                                    # past the table
    q = pool.randn(sum(counts), 2, 64, scale=2.0)
    weights = torch.rand((5, 1, 70), generator=pool.g)
    w = prompt_weights(pkv, pool, q, counts, weights, 0.125, max_len=70)
    st, flags = pkv.get_status()
    assert flags == pkv.FLAG_BAD_SEQ_LEN | pkv.FLAG_BAD_BLOCK
    for b in (1, 2, 3):
        assert same_bits(w[b], weights[b])
    good = ref.Pool(L, 1, 64, 16, "bf16", seed=4)
    for b in (0, 4):
        one = ref.Pool([L[b]], 1, 64, 16, "bf16")
        one.k, one.tables = good.k, good.tables[b:b + 1]
        at = sum(counts[:b])
        want, tol = ref.prompt_weights(one, q[at:at + counts[b]], [counts[b]], weights[b:b + 1], 0.125)
        within(w[b:b + 1], want, tol)


# --------------------------------------------------------------------------
# Selection
# --------------------------------------------------------------------------

def select(pkv, weights, L, budget, recent, max_len=None):
    B, H, W = weights.shape
    idx = torch.full((B, H, budget), 7, dtype=torch.int32, device="cuda")
    num = torch.full((B,), 7, dtype=torch.int32, device="cuda")
    pkv.select_tokens(idx, num, weights.cuda(), torch.tensor(L, dtype=torch.int32, device="cuda"),
                      max_len or W, recent)
    return idx.cpu(), num.cpu()


@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (16, 0), (16, 5), (16, 16), (64, 32), (255, 1),
                                           (300, 7)])
@pytest.mark.parametrize("kind", ["random", "ties", "equal", "special"])
def test_select(pkv, budget, recent, kind):
    L = [1, 2, 15, 16, 17, 63, 65, 256, 300, 299]
    g = torch.Generator().manual_seed(budget)
    w = torch.exp(3 * torch.randn((len(L), 3, 303), generator=g))
    if kind == "ties":
        w = torch.randint(0, 4, w.shape, generator=g).float() - 1
    elif kind == "equal":
        w = torch.full_like(w, 0.25)
    elif kind == "special":
        pick = torch.randint(0, 8, w.shape, generator=g)
        for i, x in enumerate([float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 1e-42]):
            w[pick == i] = x
    idx, num = select(pkv, w, L, budget, recent)
    want, wnum = ref.select(w, L, budget, recent)
    assert torch.equal(num, wnum)
    assert torch.equal(idx, want)


@pytest.mark.parametrize("L,budget,recent", [([5000, 4096, 4097], 1024, 100), ([40001, 9], 4000, 0),
                                             ([131072], 8192, 4096), ([400000, 77777], 30000, 1)])
def test_select_long(pkv, L, budget, recent):
    """Rows of several CTAs, and slices that do not fit shared memory."""
    g = torch.Generator().manual_seed(1)
    w = torch.exp(2 * torch.randn((len(L), 1, max(L) + 1), generator=g))
    w[:, :, ::7] = 0.0
    w[:, :, 5::11] = w[0, 0, 5]                              # ties near a border, across CTAs
    idx, num = select(pkv, w, L, budget, recent)
    want, wnum = ref.select(w, L, budget, recent)
    assert torch.equal(num, wnum)
    assert torch.equal(idx, want)


def test_select_longest_rows(pkv):
    """The longest rows that the call takes."""
    L = [1 << 21, 5, (1 << 21) - 77]
    g = torch.Generator().manual_seed(2)
    w = torch.randn((3, 1, 1 << 21), generator=g)
    w[0, 0, ::3] = 0.5
    idx, num = select(pkv, w, L, 5000, 17)
    want, wnum = ref.select(w, L, 5000, 17)
    assert torch.equal(num, wnum) and torch.equal(idx, want)


def test_select_bad_lengths(pkv):
    w = torch.rand((4, 2, 64))
    idx, num = select(pkv, w, [0, 64, -3, 65], 8, 2)
    st, flags = pkv.get_status()
    assert flags == pkv.FLAG_BAD_SEQ_LEN
    want, _ = ref.select(w[1:2], [64], 8, 2)
    assert num.tolist() == [0, 8, 0, 0] and torch.equal(idx[1:2], want)
    assert (idx[[0, 2, 3]] == -1).all()


# --------------------------------------------------------------------------
# Eviction
# --------------------------------------------------------------------------

def random_keep(pool, budget, heads, g):
    B = len(pool.L)
    idx = torch.full((B, heads, budget), -1, dtype=torch.int32)
    num = torch.tensor([min(n, budget) for n in pool.L], dtype=torch.int32)
    for b, n in enumerate(pool.L):
        for h in range(heads):
            m = int(num[b])
            idx[b, h, :m] = torch.randperm(n, generator=g)[:m].sort().values.to(torch.int32)
    return idx, num


def evict(pkv, pool, idx, num, dst, weights):
    k, v, sc, bt, sl = pool.on()
    w = None if weights is None else weights.cuda()
    pkv.evict_tokens(k, v, bt, sl, idx.cuda(), num.cuda(),
                     dst_block_tables=None if dst is None else dst.cuda(), weights=w, **sc)
    return k, v, sc["k_scale"], sc["v_scale"], w


def check_evict(got, want):
    for a, b in zip(got, want):
        if b is not None and a is not None:
            assert same_bits(a, b)


@pytest.mark.parametrize("dtype,block,dim", POOLS)
@pytest.mark.parametrize("budget", [1, 16, 33, 70, 400])
@pytest.mark.parametrize("fresh", [False, True])
def test_evict(pkv, dtype, block, dim, budget, fresh):
    L = [1, 31, 70, 33, 300, 250]
    pool = ref.Pool(L, 3, dim, block, dtype, seed=budget, extra=100)
    idx, num = random_keep(pool, budget, 3, pool.g)
    idx[4, 0, :num[4]] = torch.arange(int(num[4]))           # rows that stay
    idx[5, 1, :num[5]] = torch.arange(250 - int(num[5]), 250)  # the last ones
    dst = pool.tables
    if fresh:
        n = (int(num.max()) + block - 1) // block
        need = n * len(L)
        while len(pool.free) < need:                          # small budgets only use a part
            pool = ref.Pool(L, 3, dim, block, dtype, seed=budget, extra=need + 3)
            idx, num = random_keep(pool, budget, 3, pool.g)
        dst = pool.free[:need].view(len(L), n).contiguous()
    weights = torch.rand((len(L), 3, 305), generator=pool.g)
    got = evict(pkv, pool, idx, num, dst if fresh else None, weights)
    check_evict(got, ref.evict(pool, idx, num, dst, weights))


@pytest.mark.parametrize("dtype,block,dim", [("bf16", 16, 64), ("int8", 16, 64), ("fp8", 32, 128)])
@pytest.mark.parametrize("fresh", [False, True])
def test_evict_many_rounds(pkv, dtype, block, dim, fresh):
    """Many rounds per CTA and clusters of CTAs, with weights that always move
    in place: lists whose sources lie far and near."""
    L = [5000, 3001]
    pool = ref.Pool(L, 1, dim, block, dtype, seed=3, extra=2 * (2500 // block + 1) if fresh else 3)
    idx, num = random_keep(pool, 2500, 1, pool.g)
    idx[0, 0] = torch.cat([torch.arange(1000), torch.arange(3500, 5000)])
    n = 2500 // block + 1
    dst = pool.free[:2 * n].view(2, n).contiguous() if fresh else pool.tables
    weights = torch.rand((2, 1, 5000), generator=pool.g)
    want = ref.evict(pool, idx, num, dst, weights)
    for _ in range(5):
        check_evict(evict(pkv, pool, idx, num, dst if fresh else None, weights), want)


@pytest.mark.parametrize("dtype", ["bf16", "int8"])
def test_evict_nothing_kept_and_padding(pkv, dtype):
    """Sequences that keep nothing, or are padding of length 0, beside one that
    is packed."""
    pool = ref.Pool([50, 0, 70], 2, 64, 16, dtype, seed=9)
    idx, num = random_keep(pool, 20, 2, pool.g)
    num[0] = 0
    weights = torch.rand((3, 2, 80), generator=pool.g)
    got = evict(pkv, pool, idx, num, None, weights)
    check_evict(got, ref.evict(pool, idx, num, pool.tables, weights))


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_evict_mixed_destinations(pkv, dtype):
    """Some destination blocks replaced, some in place; no weights."""
    pool = ref.Pool([200, 150], 2, 128, 16, dtype, seed=6, extra=20)
    idx, num = random_keep(pool, 100, 2, pool.g)
    dst = torch.full((2, 9), -1, dtype=torch.int32)
    dst[:, :7] = pool.tables[:, :7]
    dst[0, :4] = pool.free[:4]
    dst[1, 2] = pool.free[5]
    got = evict(pkv, pool, idx, num, dst, None)
    check_evict(got[:4], ref.evict(pool, idx, num, dst, torch.zeros(2, 2, 300))[:4])


def test_evict_zero_and_nan_values(pkv):
    """A block of zeros, tiny scales, a zero scale and NaN codes."""
    pool = ref.Pool([64, 64], 1, 64, 16, "fp8", seed=1, extra=8)
    ref.raw(pool.k)[pool.tables[0, 1].item()] = 0
    ref.raw(pool.k)[pool.tables[0, 2].item(), 3] = 0x7F
    pool.k_scale[pool.tables[0, 3].item()] = 0.0
    pool.v_scale[pool.tables[1, 0].item()] = 1e-44
    pool.v_scale[pool.tables[1, 2].item()] = 3e38
    idx, num = random_keep(pool, 40, 1, pool.g)
    idx[0, 0, :16] = torch.arange(16, 32)                     # block 0: all zeros
    idx[0, 0, 16:40] = torch.arange(32, 56)
    weights = torch.rand((2, 1, 64), generator=pool.g)
    got = evict(pkv, pool, idx, num, None, weights)
    check_evict(got, ref.evict(pool, idx, num, pool.tables, weights))
    assert got[2][pool.tables[0, 0].item(), 0] == 0


@pytest.mark.parametrize("dtype", ["int8", "fp8"])
@pytest.mark.parametrize("large,small", [(70, -70), (64, -64), (80, -40), (40, -80), (79, 1), (80, -80), (100, -30),
                                         (30, -100), (8, -126)])
@pytest.mark.parametrize("fresh", [False, True])
def test_evict_scales_far_apart(pkv, dtype, large, small, fresh):
    """A row of zeros under a scale 2^large packed beside rows under 2^small:
    the zeros are codes of 0 under the new scale, whatever the two's ratio."""
    pool = ref.Pool([64, 50], 2, 64, 16, dtype, seed=4, extra=8)
    for b in (0, 1):
        blocks = pool.tables[b].long()
        for cache, scale in ((pool.k, pool.k_scale), (pool.v, pool.v_scale)):
            scale[blocks] = 2.0 ** small
            scale[blocks[2]] = 2.0 ** large
            ref.raw(cache)[blocks[2]] = 0
            if dtype == "fp8":
                ref.raw(cache)[blocks[2], :, :, ::3] = 0x80           # -0
    idx, num = random_keep(pool, 30, 2, pool.g)
    for b in (0, 1):
        idx[b, :, :8] = torch.arange(1, 9)
        idx[b, :, 8:16] = torch.arange(33, 41)                  # the zeros, beside them
        idx[b, :, 16:24] = torch.arange(41, 49)                 # zeros in the next block
        idx[b, :, 24:30] = torch.tensor([49, 49, 49, 49, 49, 49]) if b else torch.arange(49, 55)
    num[1] = 25                                                 # the second keeps one row after them
    weights = torch.rand((2, 2, 64), generator=pool.g)
    dst = pool.free[:4].view(2, 2).contiguous() if fresh else None
    got = evict(pkv, pool, idx, num, dst, weights)
    check_evict(got, ref.evict(pool, idx, num, pool.tables if dst is None else dst, weights))


def test_evict_bad_lists(pkv):
    """A list that does not ascend in range leaves its head alone, a bad
    length its sequence, a bad block its destination block."""
    L = [64, 64, 64, 64]
    pool = ref.Pool(L, 2, 64, 16, "bf16", seed=3, extra=4)
    idx, num = random_keep(pool, 32, 2, pool.g)
    weights = torch.rand((4, 2, 64), generator=pool.g)
    want = ref.evict(pool, idx, num, pool.tables, weights)
    bad = idx.clone()
    bad[0, 1, 5] = bad[0, 1, 4]                               # twice the same row
    bad[1, 0, 31] = 64                                        # past the end
    num2 = num.clone()
    num2[2] = 33                                              # more than the list holds
    got = evict(pkv, pool, bad, num2, None, weights)
    st, flags = pkv.get_status()
    assert flags == pkv.FLAG_BAD_INDEX | pkv.FLAG_BAD_SEQ_LEN
    for cache, w, old in ((got[0], want[0], pool.k), (got[1], want[1], pool.v)):
        for b in range(4):
            ids = pool.tables[b].long()
            for h in range(2):
                left = (b, h) in ((0, 1), (1, 0)) or b == 2
                assert same_bits(ref.take(cache, ids.cuda(), slice(None), h),
                                 ref.take(old if left else w, ids, slice(None), h)), (b, h)
    for b in range(4):
        for h in range(2):
            left = (b, h) in ((0, 1), (1, 0)) or b == 2
            assert same_bits(got[4][b, h], (weights if left else want[4])[b, h])


# --------------------------------------------------------------------------
# Self-scaling append
# --------------------------------------------------------------------------

def append(pkv, pool, k_new, v_new, counts, decode=False, max_n=None):
    k, v, sc, bt, sl = pool.on()
    qs = None if decode else torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    pkv.append_scaled(k_new.cuda(), v_new.cuda(), k, v, sc["k_scale"], sc["v_scale"], bt, sl, qs,
                      max_n or max(counts))
    return k, sc["k_scale"], v, sc["v_scale"]


EIGHT = [p for p in POOLS if p[0] != "bf16"]


@pytest.mark.parametrize("dtype,block,dim", EIGHT)
@pytest.mark.parametrize("size", [0.3, 1.0, 4.0])
def test_append_one_token(pkv, dtype, block, dim, size):
    """Opened blocks, scales that hold and scales that grow."""
    L = [1, 2, block, block + 1, 2 * block, 100, 2 * block + 1]
    pool = ref.Pool(L, 3, dim, block, dtype, seed=int(size * 10))
    n = len(L)
    k_new, v_new = pool.randn(n, 3, dim, scale=size), pool.randn(n, 3, dim, scale=size)
    got = append(pkv, pool, k_new, v_new, [1] * n, decode=True)
    want = ref.append(pool, k_new, v_new, [1] * n)
    for a, b in zip(got, want):
        assert same_bits(a, b)


@pytest.mark.parametrize("dtype,block,dim", EIGHT)
def test_append_many_tokens(pkv, dtype, block, dim):
    L = [1, 40, 100, 64, 33, 5, 200]
    counts = [1, 40, 3, 0, 17, 4, 129]
    pool = ref.Pool(L, 2, dim, block, dtype, seed=2)
    T = sum(counts)
    size = torch.exp(torch.randn((T, 1, 1), generator=pool.g))
    k_new, v_new = ((torch.randn((T, 2, dim), generator=pool.g) * size).to(torch.bfloat16) for _ in range(2))
    got = append(pkv, pool, k_new, v_new, counts)
    for a, b in zip(got, ref.append(pool, k_new, v_new, counts)):
        assert same_bits(a, b)


@pytest.mark.parametrize("dtype", ["int8", "fp8"])
def test_append_special_values(pkv, dtype):
    """Zeros, infinities, NaN, tiny and huge magnitudes; a stale NaN scale on
    an opened block."""
    pool = ref.Pool([33, 18, 17, 20, 40, 48], 1, 64, 16, dtype, seed=1)
    counts = [1, 2, 17, 4, 1, 1]
    pool.k_scale[pool.tables[0, 2].item()] = float("nan")     # row 0 of the block is new
    T = sum(counts)
    k_new, v_new = pool.randn(T, 1, 64), pool.randn(T, 1, 64)
    k_new[1:3] = 0.0
    k_new[3, 0, 5], k_new[4, 0, 6], k_new[5, 0, 7] = float("inf"), -float("inf"), float("nan")
    v_new[3:6] *= 1e-38
    v_new[-1] *= 1e30
    k_new[-2] = 1e-40                                         # bf16 subnormals
    got = append(pkv, pool, k_new, v_new, counts)
    for a, b in zip(got, ref.append(pool, k_new, v_new, counts)):
        assert same_bits(a, b)


@pytest.mark.parametrize("dtype,block,dim", EIGHT)
def test_append_codes_are_those_of_reshape_and_cache(pkv, dtype, block, dim):
    """Under the scales that the append has made, reshape_and_cache stores the
    same codes, the sign of a zero among them: blocks of small and large values
    with zeros of both signs, of zeros alone, and with infinities and NaN."""
    L = [5 * block, 3, block + 1]
    pool = ref.Pool(L, 2, dim, block, dtype, seed=12)
    T = sum(L)
    k_new, v_new = pool.randn(T, 2, dim), pool.randn(T, 2, dim, scale=1e-20)
    for x in (k_new, v_new):
        x[:, :, 1::3] = -0.0
        x[:, :, 2::7] = 0.0
        x[block:2 * block] = -0.0
        x[2 * block, 0, 5], x[2 * block + 1, 0, 6], x[2 * block + 2, 0, 7] = float("inf"), -float("inf"), float("nan")
        x[3 * block:4 * block] *= 1e-19                       # (of v: bf16's subnormals)
    got = append(pkv, pool, k_new, v_new, L)
    for a, b in zip(got, ref.append(pool, k_new, v_new, L)):
        assert same_bits(a, b)
    k, v, _, bt, _ = pool.on()
    pos = torch.tensor([i for n in L for i in range(n)], dtype=torch.int32, device="cuda")
    seq = torch.tensor([b for b, n in enumerate(L) for _ in range(n)], dtype=torch.int32, device="cuda")
    slots = torch.empty(T, dtype=torch.int64, device="cuda")
    pkv.token_slot_mapping(bt, pos, pool.num_blocks, block, slots, seq_idx=seq)
    pkv.reshape_and_cache(k_new.cuda(), v_new.cuda(), k, v, slots, got[1], got[3])
    assert same_bits(got[0], k.cpu()) and same_bits(got[2], v.cpu())


def test_append_recodes_minus_128(pkv):
    """A pool whose int8 codes hold -128 (no call of the library writes it):
    coded again, it clamps to -127."""
    pool = ref.Pool([20, 18], 1, 64, 16, "int8", seed=1)
    for b in (0, 1):
        pool.k[pool.tables[b, 1].item()][:, :, ::3] = -128
        pool.v[pool.tables[b, 1].item()] = 127
    new = pool.randn(2, 1, 64)
    top = pool.k_scale[pool.tables[:, 1].long(), 0] * 127
    new[:, 0, 0] = (top * 1.005).to(torch.bfloat16)           # the scale grows by less than one code step
    got = append(pkv, pool, new, new, [1, 1], decode=True)
    for a, b in zip(got, ref.append(pool, new, new, [1, 1])):
        assert same_bits(a, b)


@pytest.mark.parametrize("dtype", ["int8", "fp8"])
@pytest.mark.parametrize("size", [1e-30, 1e-26, 1e-20, 1.0, 1e20, 1e26])
def test_append_codes_next_to_borders(pkv, dtype, size):
    """Values whose quotients by the scale fall on or next to the border of two
    codes, at every magnitude of the scale."""
    pool = ref.Pool([16 * 12], 2, 64, 16, dtype, seed=5)
    n = 16 * 12
    new = []
    for _ in range(2):
        # few significant bits, so that x * Q / amax is often a midpoint
        x = torch.randint(-15, 16, (n, 2, 64), generator=pool.g).double()
        x[::16, :, 0] = torch.randint(8, 16, (12, 2), generator=pool.g).double() * 2
        new.append((x * size).to(torch.bfloat16))
    got = append(pkv, pool, *new, [n])
    for a, b in zip(got, ref.append(pool, *new, [n])):
        assert same_bits(a, b)


def test_append_then_attend(pkv):
    """A prompt and a few decode steps through the append, read by the decode
    attention: the stored values are within half a code step of the tokens."""
    d, block = 64, 16
    pool = ref.Pool([20, 33], 2, d, block, "int8", seed=5, width=4, extra=4)
    pool.tables[:, 2:] = torch.stack([pool.free[:2], torch.cat([pool.tables[1, 2:3], pool.free[2:3]])])
    k, v, sc, bt, sl = pool.on()
    T = 53
    tokens = [(pool.randn(20, 2, d), pool.randn(20, 2, d)), (pool.randn(33, 2, d), pool.randn(33, 2, d))]
    qs = torch.tensor([0, 20, 53], dtype=torch.int32, device="cuda")
    pkv.append_scaled(*(torch.cat([tokens[0][i], tokens[1][i]]).cuda() for i in (0, 1)), k, v,
                      sc["k_scale"], sc["v_scale"], bt, sl, qs, 33)
    for _ in range(6):
        new = pool.randn(2, 2, d, scale=1.5), pool.randn(2, 2, d, scale=1.5)
        for b in (0, 1):
            tokens[b] = tuple(torch.cat([tokens[b][i], new[i][b:b + 1]]) for i in (0, 1))
        sl += 1
        pkv.append_scaled(new[0].cuda(), new[1].cuda(), k, v, sc["k_scale"], sc["v_scale"], bt, sl)
    assert T + 12 == sum(len(t[0]) for t in tokens)
    for name, cache, scale in (("k", k, sc["k_scale"]), ("v", v, sc["v_scale"])):
        for b in (0, 1):
            n = len(tokens[b][0])
            ids = bt[b, :(n + 15) // 16].long()
            val = (ref.f64(ref.take(cache, ids)) * scale[ids].double()[:, None, :, None]).reshape(-1, 2, d)[:n].cpu()
            x = tokens[b][0 if name == "k" else 1].double()
            # one coding, and one more (of a coded value) for each growth of
            # the scale: half a step each, at most block - 1 growths
            step = scale[ids].double().repeat_interleave(block, 0)[:n].cpu()
            assert ((val - x).abs() <= step[:, :, None] * 0.5 * 8).all()
            assert ((val - x).abs().mean() <= step.mean() * 0.5)
    assert pkv.get_status()[1] == 0


@pytest.mark.parametrize("dtype,block", [("int8", 16), ("fp8", 32)])
def test_appended_pool_is_attended(pkv, dtype, block):
    """Prompts and decode steps through the append, then the plain decode, the
    decode with weights, the weights of several queries and the differential
    attention over what it stored, against 64 bits of the stored codes."""
    d, H, G = 64, 2, 2
    L = [20, 33, 100]
    pool = ref.Pool([n + 6 for n in L], H, d, block, dtype, seed=5)
    k, v, sc, bt, sl = pool.on()
    for x in sc.values():
        x.fill_(float("nan"))                                 # the append makes every scale
    sl.copy_(torch.tensor(L))
    qs = torch.tensor(np.concatenate([[0], np.cumsum(L)]), dtype=torch.int32, device="cuda")
    T = sum(L)
    pkv.append_scaled(pool.randn(T, H, d).cuda(), pool.randn(T, H, d).cuda(), k, v, sc["k_scale"], sc["v_scale"],
                      bt, sl, qs, max(L))
    for i in range(6):
        sl += 1
        size = 0.5 + i
        pkv.append_scaled(pool.randn(3, H, d, scale=size).cuda(), pool.randn(3, H, d, scale=size).cuda(), k, v,
                          sc["k_scale"], sc["v_scale"], bt, sl)
    pool.k, pool.v, pool.k_scale, pool.v_scale = k.cpu(), v.cpu(), sc["k_scale"].cpu(), sc["v_scale"].cpu()
    assert sl.tolist() == pool.L
    top, scale = max(pool.L), d ** -0.5
    q = pool.randn(3, H * G, d)
    weights = torch.rand((3, H, top), generator=pool.g)
    want, tol, ww, wtol = ref.decode_weights(pool, q, weights, scale)
    out, w = decode_weights(pkv, pool, q, weights, scale)
    within(out, want, tol)
    within(w, ww, wtol)
    plain = torch.full_like(out, float("nan"))
    pkv.paged_attention_decode(plain, q.cuda(), k, v, bt, sl, top, scale,
                               workspace(pkv.workspace_bytes(3, H * G, d, top, block)), **sc)
    within(plain, want, tol)
    counts = [4, 1, 7]
    q = pool.randn(12, H * G, d)
    within(prompt_weights(pkv, pool, q, counts, weights, scale), *ref.prompt_weights(pool, q, counts, weights, scale))
    q, lam = pool.randn(3, 4, d), torch.tensor([0.3, 0.8])
    within(diff(pkv, pool, q, scale, lam, None), *ref.diff_attention(pool, q, scale, lam, None, 1e-5))


def test_append_bad_sequences(pkv):
    pool = ref.Pool([20, 20, 40, 64], 1, 64, 16, "int8", seed=3)
    counts = [2, 21, 3, 1]
    pool.tables[2, 2] = pool.num_blocks + 5
    pool.seq_lens[3] = 65                                     # past the table
    k_new, v_new = pool.randn(27, 1, 64), pool.randn(27, 1, 64)
    got = append(pkv, pool, k_new, v_new, counts)
    st, flags = pkv.get_status()
    assert flags == pkv.FLAG_BAD_SEQ_LEN | pkv.FLAG_BAD_BLOCK
    pool.L = [20, 20, 40, 64]
    want = ref.append(pool, k_new, v_new, [2, 0, 0, 0])
    # sequence 2's three tokens lie in the bad block alone
    for a, b in zip(got, want):
        assert same_bits(a, b)


# --------------------------------------------------------------------------
# Differential attention
# --------------------------------------------------------------------------

def diff(pkv, pool, q, scale, lam, norm, eps=1e-5, max_len=None):
    k, v, sc, bt, sl = pool.on()
    B, rows, d = q.shape
    max_len = max_len or max(pool.L)
    out = torch.full((B, rows // 2, 2 * d), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = workspace(pkv.diff_workspace_bytes(B, rows // 2, d, max_len, pool.block))
    pkv.paged_diff_attention_decode(out, q.cuda(), k, v, bt, sl, max_len, scale, lam.cuda(),
                                    None if norm is None else norm.cuda(), eps, ws, **sc)
    return out


@pytest.mark.parametrize("dtype,block,dim", POOLS)
@pytest.mark.parametrize("group,norm", [(1, True), (2, False), (3, True), (4, False), (5, True), (9, False)])
def test_diff(pkv, dtype, block, dim, group, norm):
    L = [1, 2, block, block + 1, 100, 257]
    pool = ref.Pool(L, 4, dim, block, dtype, seed=group)
    H = 2 * group
    q = pool.randn(len(L), 2 * H, dim, scale=2.0)
    lam = 0.2 + 0.6 * torch.rand(H, generator=pool.g)
    if not norm:
        lam[0] = -1.5
    weight = 0.5 + torch.rand(2 * dim, generator=pool.g) if norm else None
    out = diff(pkv, pool, q, dim ** -0.5, lam, weight)
    want, tol = ref.diff_attention(pool, q, dim ** -0.5, lam, weight, 1e-5)
    within(out, want, tol)


@pytest.mark.parametrize("dtype,dim,L", [("bf16", 128, [1500, 255, 257]), ("int8", 64, [2049, 513]),
                                         ("fp8", 128, [1025, 3]), ("bf16", 64, [3000])])
def test_diff_partitions(pkv, dtype, dim, L):
    pool = ref.Pool(L, 2, dim, 16, dtype, seed=5)
    q = pool.randn(len(L), 8, dim, scale=2.0)
    lam = 0.2 + 0.6 * torch.rand(4, generator=pool.g)
    weight = 0.5 + torch.rand(2 * dim, generator=pool.g)
    out = diff(pkv, pool, q, dim ** -0.5, lam, weight)
    want, tol = ref.diff_attention(pool, q, dim ** -0.5, lam, weight, 1e-5)
    within(out, want, tol)


def test_diff_lambda_zero_is_one_map(pkv):
    """lambda = 0: two attentions over the halves of V by the first map."""
    pool = ref.Pool([300, 40], 2, 64, 16, "bf16", seed=2)
    q = pool.randn(2, 4, 64, scale=2.0)
    out = diff(pkv, pool, q, 0.125, torch.zeros(2), None)
    for h in (0, 1):
        for b in (0, 1):
            p, rel = ref.softmax_bound(q[b, 2 * h:2 * h + 1].double(), pool.rows("k", b, 0), 0.125)
            V = torch.cat([pool.rows("v", b, 0), pool.rows("v", b, 1)], dim=1)
            tol = 2.0 ** -8 * (p @ V).abs() + (2.0 ** -8 + rel) * 1.01 * (p @ V.abs())
            within(out[b, h], (p @ V)[0], tol[0])


def test_diff_bad_sequences(pkv):
    L = [40, 0, 600, 64]
    pool = ref.Pool(L, 2, 64, 16, "bf16", seed=4)
    good = [pool.tables[0].clone()]
    pool.tables[2, 20] = -5
    pool.seq_lens[3] = 1000
    q = pool.randn(4, 4, 64, scale=2.0)
    lam = torch.full((2,), 0.5)
    out = diff(pkv, pool, q, 0.125, lam, torch.ones(128), max_len=700)
    st, flags = pkv.get_status()
    assert flags == pkv.FLAG_BAD_SEQ_LEN | pkv.FLAG_BAD_BLOCK
    assert (out[1:] == 0).all()
    one = ref.Pool([40], 2, 64, 16, "bf16")
    one.k, one.v, one.tables = pool.k, pool.v, good[0][None]
    want, tol = ref.diff_attention(one, q[:1], 0.125, lam, torch.ones(128), 1e-5)
    within(out[:1], want, tol)


@pytest.mark.parametrize("dtype,block,dim,L", [("int8", 16, 128, [2049, 513, 7]), ("fp8", 32, 64, [1025, 40]),
                                               ("int8", 32, 64, [300]), ("fp8", 16, 128, [90, 1])])
@pytest.mark.parametrize("ratio", [2.0 ** -10, 1e-4, 1e-6, 2.0 ** -40, 1e6])
@pytest.mark.parametrize("norm", [False, True])
def test_diff_value_halves_of_different_scales(pkv, dtype, block, dim, L, ratio, norm):
    """The two pool heads of a value have scales of their own, whatever their
    ratio: each half keeps the precision of its own probabilities.  (The bound
    of an element goes by its own half: p in fp16 is off by 2^-11 p, below
    fp16's smallest normal number by 2^-25 of the largest, sum p = 1, which
    over 2049 tokens is 2^-14 of the half's values; the bound counts 2^-8.)"""
    pool = ref.Pool(L, 4, dim, block, dtype, seed=6)
    pool.v_scale[:, 1::2] *= ratio
    q = pool.randn(len(L), 12, dim, scale=2.0)
    lam = 0.2 + 0.6 * torch.rand(6, generator=pool.g)
    weight = 0.5 + torch.rand(2 * dim, generator=pool.g) if norm else None
    out = diff(pkv, pool, q, dim ** -0.5, lam, weight)
    want, tol = ref.diff_attention(pool, q, dim ** -0.5, lam, weight, 1e-5)
    within(out, want, tol)


def test_diff_value_half_of_zeros(pkv):
    """A V head whose scales are all zero, and one whose values are all zero."""
    for head in (0, 1):
        pool = ref.Pool([300, 20], 2, 64, 16, "int8", seed=7)
        pool.v_scale[:, head] = 0.0
        ref.raw(pool.v)[pool.tables[1, :2].long(), :, 1 - head] = 0
        q = pool.randn(2, 4, 64, scale=2.0)
        lam = torch.tensor([0.3, 0.7])
        out = diff(pkv, pool, q, 0.125, lam, None)
        want, tol = ref.diff_attention(pool, q, 0.125, lam, None, 1e-5)
        within(out, want, tol)


@pytest.mark.parametrize("dtype,block,dim,L", [("bf16", 16, 64, [1, 200]), ("bf16", 32, 128, [700, 33]),
                                               ("bf16", 16, 128, [2500]), ("int8", 16, 128, [700, 33]),
                                               ("fp8", 32, 64, [300])])
@pytest.mark.parametrize("norm", [False, True])
def test_diff_of_maps_that_cancel(pkv, dtype, block, dim, L, norm):
    """Two maps that are nearly one, lambda near 1: the difference is a small
    part of either, and the errors of P count so many times more.  P as two
    bf16 numbers is off by 2^-16 (2^-8 of what the first left, itself 2^-8 of P);
    as fp16 by 2^-11, and by 2^-25 of the sum below fp16's normal numbers, which
    over 700 tokens is 2^-15; the fp32 sums over a warp's third of the tokens,
    truncated, by 2^-23 a step of 16 and the rescaling, 2^-16 over 2500."""
    pool = ref.Pool(L, 2, dim, block, dtype, seed=8)
    q = pool.randn(len(L), 8, dim, scale=2.0)
    ref.raw(pool.k)[:, :, 1] = ref.raw(pool.k)[:, :, 0]
    if dtype != "bf16":
        pool.k_scale[:, 1] = pool.k_scale[:, 0]
    q[:, 1::2] = (q[:, ::2].float() * (1 + 0.1 * torch.randn(q[:, ::2].shape, generator=pool.g))).to(torch.bfloat16)
    lam = torch.full((4,), 0.96875)
    weight = 0.5 + torch.rand(2 * dim, generator=pool.g) if norm else None
    out = diff(pkv, pool, q, dim ** -0.5, lam, weight)
    p_off = 2.0 ** -16 + 2.0 ** -16 if dtype == "bf16" else 2.0 ** -11 + 2.0 ** -15 + 2.0 ** -16
    want, tol = ref.diff_attention(pool, q, dim ** -0.5, lam, weight, 1e-5, p_off)
    within(out, want, tol)


@pytest.mark.parametrize("dim,L", [(64, 40), (128, 700)])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_diff_values_that_are_not_finite(pkv, dim, L, value):
    """One such value makes its element not finite (NaN, the difference of two
    infinities, under a lambda that is not negative) and no other; with a norm
    it reaches its row, and no other row."""
    pool = ref.Pool([L, 50], 4, dim, 16, "bf16", seed=3)
    q = pool.randn(2, 8, dim, scale=2.0)
    lam = torch.tensor([0.4, -0.4, 0.0, 0.9])
    want, tol = ref.diff_attention(pool, q, dim ** -0.5, lam, None, 1e-5)
    at = L // 2
    pool.v[pool.tables[0, at // 16].item(), at % 16, 1, 5] = value   # element dim + 5 of KV head 0's heads
    out = diff(pkv, pool, q, dim ** -0.5, lam, None).cpu()
    assert torch.isnan(out[0, 0, dim + 5]) and not torch.isfinite(out[0, 1, dim + 5])
    out[0, :2, dim + 5] = want[0, :2, dim + 5]
    within(out, want, tol)
    out = diff(pkv, pool, q, dim ** -0.5, lam, torch.ones(2 * dim)).cpu()
    assert torch.isnan(out[0, 0]).all() and torch.isfinite(out[0, 2:].float()).all() and torch.isfinite(out[1].float()).all()
