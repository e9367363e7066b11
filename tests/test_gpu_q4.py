"""GPU parity of the rotated append, the 4-bit pool with its attention, and the
verification of drafted tokens, against their 64-bit references.  Rows, codes,
scales and tokens are compared exactly; the attention's tolerance is the
reference's own bound (q4_reference.attention)."""
import math

import pytest
import torch

import q4_reference as ref

pytestmark = pytest.mark.gpu

SHAPES = [(16, 64), (32, 64), (16, 128), (32, 128)]


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_97_gb300 as pkv
    pkv.load()
    return pkv


@pytest.fixture(autouse=True)
def clean_status(pkv):
    pkv.get_status()
    yield
    st, flags = pkv.get_status()
    assert flags == 0, f"status word 0x{flags:x}"


def flags_of(pkv):
    return pkv.get_status()[1]


def same_bits(got, want):
    return torch.equal(got.cpu().contiguous().view(torch.uint8), want.cpu().contiguous().view(torch.uint8))


def within(got, want, tol):
    off = (got.cpu().double() - want).abs()
    assert torch.isfinite(off).all()
    assert (off <= tol).all(), f"{(off / (tol + 1e-300)).max().item():.2f} of the bound"


def poison(n):
    return torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")


def starts(n):
    out = [0]
    for x in n:
        out.append(out[-1] + x)
    return torch.tensor(out, dtype=torch.int32)


# --------------------------------------------------------------------------
# Rotated append and reading back
# --------------------------------------------------------------------------

class Step:
    """New rows of sequences with L tokens, n of them new, in one projection."""

    def __init__(self, L, n, hq, hkv, d, block, rotary, axes=1, max_pos=600, seed=0, packed=True, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.L, self.n, self.block, self.d, self.hkv = L, n, block, d, hkv
        T = sum(n)
        self.T, self.start = T, starts(n)
        x = (scale * torch.randn((T + 2, hq + 2 * hkv, d), generator=g)).to(torch.bfloat16)
        self.x = x
        self.q, self.k, self.v = x[:T, :hq], x[:T, hq:hq + hkv], x[:T, hq + hkv:]
        dev = x.cuda() if packed else None
        self.dq, self.dk, self.dv = ((dev[:T, :hq], dev[:T, hq:hq + hkv], dev[:T, hq + hkv:]) if packed else
                                     (self.q.cuda().contiguous(), self.k.cuda().contiguous(), self.v.cuda().contiguous()))
        nb = [(m + block - 1) // block for m in L]
        self.num_blocks = sum(nb) + 2
        perm = torch.randperm(self.num_blocks, generator=g).to(torch.int32)
        self.tables = torch.full((len(L), max(max(nb), 1)), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(nb):
            self.tables[b, :m] = perm[at:at + m]
            at += m
        self.seq = torch.repeat_interleave(torch.arange(len(L)), torch.tensor(n))
        self.pos = torch.cat([torch.arange(m - k, m) for m, k in zip(L, n)]) if T else torch.zeros(0, dtype=torch.long)
        self.blk, self.row = self.tables[self.seq, self.pos // block].long(), self.pos % block
        self.cos_sin = ref.table(max_pos, rotary) if rotary else None
        self.given = torch.randint(0, max_pos, (axes, T), generator=g, dtype=torch.int32) if axes > 1 else None
        half = rotary // 2
        self.sections = None if axes == 1 else [half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1)

    def where(self):
        return self.given if self.given is not None else self.pos[None]

    def rotated(self, x, interleaved):
        return x if self.cos_sin is None else ref.rotated(x, self.cos_sin, self.where(), interleaved, self.sections)

    def how(self, interleaved=False):
        cs = None if self.cos_sin is None else self.cos_sin.cuda()
        return (cs, self.tables.cuda(), torch.tensor(self.L, dtype=torch.int32).cuda()), dict(
            positions=None if self.given is None else self.given.cuda(), sections=self.sections,
            interleaved=interleaved, query_start=self.start.cuda(), max_query_len=max(max(self.n), 1))


def expected_q4(s, k, v):
    """The pool's bytes after the append on a pool of 0xFF."""
    rec = torch.full((s.num_blocks, s.hkv, ref.record_bytes(s.block, s.d)), 0xFF, dtype=torch.uint8)
    at, nib = ref.group_word_nibble(s.d)
    half, par = s.block * s.d // 2, s.block * s.d // 16
    for i, x in enumerate((k, v)):
        c, scale, low = ref.quantise(x)
        b = torch.zeros(*c.shape[:-1], s.d // 2, dtype=torch.uint8)
        b[..., at[nib == 0]] = (c[..., nib == 0] + 16 * c[..., nib == 1]).to(torch.uint8)
        codes = rec[..., i * half:(i + 1) * half].unflatten(-1, (s.block, s.d // 2))
        pairs = rec[..., s.block * s.d + i * par:s.block * s.d + (i + 1) * par].unflatten(-1, (s.block, s.d // 16))
        pair = torch.stack((scale, low), dim=-1).to(torch.bfloat16).flatten(-2).contiguous().view(torch.uint8)
        for h in range(s.hkv):
            codes[s.blk, h, s.row] = b[:, h]
            pairs[s.blk, h, s.row] = pair[:, h]
    return rec


CASES = [  # L, n, rotary of 64 / 128, interleaved, axes
    ([1, 16, 17, 100, 33], [1, 1, 1, 1, 1], (64, 128), False, 1),
    ([40, 5, 130], [40, 0, 7], (32, 64), False, 1),
    ([70, 33], [9, 33], (64, 128), True, 1),
    ([50, 19], [50, 3], (48, 96), True, 3),
    ([50, 19], [50, 3], (16, 112), False, 3),
    ([37], [37], (64, 128), False, 4),
    ([20, 3], [4, 3], (0, 0), False, 1),
]


@pytest.mark.parametrize("block,dim", SHAPES)
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("kind", ["bf16", "int8", "fp8", "q4"])
def test_append_rotary(pkv, block, dim, case, kind):
    L, n, rotary, inter, axes = CASES[case]
    hq, hkv = (6, 3) if case % 2 else (8, 1)
    s = Step(L, n, hq, hkv, dim, block, rotary[dim == 128], axes, seed=case, packed=case != 2)
    q_out = torch.full((s.T + 2, hq, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    where, how = s.how(inter)
    want_q, k = s.rotated(s.q, inter), s.rotated(s.k, inter)
    if kind == "q4":
        kv = torch.full((s.num_blocks, hkv, ref.record_bytes(block, dim)), 0xFF, dtype=torch.uint8, device="cuda")
        pkv.append_rotary_q4(q_out[:s.T], s.dq, s.dk, s.dv, kv, *where, block, **how)
        assert same_bits(kv, expected_q4(s, k, s.v))
    else:
        dt = {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.float8_e4m3fn}[kind]
        caches = [torch.zeros((s.num_blocks, block, hkv, dim), dtype=dt, device="cuda") for _ in range(4)]
        sc = [None, None]
        if kind != "bf16":
            g = torch.Generator().manual_seed(1)
            sc = [((torch.rand((s.num_blocks, hkv), generator=g) + 0.5) / 40).cuda() for _ in range(2)]
        pkv.append_rotary(q_out[:s.T], s.dq, s.dk, s.dv, caches[0], caches[1], *where, k_scale=sc[0], v_scale=sc[1],
                          **how)
        slots = (s.blk * block + s.row).cuda()
        pkv.reshape_and_cache(k.contiguous().cuda(), s.v.contiguous().cuda(), caches[2], caches[3], slots, *sc)
        assert same_bits(caches[0], caches[2]) and same_bits(caches[1], caches[3])
    assert same_bits(q_out[:s.T], want_q)
    assert (q_out[s.T:] == 7).all()


def test_append_rotary_many_rows(pkv):
    """Enough tokens for four rows a lane group, an odd number of them."""
    L = [1500, 1201, 777]
    s = Step(L, [1500, 900, 777], 12, 2, 128, 16, 128, 3, max_pos=2000, seed=3)
    where, how = s.how()
    kv = torch.full((s.num_blocks, 2, ref.record_bytes(16, 128)), 0xFF, dtype=torch.uint8, device="cuda")
    q_out = torch.empty((s.T, 12, 128), dtype=torch.bfloat16, device="cuda")
    pkv.append_rotary_q4(q_out, s.dq, s.dk, s.dv, kv, *where, 16, **how)
    k = s.rotated(s.k, False)
    assert same_bits(q_out, s.rotated(s.q, False)) and same_bits(kv, expected_q4(s, k, s.v))
    # in place, and without queries
    kv2 = torch.full_like(kv, 0xFF)
    pkv.append_rotary_q4(s.dq, s.dq, s.dk, s.dv, kv2, *where, 16, **how)
    assert same_bits(s.dq, q_out) and same_bits(kv2, kv)
    kv2.fill_(0xFF)
    pkv.append_rotary_q4(None, None, s.dk, s.dv, kv2, *where, 16, **how)
    assert same_bits(kv2, kv)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "q4"])
def test_append_rotary_rounds_every_step(pkv, inter, kind):
    """Enough elements that a product and a sum rounded as one would show (they
    differ in one bf16 element of some 10^4)."""
    s = Step([900], [900], 8, 8, 128, 16, 128, 1, max_pos=1000, seed=31)
    where, how = s.how(inter)
    q_out = torch.empty((900, 8, 128), dtype=torch.bfloat16, device="cuda")
    k = s.rotated(s.k, inter)
    if kind == "q4":
        kv = torch.full((s.num_blocks, 8, ref.record_bytes(16, 128)), 0xFF, dtype=torch.uint8, device="cuda")
        pkv.append_rotary_q4(q_out, s.dq, s.dk, s.dv, kv, *where, 16, **how)
        assert same_bits(kv, expected_q4(s, k, s.v))
    else:
        kc, vc = (torch.zeros((s.num_blocks, 16, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        pkv.append_rotary(q_out, s.dq, s.dk, s.dv, kc, vc, *where, **how)
        assert same_bits(kc[s.blk.cuda(), s.row.cuda()], k) and same_bits(vc[s.blk.cuda(), s.row.cuda()], s.v)
    assert same_bits(q_out, s.rotated(s.q, inter))


def test_append_one_token_without_offsets(pkv):
    L = [1, 16, 33, 64]
    s = Step(L, [1] * 4, 4, 2, 64, 16, 64, seed=9)
    (cs, bt, sl), how = s.how()
    kv = [torch.zeros((s.num_blocks, 2, ref.record_bytes(16, 64)), dtype=torch.uint8, device="cuda") for _ in "ab"]
    q = [torch.empty((4, 4, 64), dtype=torch.bfloat16, device="cuda") for _ in "ab"]
    pkv.append_rotary_q4(q[0], s.dq, s.dk, s.dv, kv[0], cs, bt, sl, 16)
    pkv.append_rotary_q4(q[1], s.dq, s.dk, s.dv, kv[1], cs, bt, sl, 16, **how)
    assert same_bits(q[0], q[1]) and same_bits(kv[0], kv[1])


def test_q4_values_where_they_are_awkward(pkv):
    """Equal values, zeros of both signs, NaN, infinities, huge and tiny ranges."""
    d = 64
    rows = [torch.full((d,), 3.0), torch.zeros(d), -torch.zeros(d), torch.linspace(-1, 1, d)]
    rows += [torch.cat((torch.tensor([math.nan, math.inf, -math.inf, 1e38, -3e38]), torch.ones(d - 5)))]
    rows += [torch.linspace(1e-40, 3e-38, d), torch.linspace(-3e38, 3e38, d), torch.full((d,), math.nan)]
    rows += [torch.linspace(100.0, 101.0, d), torch.linspace(0, 15, d).round()]
    x = torch.stack(rows).to(torch.bfloat16)[:, None].contiguous()
    T = x.shape[0]
    kv = torch.zeros((1, 1, ref.record_bytes(16, d)), dtype=torch.uint8, device="cuda")
    bt, sl = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([T], dtype=torch.int32, device="cuda")
    qs = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    pkv.append_rotary_q4(None, None, x.cuda(), x.flip(0).cuda(), kv, None, bt, sl, 16, query_start=qs, max_query_len=T)
    (kc, ks, km), (vc, vs, vm) = ref.unpack(kv.cpu(), 16, d)
    for (c, s, m), want in (((kc, ks, km), x), ((vc, vs, vm), x.flip(0))):
        wc, ws, wm = ref.quantise(want[:, 0])
        assert torch.equal(c[0, 0, :T], wc) and torch.equal(s[0, 0, :T], ws.double()) and torch.equal(m[0, 0, :T], wm.double())
    # half a scale at most (the fp32 steps add 2^-20 of 15 scales), and the values that read_q4 gives
    value = km[0, 0, :T] + ks[0, 0, :T] * kc[0, 0, :T]
    fine = torch.nan_to_num(x[:, 0].double(), nan=0.0).clamp(-2.0 ** 126, 2.0 ** 126)
    assert ((value - fine).abs() <= ks[0, 0, :T] * (0.5 + 2.0 ** -16)).all()
    out = [torch.empty((T, 1, d), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    pkv.read_q4(*out, kv, bt, sl, 16, query_start=qs, max_query_len=T)
    assert same_bits(out[0][:, 0], value.float().to(torch.bfloat16))


@pytest.mark.parametrize("block,dim", SHAPES)
def test_read_and_copy(pkv, block, dim):
    pool = ref.Pool4([70, 1, 33], 3, dim, block, seed=2)
    kv, bt, sl = pool.on()
    n = [70, 0, 5]
    out = [torch.full((77, 3, dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    pkv.read_q4(*out, kv, bt, sl, block, query_start=starts(n).cuda(), max_query_len=70)
    for i in range(2):
        want = []
        for b in (0, 2):
            c, s, m = pool.rows(b, pool.L[b])[i]
            want.append((m + s * c).float().to(torch.bfloat16).transpose(0, 1)[-n[b]:])
        assert same_bits(out[i][:75], torch.cat(want)) and (out[i][75:] == 7).all()
    before = kv.clone()
    free = [i for i in range(pool.num_blocks) if i not in pool.records]
    src = list(pool.records)[:2]
    pairs = torch.tensor([[src[0], free[0]], [src[1], free[1]], [src[0], src[0]]], dtype=torch.int32, device="cuda")
    pkv.copy_blocks_q4(kv, pairs, block)
    before[free[0]], before[free[1]] = before[src[0]], before[src[1]]
    assert same_bits(kv, before)


def test_append_faults_are_flagged(pkv):
    """Bad lengths, blocks and positions: nothing stored, zeros in q_out, other sequences right."""
    L, n = [40, 20, 30, 9], [4, 3, 2, 9]
    s = Step(L, n, 4, 2, 64, 16, 64, 2, max_pos=100, seed=4)
    (cs, bt, sl), how = s.how()
    kv = torch.full((s.num_blocks, 2, ref.record_bytes(16, 64)), 0xFF, dtype=torch.uint8, device="cuda")
    q_out = torch.full((s.T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    sl[0] = 3                                       # fewer tokens than new ones
    bt[1, 1] = s.num_blocks                         # outside the pool (tokens 17 .. 19)
    how["positions"][1, 7] = 100                    # sequence 2's first token, second axis
    pkv.append_rotary_q4(q_out, s.dq, s.dk, s.dv, kv, cs, bt, sl, 16, **how)
    assert flags_of(pkv) == pkv.FLAG_BAD_SEQ_LEN | pkv.FLAG_BAD_BLOCK | pkv.FLAG_BAD_INDEX
    want_q = s.rotated(s.q, False).clone()
    want_q[:4] = 0
    want_q[7] = 0
    assert same_bits(q_out, want_q)
    want = expected_q4(s, s.rotated(s.k, False), s.v)
    ok = torch.ones(s.T, dtype=torch.bool)
    ok[:8] = False
    blank = torch.full_like(want, 0xFF)
    keep = Step.__new__(Step)
    keep.__dict__.update(s.__dict__)
    keep.blk, keep.row = s.blk[ok], s.row[ok]
    del blank
    assert same_bits(kv, expected_q4(keep, s.rotated(s.k, False)[ok], s.v[ok]))
    out = [torch.full((s.T, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    pkv.read_q4(*out, kv, bt, sl, 16, query_start=how["query_start"], max_query_len=9)
    assert flags_of(pkv) == pkv.FLAG_BAD_SEQ_LEN | pkv.FLAG_BAD_BLOCK
    assert (out[0][:7] == 0).all()


# --------------------------------------------------------------------------
# Attention over the 4-bit pool
# --------------------------------------------------------------------------

def decode(pkv, pool, q, scale, max_len=None, dev=None):
    kv, bt, sl = dev or pool.on()
    hq = q.shape[1]
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = poison(pkv.q4_workspace_bytes(hq, pool.heads, pool.dim))
    return pkv.paged_attention_decode_q4(out, q.cuda(), kv, bt, sl, pool.block, max_len or max(max(pool.L), 1), scale, ws)


def multi(pkv, pool, q, n, scale, max_len=None, max_n=None, dev=None, room=None):
    """room: sequences whose long queries find room in the workspace (None: none, -1: all)."""
    kv, bt, sl = dev or pool.on()
    hq, most = q.shape[1], max_n or max(max(n), 1)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    size = pkv.q4_workspace_bytes(hq, pool.heads, pool.dim, most)
    if room is not None:
        longest = max_len or max(max(pool.L), 1)
        size = pkv.q4_long_workspace_bytes(len(n), q.shape[0], most, longest, hq, pool.heads, pool.dim)
        if room > 0:
            slot = (longest + 127) // 128 * pool.heads * (512 * pool.dim + 8)
            size = pkv.q4_workspace_bytes(hq, pool.heads, pool.dim, most) + room * slot + 4 * (3 * len(n) + 2) + 1024
    ws = poison(size)
    return pkv.paged_attention_multi_q4(out, q.cuda(), kv, bt, sl, starts(n).cuda(), pool.block,
                                        max_len or max(max(pool.L), 1), most, scale, ws)


def check(out, pool, q, n, scale, wide=False):
    at = 0
    for b, m in enumerate(n):
        if m == 0:
            continue
        L = pool.L[b]
        want, tol = ref.attention(pool.rows(b, L), q[at:at + m], scale, torch.arange(L - m, L),
                                  wide and m * q.shape[1] // pool.heads >= 128)
        within(out[at:at + m], want, tol)
        at += m


@pytest.mark.parametrize("block,dim", SHAPES)
@pytest.mark.parametrize("group", [1, 3, 4, 8])
@pytest.mark.parametrize("bound", [0, 4096])
def test_decode(pkv, block, dim, group, bound):
    """One CTA per sequence, and (a larger bound) ranges over the batch."""
    L = [1, 2, 15, 16, 17, 31, 32, 33, 100, 257]
    pool = ref.Pool4(L, 2, dim, block, seed=group, width=256)
    q = pool.randn(len(L), 2 * group, dim, scale=2.0)
    check(decode(pkv, pool, q, dim ** -0.5, bound or None), pool, q, [1] * len(L), dim ** -0.5)


@pytest.mark.parametrize("block,dim,heads,L", [(16, 128, 1, [3000]), (16, 64, 8, [2500, 1, 900, 4000]),
                                               (32, 128, 2, [5000, 4100]), (32, 64, 5, [700] * 7),
                                               (16, 128, 700, [600])])
def test_decode_ranges(pkv, block, dim, heads, L):
    """Sequences cut by the ranges, one over many CTAs, more KV heads than a wave holds."""
    pool = ref.Pool4(L, heads, dim, block, seed=5)
    q = pool.randn(len(L), heads * (2 if heads < 100 else 1), dim, scale=2.0)
    check(decode(pkv, pool, q, dim ** -0.5, max(max(L), 513)), pool, q, [1] * len(L), dim ** -0.5)


def test_decode_many_short_sequences(pkv):
    g = torch.Generator().manual_seed(3)
    L = torch.randint(1, 40, (700,), generator=g).tolist()
    L[17], L[600] = 900, 513
    pool = ref.Pool4(L, 1, 64, 16, seed=6)
    q = pool.randn(len(L), 4, 64, scale=2.0)
    check(decode(pkv, pool, q, 0.125), pool, q, [1] * len(L), 0.125)


@pytest.mark.parametrize("block,dim", SHAPES)
@pytest.mark.parametrize("group,n", [(4, [5, 1, 0, 2, 5]), (8, [1, 1, 1, 1, 1]), (1, [8, 3, 1, 7, 2]),
                                     (3, [10, 2, 9, 1, 4]), (5, [6, 6, 1, 0, 3]), (8, [17, 1, 40, 2, 33]),
                                     (2, [60, 33, 0, 17, 100])])
@pytest.mark.parametrize("bound", [0, 4096])
def test_multi(pkv, block, dim, group, n, bound):
    """Every number of column tiles, with causal limits inside blocks and tiles."""
    L = [100, 17, 3, 33, 130]
    n = [min(a, b) for a, b in zip(n, L)]
    pool = ref.Pool4(L, 2, dim, block, seed=group, width=256)
    q = pool.randn(sum(n), 2 * group, dim, scale=2.0)
    check(multi(pkv, pool, q, n, dim ** -0.5, bound or None), pool, q, n, dim ** -0.5)


@pytest.mark.parametrize("dim,heads,group,L,n", [(128, 2, 4, [2000, 1100], [5, 3]), (64, 1, 8, [1500], [300]),
                                                 (128, 2, 4, [900, 700], [900, 700]), (128, 8, 2, [600], [600]),
                                                 (64, 2, 1, [1024, 513], [16, 513])])
def test_multi_long(pkv, dim, heads, group, L, n):
    """Long contexts and prompts, cut by ranges and not."""
    pool = ref.Pool4(L, heads, dim, 16, seed=8)
    q = pool.randn(sum(n), heads * group, dim, scale=2.0)
    check(multi(pkv, pool, q, n, dim ** -0.5), pool, q, n, dim ** -0.5)


@pytest.mark.parametrize("block,dim", SHAPES)
@pytest.mark.parametrize("heads,group,L,n", [
    (1, 1, [128], [128]), (2, 4, [300, 40, 257, 33, 128], [40, 1, 0, 33, 32]), (1, 8, [500, 16], [33, 16]),
    (2, 3, [600, 90, 700, 45], [600, 3, 50, 44]), (3, 5, [1200], [1200]), (1, 2, [70, 64, 1000], [63, 64, 129]),
    (8, 4, [900, 700], [900, 5])])
@pytest.mark.parametrize("room", [-1, 1])
def test_multi_tensor_cores(pkv, block, dim, heads, group, L, n, room):
    """Long queries through widened operands, beside short ones, at the border of
    128 rows, with chunks, tiles and pairs of tiles that end anywhere, and with room
    for one sequence only."""
    pool = ref.Pool4(L, heads, dim, block, seed=len(L) + group)
    q = pool.randn(sum(n), heads * group, dim, scale=2.0)
    check(multi(pkv, pool, q, n, dim ** -0.5, room=room), pool, q, n, dim ** -0.5, wide=True)


@pytest.mark.parametrize("group,dim", [(8, 64), (4, 128), (3, 64)])
def test_multi_tensor_cores_many_sequences(pkv, group, dim):
    """More long sequences than a warp has lanes, of equal and unequal chunks, one of
    them bad, short ones between them, and rows that belong to none at the end."""
    g = torch.Generator().manual_seed(group)
    L = (torch.randint(64, 420, (90,), generator=g)).tolist()
    n = [min(x, int(m)) for x, m in zip(L, torch.randint(1, 120, (90,), generator=g).tolist())]
    n[40], n[41], n[89] = 0, 1, min(L[89], 64)
    pool = ref.Pool4(L, 2, dim, 16, seed=33)
    q = pool.randn(sum(n), 2 * group, dim, scale=2.0)
    kv, bt, sl = pool.on()
    bt[7, 0] = -5
    out = multi(pkv, pool, q, n, dim ** -0.5, dev=(kv, bt, sl), room=-1)
    assert flags_of(pkv) == pkv.FLAG_BAD_BLOCK
    at = sum(n[:7])
    assert (out[at:at + n[7]] == 0).all()
    bt[7, 0] = pool.tables[7, 0]
    again = multi(pkv, pool, q, n, dim ** -0.5, dev=(kv, bt, sl), room=-1)
    assert same_bits(again[:at], out[:at].cpu()) and same_bits(again[at + n[7]:], out[at + n[7]:].cpu())
    check(again, pool, q, n, dim ** -0.5, wide=True)


@pytest.mark.parametrize("scale,vspread,kspread", [(-0.2, 1.0, 1.0), (0.0, 1.0, 1.0), (3.0, 1.0, 1.0),
                                                   (0.1, 1e-20, 1e10), (0.1, 1e20, 1e-10)])
def test_multi_tensor_cores_scales(pkv, scale, vspread, kspread):
    pool = ref.Pool4([700, 300], 2, 128, 16, seed=19, vscale=lambda s, g: vspread, kscale=lambda s, g: kspread)
    q = (pool.randn(350, 8, 128).float() / kspread).to(torch.bfloat16)
    check(multi(pkv, pool, q, [150, 200], scale, room=-1), pool, q, [150, 200], scale, wide=True)


@pytest.mark.parametrize("scale,qsize", [(0.0, 1.0), (0.1, 2.0 ** -100), (-1e-30, 1e-20)])
@pytest.mark.parametrize("kspread", [0.0, 1e-25])
def test_multi_tensor_cores_scores_of_nothing(pkv, scale, qsize, kspread):
    """A factor of the scores below fp32's range: a masked score is still none."""
    pool = ref.Pool4([200, 300], 2, 64, 16, seed=34, kscale=lambda s, g: kspread)
    q = (pool.randn(190, 8, 64).float() * qsize).to(torch.bfloat16)
    check(multi(pkv, pool, q, [150, 40], scale, room=-1), pool, q, [150, 40], scale, wide=True)


def test_multi_tensor_cores_rising_scores(pkv):
    """Scores and V's magnitudes that rise along the sequence move the references
    in every chunk."""
    def rising(shape, g):
        return torch.exp2(torch.arange(shape[0]).view(-1, 1, 1, 1) / 4.0).expand(shape)
    pool = ref.Pool4([1000], 1, 64, 16, seed=20, vscale=rising, kscale=lambda s, g: rising(s, g) ** 0.25)
    q = pool.randn(200, 4, 64)
    check(multi(pkv, pool, q, [200], 1.0, room=-1), pool, q, [200], 1.0, wide=True)


def test_multi_tensor_cores_faults(pkv):
    """Bad blocks, lengths and offsets among long queries; repeats give the same bits."""
    L, n = [400, 300, 500, 260], [100, 150, 200, 64]
    pool = ref.Pool4(L, 2, 64, 16, seed=21)
    q = pool.randn(sum(n), 8, 64)
    kv, bt, sl = pool.on()
    first = multi(pkv, pool, q, n, 0.125, dev=(kv, bt, sl), room=-1)
    assert same_bits(first, multi(pkv, pool, q, n, 0.125, dev=(kv, bt, sl), room=-1).cpu())
    bt[0, 3], sl[2] = pool.num_blocks, 501
    out = multi(pkv, pool, q, n, 0.125, dev=(kv, bt, sl), room=-1)
    assert flags_of(pkv) == pkv.FLAG_BAD_BLOCK | pkv.FLAG_BAD_SEQ_LEN
    assert (out[:100] == 0).all() and (out[250:450] == 0).all()
    assert same_bits(out[100:250], first[100:250].cpu()) and same_bits(out[450:], first[450:].cpu())


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales_of_the_scores(pkv, scale):
    pool = ref.Pool4([700, 40], 2, 64, 16, seed=11)
    q = pool.randn(2, 6, 64)
    check(decode(pkv, pool, q, scale), pool, q, [1, 1], scale)


@pytest.mark.parametrize("spread", [1e-30, 1e-6, 1e4, 1e30])
@pytest.mark.parametrize("L", [[300, 33], [700, 600]])
def test_any_v_scale(pkv, spread, L):
    """V scales all tiny or huge, keys' scales likewise with queries to match."""
    pool = ref.Pool4(L, 2, 128, 16, seed=12, vscale=lambda shape, g: spread, kscale=lambda shape, g: 1 / spread)
    q = (pool.randn(2, 8, 128).float() * spread).to(torch.bfloat16)
    check(decode(pkv, pool, q, 0.1), pool, q, [1, 1], 0.1)


def test_mixed_v_scales(pkv):
    """Scales of a row 2^-20 .. 2^20 of its neighbours': the weights keep their precision."""
    def mixed(shape, g):
        return torch.exp2(torch.randint(-20, 21, shape, generator=g).float())
    pool = ref.Pool4([400, 700], 2, 128, 16, seed=13, vscale=mixed)
    q = pool.randn(2, 8, 128, scale=3.0)
    check(decode(pkv, pool, q, 0.1), pool, q, [1, 1], 0.1)


@pytest.mark.parametrize("block,dim", SHAPES)
@pytest.mark.parametrize("n,room", [(1, None), (6, None), (150, None), (150, -1)])
@pytest.mark.parametrize("L", [300, 900])
@pytest.mark.parametrize("small_first", [True, False])
def test_values_far_apart(pkv, block, dim, n, room, L, small_first):
    """Tokens with nearly all of the weight and values of 2^-100 beside tokens of
    nearly no weight and values of 2^100: the weights' sum is the first ones' although
    the products' reference is the second ones'."""
    def split(small, large):
        def factor(shape, g):
            at = torch.arange(shape[0])[:, None, None, None] * block + torch.arange(block)[:, None]
            return torch.where((at < L // 2) == small_first, small, large).expand(shape)
        return factor
    # positive keys: the first kind's scores are 8 to 25, the others' within 0.03
    pool = ref.Pool4([L], 2, dim, block, seed=31, low=0.0, kscale=split(1.0, 1e-3), vscale=split(2.0 ** -100, 2.0 ** 100))
    q = torch.ones(n, 8, dim, dtype=torch.bfloat16)
    scale = 6.4 / dim
    got = decode(pkv, pool, q, scale) if n == 1 else multi(pkv, pool, q, [n], scale, room=room)
    check(got, pool, q, [n], scale, wide=True)    # (the smaller workspace has room for one as well)


def test_multi_tensor_cores_largest_values(pkv):
    """Values up to nearly the format's 2^126."""
    pool = ref.Pool4([300], 1, 64, 16, seed=32, vscale=lambda shape, g: 2.0 ** 123)
    q = pool.randn(50, 4, 64)
    check(multi(pkv, pool, q, [50], 0.125, room=-1), pool, q, [50], 0.125, wide=True)


def test_rows_of_equal_values(pkv):
    """Zero rows and constant rows have the least scale there is."""
    x = torch.zeros((600, 2, 64), dtype=torch.bfloat16)
    x[300:] = 2.0
    kv = torch.full((40, 2, ref.record_bytes(16, 64)), 0xFF, dtype=torch.uint8, device="cuda")
    bt = torch.arange(38, dtype=torch.int32, device="cuda")[None].contiguous()
    sl, qs = torch.tensor([600], dtype=torch.int32, device="cuda"), torch.tensor([0, 600], dtype=torch.int32, device="cuda")
    pkv.append_rotary_q4(None, None, x.cuda(), x.cuda(), kv, None, bt, sl, 16, query_start=qs, max_query_len=600)
    q = torch.randn((1, 4, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    out = torch.empty_like(q, device="cuda")
    pkv.paged_attention_decode_q4(out, q.cuda(), kv, bt, sl, 16, 600, 0.125, poison(pkv.q4_workspace_bytes(4, 2, 64)))
    rows = ref.rows_of(kv.cpu()[:38], 16, 64, 600)
    want, tol = ref.attention(rows, q, 0.125, torch.tensor([599]))
    within(out, want, tol)


def test_queries_of_any_size(pkv):
    """A head's queries 2^60 times another's are exact on their own; an infinity
    leaves its own head NaN and the others right."""
    pool = ref.Pool4([50, 600], 1, 64, 16, seed=14)
    q = pool.randn(2, 4, 64)
    q[:, 1] *= 2.0 ** -20
    q[:, 2] = 0
    check(decode(pkv, pool, q, 0.1), pool, q, [1, 1], 0.1)
    tiny = (q.float() * 2.0 ** -100).to(torch.bfloat16)
    check(decode(pkv, pool, tiny, 2.0 ** 97), pool, tiny, [1, 1], 2.0 ** 97)
    q[0, 3, 5] = math.inf
    out = decode(pkv, pool, q, 0.1).cpu()
    assert torch.isnan(out[0, 3]).all()
    want, tol = ref.attention(pool.rows(0, 50), q[:1, :3].clone(), 0.1, torch.tensor([49]))
    within(out[:1, :3], want, tol)


def test_faults_are_flagged(pkv):
    """Bad lengths and blocks zero their sequence's rows, in both ways of running."""
    for bound in (256, 4096):
        L = [100, 40, 33, 200, 16]
        pool = ref.Pool4(L, 2, 64, 16, seed=15, width=256)
        q = pool.randn(5, 8, 64)
        kv, bt, sl = pool.on()
        sl[1], sl[4] = 0, bound + 1
        bt[3, 7] = -5
        out = decode(pkv, pool, q, 0.125, bound, (kv, bt, sl))
        assert flags_of(pkv) == pkv.FLAG_BAD_BLOCK | pkv.FLAG_BAD_SEQ_LEN
        assert (out[[1, 3, 4]] == 0).all()
        for b in (0, 2):
            want, tol = ref.attention(pool.rows(b, L[b]), q[b:b + 1], 0.125, torch.tensor([L[b] - 1]))
            within(out[b:b + 1], want, tol)
        # several queries: more than the bound, more than tokens, offsets outside
        n = [3, 3, 3, 3, 3]
        q = pool.randn(15, 8, 64)
        sl[1] = 2
        out = multi(pkv, pool, q, n, 0.125, bound, 3, (kv, bt, sl))
        assert flags_of(pkv) == pkv.FLAG_BAD_BLOCK | pkv.FLAG_BAD_SEQ_LEN
        assert (out[3:6] == 0).all() and (out[9:15] == 0).all()
        want, tol = ref.attention(pool.rows(2, 33), q[6:9], 0.125, torch.arange(30, 33))
        within(out[6:9], want, tol)
        start = torch.tensor([0, 3, 1, 6, 9, 16], dtype=torch.int32, device="cuda")
        out = torch.full((15, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = poison(pkv.q4_workspace_bytes(8, 2, 64, 8))
        bt[3, 7] = pool.tables[3, 7]
        sl.copy_(pool.seq_lens)
        pkv.paged_attention_multi_q4(out, q.cuda(), kv, bt, sl, start, 16, bound, 8, 0.125, ws)
        assert flags_of(pkv) == pkv.FLAG_BAD_SEQ_LEN
        assert (out[9:] == 7).all()                 # offsets past the rows: left as they are
        want, tol = ref.attention(pool.rows(3, 200), q[6:9], 0.125, torch.arange(197, 200))
        within(out[6:9], want, tol)


def test_ranges_are_counted_in_32_bits(pkv):
    """A call whose ranges might pass 2^30 blocks is refused (and nothing is launched)."""
    p = torch.zeros(16, dtype=torch.uint8, device="cuda").data_ptr()
    st = pkv.load().paged_attention_multi_q4(p, p, p, p, 1 << 26, p, p, 2, 1 << 22, 40, 65535, 65535, 64, 64, 16, 1 << 30,
                                             0.1, None, 0, None)
    assert st == pkv.KV_ERR_INVALID_ARG and "2^30" in pkv.load().pagedkv_last_error().decode()


def test_blocks_past_4_gib(pkv):
    blocks = (1 << 32) // (8 * ref.record_bytes(16, 128)) + 500
    pool = ref.Pool4([300, 700], 8, 128, 16, seed=16, num_blocks=blocks)
    q = pool.randn(2, 16, 128)
    check(decode(pkv, pool, q, 0.1), pool, q, [1, 1], 0.1)


def test_repeats_streams_and_graphs(pkv):
    """Equal bits from equal inputs, on two streams at once and in a replayed graph."""
    pool = ref.Pool4([1500, 40, 900], 2, 128, 16, seed=17)
    dev = pool.on()
    q = pool.randn(9, 8, 128).cuda()
    n, qs = [3, 1, 5], starts([3, 1, 5]).cuda()
    size = max(pkv.q4_workspace_bytes(8, 2, 128, 5), pkv.q4_workspace_bytes(8, 2, 128))
    first_m = multi(pkv, pool, q, n, 0.1, dev=dev)
    first_d = decode(pkv, pool, q[:3], 0.1, dev=dev)
    kv, bt, sl = dev
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q) for _ in range(2)]
    wss = [poison(size) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                pkv.paged_attention_multi_q4(outs[i], q, kv, bt, sl, qs, 16, 1500, 5, 0.1, wss[i])
    torch.cuda.synchronize()
    assert all(same_bits(o, first_m) for o in outs)
    g = torch.cuda.CUDAGraph()
    out_d = torch.empty_like(q[:3])
    with torch.cuda.graph(g):
        pkv.paged_attention_multi_q4(outs[0], q, kv, bt, sl, qs, 16, 1500, 5, 0.1, wss[0])
        pkv.paged_attention_decode_q4(out_d, q[:3], kv, bt, sl, 16, 1500, 0.1, wss[0])
    for _ in range(5):
        outs[0].zero_()
        out_d.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert same_bits(outs[0], first_m) and same_bits(out_d, first_d)


# --------------------------------------------------------------------------
# Verification of drafts
# --------------------------------------------------------------------------

def verify_case(n, V, dtype, seed, temperature=2.0, near=0.7):
    g = torch.Generator().manual_seed(seed)
    T, B = sum(n), len(n)
    logits = temperature * torch.randn((T, V), generator=g)
    st = starts(n)
    rows = torch.cat([torch.arange(int(st[b]), int(st[b + 1]) - 1) for b in range(B)]) if T else torch.zeros(0).long()
    draft = torch.softmax(logits[rows] + near * torch.randn((len(rows), V), generator=g), dim=1)
    tokens = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    if len(rows):
        tokens[rows + 1] = torch.multinomial(draft, 1, generator=g)[:, 0].to(torch.int32)
    return tokens, torch.softmax(logits, dim=1).to(dtype), draft.to(dtype), torch.rand(T, generator=g), st


def run_verify(pkv, tokens, target, draft, u, st, lens=None, max_n=None):
    T, B = tokens.shape[0], st.shape[0] - 1
    out = torch.full((T + 3,), 77, dtype=torch.int32, device="cuda")
    acc = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    lens = torch.arange(B, dtype=torch.int32) + 50 if lens is None else lens
    new = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    pkv.verify_drafts(out[:T], acc, tokens.cuda(), target.cuda(), None if draft is None else draft.cuda(), u.cuda(),
                      st.cuda(), max_query_len=max_n, seq_lens=lens.cuda(), new_lens=new)
    assert (out[T:] == 77).all()
    return out[:T].cpu(), acc.cpu(), new.cpu(), lens


def check_verify(got, tokens, target, draft, u, st):
    out, acc, new, lens = got
    for b, (kept, z) in enumerate(ref.verify(tokens, target, draft, u, st)):
        r, n = int(st[b]), int(st[b + 1] - st[b])
        assert acc[b] == len(kept)
        if n == 0:
            assert new[b] == lens[b]
            continue
        assert new[b] == lens[b] - n + 1 + len(kept)
        assert out[r:r + len(kept)].tolist() == kept
        assert z[0] <= out[r + len(kept)] <= z[1]
        assert (out[r + len(kept) + 1:r + n] == -1).all()


@pytest.mark.parametrize("V", [1, 7, 100, 1000, 4096, 32000, 50257, 262144])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("probs", [True, False])
def test_verify(pkv, V, dtype, probs):
    n = [1, 6, 3, 2, 5]
    case = list(verify_case(n, V, dtype, V))
    if not probs:
        case[2] = None
    check_verify(run_verify(pkv, *case), *case)


@pytest.mark.parametrize("B,V", [(200, 1001), (700, 64), (1, 128256), (3, 400001)])
def test_verify_batches(pkv, B, V):
    n = [(i * 7) % 5 + 1 for i in range(B)]
    case = verify_case(n, V, torch.float32, B)
    check_verify(run_verify(pkv, *case), *case)


def test_verify_borders(pkv):
    """u of 0, just below 1, 1 and NaN; equal rows (every draft kept); a residual
    without weight; probability one and zero; a row without any."""
    V = 300
    tokens, p, q, u, st = verify_case([2] * 10, V, torch.float32, 5)
    q[0], u[0] = p[0], 0.999999                     # equal rows: kept whatever u is below 1
    u[3] = 0.0
    u[2], tokens[3], p[2], q[1] = 0.5, 9, 0.0, 0.0  # the target never: refused
    p[2, 250:] = 0.02
    q[1, 9] = 1.0
    u[5], u[7], u[9] = 1 - 2.0 ** -24, 1.0, float("nan")
    p[10] = 0.0                                     # no weight at all: refused, the last token
    p[12] = q[6] * 0.5                              # nothing left after the difference: from p
    u[12], u[13] = 0.9999, 0.3
    p[14, 5], q[7, 5] = float("nan"), float("nan")
    tokens[17] = V                                  # a draft outside the vocabulary
    tokens[19] = -1
    case = (tokens, p, q, u, st)
    got = run_verify(pkv, *case)
    assert flags_of(pkv) == pkv.FLAG_BAD_INDEX
    check_verify(got, *case)
    assert got[1][0] == 1 and got[0][10] == V - 1 and got[1][8] == 0 and got[1][9] == 0


def test_verify_long_drafts_and_none(pkv):
    n = [600, 1, 40]
    tokens, p, q, u, st = verify_case(n, 50, torch.float32, 6, near=0.0)
    u[:] = 0.5                                      # equal rows: every draft is kept
    case = (tokens, p, q, u, st)
    got = run_verify(pkv, *case, torch.tensor([700, 1, 40], dtype=torch.int32))
    check_verify(got, *case)
    assert got[1].tolist() == [599, 0, 39]
    # without probabilities of the drafts a sequence may have no query
    n = [3, 0, 2, 0]
    tokens, p, q, u, st = verify_case([3, 2], 50, torch.float32, 7)
    st = starts(n)
    case = (tokens, p, None, u, st)
    check_verify(run_verify(pkv, *case), *case)


def test_verify_faults(pkv):
    tokens, p, q, u, st = verify_case([3, 3, 3], 64, torch.float32, 8)
    lens = torch.tensor([10, 2, 10], dtype=torch.int32)
    out, acc, new, _ = run_verify(pkv, tokens, p, q, u, st, lens)
    assert flags_of(pkv) == pkv.FLAG_BAD_SEQ_LEN
    assert acc[1] == 0 and new[1] == 2 and (out[3:6] == -1).all()
    want = ref.verify(tokens, p, q, u, st)
    assert [int(acc[0]), int(acc[2])] == [len(want[0][0]), len(want[2][0])]
    out, acc, new, _ = run_verify(pkv, tokens, p, q, u, st, max_n=2)
    assert flags_of(pkv) == pkv.FLAG_BAD_SEQ_LEN and (out == -1).all()
    bad = torch.tensor([0, 3, 2, 12], dtype=torch.int32)
    out, acc, new, _ = run_verify(pkv, tokens, p, q, u, bad)
    assert flags_of(pkv) == pkv.FLAG_BAD_SEQ_LEN and acc[1] == 0 and acc[2] == 0


def test_verify_lengths_in_place(pkv):
    n = [5] * 64
    tokens, p, q, u, st = verify_case(n, 32000, torch.float32, 9)
    lens = torch.full((64,), 5, dtype=torch.int32, device="cuda")
    out, acc = torch.empty(320, dtype=torch.int32, device="cuda"), torch.empty(64, dtype=torch.int32, device="cuda")
    args = [x.cuda() for x in (tokens, p, q, u, st)]
    for _ in range(10):
        lens.fill_(5)
        pkv.verify_drafts(out, acc, *args, seq_lens=lens, new_lens=lens)
        assert torch.equal(lens, acc + 1)


# --------------------------------------------------------------------------
# Together
# --------------------------------------------------------------------------

def test_speculative_steps_over_a_4_bit_cache(pkv):
    """Prompts, then speculative steps: rotated append of the last token and its
    drafts, attention, verification, and the next step on the lengths it leaves
    (the refused drafts' rows are written over); a fork's block is copied first."""
    g = torch.Generator().manual_seed(21)
    B, hq, hkv, d, bs, V, most = 3, 8, 2, 128, 16, 97, 4
    pool = pkv.KVPool(64, bs, hkv, d)
    lens = [37, 16, 5]
    bt = torch.full((B, 12), -1, dtype=torch.int32)
    for b in range(B):
        bt[b, :] = torch.tensor(pool.alloc(12))
    kv = torch.full((64, hkv, pkv.q4_record_bytes(bs, d)), 0xFF, dtype=torch.uint8, device="cuda")
    cs = ref.table(256, d).cuda()
    keys = [torch.zeros((0, hkv, d), dtype=torch.bfloat16) for _ in range(B)]
    vals = [x.clone() for x in keys]
    cs_cpu = cs.cpu()
    ws = poison(pkv.q4_workspace_bytes(hq, hkv, d, 64))
    tables = bt.cuda()

    def step(n, lens):
        T = sum(n)
        x = torch.randn((T, hq + 2 * hkv, d), generator=g).to(torch.bfloat16)
        dx, st = x.cuda(), starts(n).cuda()
        sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q = torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda")
        pkv.append_rotary_q4(q, dx[:, :hq], dx[:, hq:hq + hkv], dx[:, hq + hkv:], kv, cs, tables, sl, bs,
                             query_start=st, max_query_len=max(n))
        out = torch.empty_like(q)
        pkv.paged_attention_multi_q4(out, q, kv, tables, sl, st, bs, 192, max(n), d ** -0.5, ws)
        at = 0
        for b in range(B):
            pos = torch.arange(lens[b] - n[b], lens[b])
            keys[b] = torch.cat((keys[b][:lens[b] - n[b]],
                                 ref.rotated(x[at:at + n[b], hq:hq + hkv], cs_cpu, pos[None])))
            vals[b] = torch.cat((vals[b][:lens[b] - n[b]], x[at:at + n[b], hq + hkv:]))
            rows = []
            for y in (keys[b], vals[b]):
                c, s, m = ref.quantise(y.transpose(0, 1))
                rows.append((c.double(), s.double().repeat_interleave(64, -1), m.double().repeat_interleave(64, -1)))
            want_q = ref.rotated(x[at:at + n[b], :hq], cs_cpu, pos[None])
            assert same_bits(q[at:at + n[b]], want_q)
            want, tol = ref.attention(rows, want_q, d ** -0.5, pos)
            within(out[at:at + n[b]], want, tol)
            at += n[b]
        return sl, st

    step(lens, lens)
    kept = 0
    for r in range(6):
        n = [most + 1, 1 + r % 3, most + 1]
        lens = [a + b for a, b in zip(lens, n)]
        sl, st = step(n, lens)
        tokens, p, q, u, st_cpu = verify_case(n, V, torch.float32, 30 + r)
        out, acc, new, _ = run_verify(pkv, tokens, p, q, u, st_cpu, torch.tensor(lens, dtype=torch.int32))
        check_verify((out, acc, new, torch.tensor(lens)), tokens, p, q, u, st_cpu)
        lens = new.tolist()
        kept += int(acc.sum())
    assert kept > 0
