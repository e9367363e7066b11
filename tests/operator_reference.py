"""64-bit references of the operators around the paged decode attention
(attention weights, token selection, eviction, self-scaling append,
differential attention), and small seeded pools to run them on.  Everything
here is plain torch on the CPU; the GPU tests copy its inputs to the device."""
import math

import torch

CODE_MAX = {"int8": 127.0, "fp8": 448.0}
DTYPES = {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.float8_e4m3fn}
FLUSHED = 2.0 ** -126                   # a weight below this may be stored as 0


def f64(x):
    return x.to(torch.float32).double() if x.dtype == torch.float8_e4m3fn else x.double()


def raw(x):
    """A pool as indexable bytes when it is E4M3 (a view), else as it is."""
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def take(x, *index):
    """x[index] for pools of any type."""
    return raw(x)[index].contiguous().view(x.dtype)


def code_of(x, scale, dtype):
    """The stored codes of 64-bit x under fp32 scales (broadcast): the nearest
    to the fp32 quotient, ties to even; scale 0 reads as 1."""
    s = torch.where(scale == 0, torch.ones_like(scale), scale).double()
    y = (x / s).float()                       # one rounding: a 64-bit quotient of fp32 numbers
    if dtype == "int8":
        y = torch.where(torch.isnan(y), torch.zeros_like(y), y)
        return y.double().round().clamp(-127, 127).to(torch.int8)
    c = y.clamp(-448, 448).to(torch.float8_e4m3fn)
    nan = torch.full_like(c.view(torch.uint8), 0x7F)
    return torch.where(torch.isnan(y), nan, raw(c)).view(torch.float8_e4m3fn)


def finite_amax(x, dims):
    a = x.abs()
    return torch.where(torch.isfinite(a), a, torch.zeros_like(a)).amax(dim=dims)


class Pool:
    """K and V pools with random rows where the tables point and poison (NaN
    patterns, 127) everywhere else."""

    def __init__(self, L, heads, dim, block, dtype, seed=0, extra=3, width=None, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.g, self.L, self.heads, self.dim, self.block, self.dtype = g, list(L), heads, dim, block, dtype
        nb = [(max(n, 0) + block - 1) // block for n in L]
        self.width = width or max(max(nb), 1)
        self.num_blocks = sum(nb) + extra
        perm = torch.randperm(self.num_blocks, generator=g).to(torch.int32)
        self.tables = torch.full((len(L), self.width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(nb):
            self.tables[b, :n] = perm[at:at + n]
            at += n
        self.free = perm[at:].clone()
        self.seq_lens = torch.tensor(L, dtype=torch.int32)
        self.k_scale = self.v_scale = None
        shape = (self.num_blocks, block, heads, dim)
        self.k, self.v = (self._poison(shape) for _ in range(2))
        for x in (self.k, self.v):
            for b, n in enumerate(L):
                for t in range(max(n, 0)):
                    raw(x)[self.tables[b, t // block].item(), t % block] = raw(self._rows((heads, dim), spread))
        if dtype != "bf16":
            unit = 1 / 32 if dtype == "int8" else 1 / 112
            self.k_scale, self.v_scale = ((torch.rand((self.num_blocks, heads), generator=g) + 0.5) * unit
                                          for _ in range(2))

    def _poison(self, shape):
        if self.dtype == "int8":
            return torch.full(shape, 127, dtype=torch.int8)
        if self.dtype == "fp8":
            return torch.full(shape, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn)
        return torch.full(shape, float("nan"), dtype=torch.bfloat16)

    def _rows(self, shape, spread):
        x = torch.randn(shape, generator=self.g) * spread
        if self.dtype == "bf16":
            return x.to(torch.bfloat16)
        if self.dtype == "int8":
            return (x * 32).round().clamp(-127, 127).to(torch.int8)
        return (x * 112).clamp(-448, 448).to(torch.float8_e4m3fn)

    def randn(self, *shape, scale=1.0):
        return (torch.randn(shape, generator=self.g) * scale).to(torch.bfloat16)

    def rows(self, name, b, head, L=None):
        """Sequence b's values of one pool head, [L, dim] in 64 bits."""
        L = self.L[b] if L is None else L
        ids = self.tables[b, :(L + self.block - 1) // self.block].long()
        cache = self.k if name == "k" else self.v
        x = f64(take(cache, ids, slice(None), head))
        scale = self.k_scale if name == "k" else self.v_scale
        if scale is not None:
            x = x * scale[ids, head].double()[:, None, None]
        return x.reshape(-1, self.dim)[:L]

    def on(self, dev="cuda"):
        """(k_cache, v_cache, dict of scales, tables, seq_lens) on a device."""
        move = lambda x: None if x is None else x.to(dev)  # noqa: E731
        return (move(self.k), move(self.v), dict(k_scale=move(self.k_scale), v_scale=move(self.v_scale)),
                move(self.tables), move(self.seq_lens))


def softmax_bound(q, K, scale):
    """Softmax rows of q K^T in 64 bits and a bound on the relative error of
    every weight computed from fp32 scores: a score of d products accumulated
    in fp32 (truncation allowed: a whole unit 2^-23 per addition) is off by at
    most d 2^-23 sum |q k| |scale| (scaling by s makes s e of an error e, of size
    |s| |e|: under a negative scale the bound is no negative number), a weight
    by twice the largest of its row's (its own score and the denominator's),
    plus a few units of exp2, the division and the sums."""
    S = q @ K.T * scale
    off = q.shape[-1] * 2.0 ** -23 * (q.abs() @ K.abs().T * abs(scale)).amax(dim=-1, keepdim=True)
    off = off + S.abs().amax(dim=-1, keepdim=True) * 2.0 ** -22     # the base-2 scaling
    return torch.softmax(S, dim=-1), torch.expm1(2 * off) + 2.0 ** -19


def decode_weights(pool, q, weights, scale):
    """(out, bound of out, weights, bound of weights) of one decode step."""
    B, hq, d = q.shape
    H = pool.heads
    G = hq // H
    out, tol = torch.zeros(B, hq, d, dtype=torch.float64), torch.zeros(B, hq, d, dtype=torch.float64)
    w, wtol = weights.double().clone(), torch.zeros_like(weights, dtype=torch.float64)
    for b in range(B):
        L = pool.L[b]
        for h in range(H):
            K, V = pool.rows("k", b, h), pool.rows("v", b, h)
            p, rel = softmax_bound(q[b, h * G:(h + 1) * G].double(), K, scale)
            o = p @ V
            out[b, h * G:(h + 1) * G] = o
            # p enters the second product as bf16 (fp16 on 8-bit pools), the
            # result is bf16: half a step each
            tol[b, h * G:(h + 1) * G] = 2.0 ** -8 * o.abs() + (2.0 ** -8 + rel) * 1.01 * (p @ V.abs())
            w[b, h, L - 1] = 0
            w[b, h, :L] += p.sum(dim=0)
            wtol[b, h, :L] = (p * rel).sum(dim=0) + 2.0 ** -22 * w[b, h, :L].abs() + G * FLUSHED
    return out, tol, w, wtol


def prompt_weights(pool, q, counts, weights, scale, accumulate=True):
    H = pool.heads
    G = q.shape[1] // H
    w, wtol = weights.double().clone(), torch.zeros_like(weights, dtype=torch.float64)
    at = 0
    for b, n in enumerate(counts):
        L = pool.L[b]
        for h in range(H):
            if n == 0:
                continue
            K = pool.rows("k", b, h)
            acc, off = torch.zeros(L, dtype=torch.float64), torch.zeros(L, dtype=torch.float64)
            for i in range(n):
                end = L - n + i + 1
                p, rel = softmax_bound(q[at + i, h * G:(h + 1) * G].double(), K[:end], scale)
                acc[:end] += p.sum(dim=0)
                off[:end] += (p * rel).sum(dim=0)
            w[b, h, (L - n if accumulate else 0):L] = 0
            w[b, h, :L] += acc
            # sums of n G weights in fp32, each flushed to 0 below fp32's
            # smallest normal number, 2^-126
            wtol[b, h, :L] = off + (n * G * 2.0 ** -24 + 2.0 ** -22) * w[b, h, :L].abs() + n * G * FLUSHED
        at += n
    return w, wtol


def diff_attention(pool, q, scale, lam, norm_weight, eps, p_off=2.0 ** -8):
    """(out, bound of out); p_off bounds the relative error with which a
    softmax weight enters the product with V."""
    B, rows, d = q.shape
    H, Hkv = rows // 2, pool.heads // 2
    G = H // Hkv
    out, tol = (torch.zeros(B, H, 2 * d, dtype=torch.float64) for _ in range(2))
    for b in range(B):
        for h in range(H):
            j = h // G
            V = torch.cat([pool.rows("v", b, 2 * j), pool.rows("v", b, 2 * j + 1)], dim=1)
            a, e = [], []
            for m in (0, 1):
                p, rel = softmax_bound(q[b, 2 * h + m:2 * h + m + 1].double(), pool.rows("k", b, 2 * j + m), scale)
                a.append((p @ V)[0])
                e.append(((p_off + rel) * 1.01 * (p @ V.abs()))[0])
            y = a[0] - lam[h].double() * a[1]
            off = e[0] + lam[h].double().abs() * e[1] + 2.0 ** -22 * (a[0].abs() + a[1].abs())
            if norm_weight is not None:
                # the norm moves by at most the norm of the errors
                size = torch.sqrt((y ** 2).mean() + eps)
                moved = torch.sqrt((off ** 2).mean()) / size
                assert moved < 0.5, "a case whose difference cancels says nothing"
                y, off = y / size * norm_weight.double(), (off / size + y.abs() / size * moved) / (1 - moved) * norm_weight.double().abs()
            out[b, h] = y
            tol[b, h] = off * 1.01 + 2.0 ** -8 * (y.abs() + off)
    return out, tol


def select(weights, L, budget, recent):
    """(keep_idx, keep_len) by a stable sort."""
    B, H, _ = weights.shape
    idx = torch.full((B, H, budget), -1, dtype=torch.int32)
    for b in range(B):
        n = L[b]
        for h in range(H):
            if n <= budget:
                keep = torch.arange(n)
            else:
                w = weights[b, h, :n - recent].double()
                w = torch.where(torch.isnan(w), torch.full_like(w, -math.inf), w)
                heavy = torch.sort(-w, stable=True).indices[:budget - recent]
                keep = torch.cat([heavy, torch.arange(n - recent, n)]).sort().values
            idx[b, h, :len(keep)] = keep.to(torch.int32)
    return idx, torch.tensor([min(n, budget) for n in L], dtype=torch.int32)


def evict(pool, keep_idx, keep_len, dst_tables, weights):
    """The pools, scales and weights after packing: clones of the pool's."""
    bs, dtype = pool.block, pool.dtype
    k, v = pool.k.clone(), pool.v.clone()
    ks = None if pool.k_scale is None else pool.k_scale.clone()
    vs = None if pool.v_scale is None else pool.v_scale.clone()
    w = weights.clone()
    for b in range(len(pool.L)):
        m = int(keep_len[b])
        for h in range(pool.heads):
            idx = keep_idx[b, h, :m].long()
            w[b, h, :m] = weights[b, h, idx]
            for cache, new, scale, nscale in ((pool.k, k, pool.k_scale, ks), (pool.v, v, pool.v_scale, vs)):
                for j in range(0, m, bs):
                    src = idx[j:j + bs]
                    dst, sb = int(dst_tables[b, j // bs]), pool.tables[b, src // bs].long()
                    still = bool((src == torch.arange(j, j + len(src))).all()) and dst == int(pool.tables[b, j // bs])
                    if still:
                        continue
                    rows = take(cache, sb, src % bs, h)
                    if dtype != "bf16":
                        x = (f64(rows) * scale[sb, h].double()[:, None]).float().double()
                        s = (finite_amax(x, (0, 1)) / CODE_MAX[dtype]).float()
                        rows = code_of(x, s, dtype)
                        nscale[dst, h] = s
                    raw(new)[dst, :len(src), h] = raw(rows)
    return k, v, ks, vs, w


def append(pool, new_k, new_v, counts):
    """The pools and scales after appending each sequence's last counts[b]
    tokens: clones of the pool's."""
    bs, dtype = pool.block, pool.dtype
    out = []
    for name, x in (("k", new_k), ("v", new_v)):
        cache = (pool.k if name == "k" else pool.v).clone()
        scale = (pool.k_scale if name == "k" else pool.v_scale).clone()
        at = 0
        for b, n in enumerate(counts):
            L = pool.L[b]
            first = L - n
            for j in range(first // bs, (L + bs - 1) // bs) if n else ():
                p = int(pool.tables[b, j])
                r0, r1 = max(first - j * bs, 0), min(L - j * bs, bs)
                rows = x[at + j * bs + r0 - first:at + j * bs + r1 - first].double()
                old = scale[p].clone()
                s = (finite_amax(rows, (0, 2)) / CODE_MAX[dtype]).float()
                if r0 > 0:
                    s = torch.maximum(s, old)
                    keep = take(cache, p, slice(0, r0))
                    was = (f64(keep) * old.double()[:, None]).float().double()
                    again = code_of(was, s[:, None], dtype)
                    grown = (s > old)[:, None].expand(keep.shape)
                    raw(cache)[p, :r0] = torch.where(grown, raw(again), raw(keep))
                raw(cache)[p, r0:r1] = raw(code_of(rows, s[:, None], dtype))
                scale[p] = s
            at += n
        out += [cache, scale]
    return out
