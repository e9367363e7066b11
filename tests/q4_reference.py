"""64-bit references of the rotated append, the 4-bit pool and its attention, and
the verification of drafted tokens.  Plain torch and numpy on the CPU."""
import math

import numpy as np
import torch


def group_word_nibble(d):
    """Byte and nibble of every element of a row's codes."""
    e = torch.arange(d)
    word = e % 64 // 8 * (d // 64) + e // 64
    return word * 4 + e % 8 // 2, e % 2


def record_bytes(block, d):
    return block * d * 9 // 8


def unpack(kv, block, d):
    """(codes, scale, min) of K and of V from records [..., bytes]: int64
    [..., block, d], fp64 [..., block, d / 64] twice."""
    at, nib = group_word_nibble(d)
    out, half, par = [], block * d // 2, block * d // 16
    for i in range(2):
        c = kv[..., i * half:(i + 1) * half].reshape(*kv.shape[:-1], block, d // 2)[..., at].long()
        codes = torch.where(nib == 1, c >> 4, c & 15)
        p = kv[..., block * d + i * par:block * d + (i + 1) * par].contiguous().view(torch.bfloat16)
        p = p.reshape(*kv.shape[:-1], block, d // 64, 2).double()
        out.append((codes, p[..., 0], p[..., 1]))
    return out


def pack(codes, scale, low, block, d):
    """Records of K and V parts: codes [2, ..., block, d], pairs [2, ..., block, d / 64]."""
    at, nib = group_word_nibble(d)
    lead = codes.shape[1:-2]
    parts = []
    for i in range(2):
        b = torch.zeros(*lead, block, d // 2, dtype=torch.uint8)
        lo, hi = codes[i][..., nib == 0], codes[i][..., nib == 1]
        b[..., at[nib == 0]] = (lo + 16 * hi).to(torch.uint8)
        parts.append(b.flatten(-2))
    for i in range(2):
        pair = torch.stack((scale[i], low[i]), dim=-1).to(torch.bfloat16).contiguous()
        parts.append(pair.flatten(-3).view(torch.uint8))
    return torch.cat(parts, dim=-1)


def quantise(x):
    """(codes, scale, min) of bf16 rows [..., d] by the definition, in fp32 steps."""
    x = x.float()
    x = torch.where(torch.isnan(x), torch.zeros_like(x), x).clamp(-2.0 ** 126, 2.0 ** 126) + 0.0
    g = x.unflatten(-1, (-1, 64))
    lo, hi = g.amin(dim=-1), g.amax(dim=-1)
    step = (hi - lo) * torch.full_like(lo, 1 / 15)
    step = ((step.view(torch.int32) + 0xFFFF) & -65536).view(torch.float32).clamp(min=2.0 ** -126)
    inv = torch.ones_like(step) / step
    c = torch.round((g - lo[..., None]) * inv[..., None]).clamp(0, 15)
    return c.flatten(-2).long(), step, lo


def rotated(x, cos_sin, pos, interleaved=False, sections=None):
    """bf16 rows [T, H, d] rotated in fp32 (every product and sum rounded once);
    pos [axes, T]."""
    R = cos_sin.shape[1]
    half = R // 2
    axis = torch.repeat_interleave(torch.arange(pos.shape[0]), torch.tensor(sections or [half]))
    j = torch.arange(half)
    cos = cos_sin[pos[axis].long(), j[:, None]].T[:, None]
    sin = cos_sin[pos[axis].long(), half + j[:, None]].T[:, None]
    first, second = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, half), slice(half, R))
    y = x.clone()
    a, b = x[..., first].float(), x[..., second].float()
    y[..., first] = (a * cos - b * sin).to(torch.bfloat16)
    y[..., second] = (b * cos + a * sin).to(torch.bfloat16)
    return y


def table(positions, rotary_dim, base=10000.0):
    half = rotary_dim // 2
    f = base ** (-torch.arange(half, dtype=torch.float64) / half)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return torch.cat((a.cos(), a.sin()), dim=1).float()


class Pool4:
    """A 4-bit pool with random rows where the tables point and 0xFF (codes 15,
    NaN pairs) everywhere else, rows past a sequence's end among it."""

    def __init__(self, L, heads, dim, block, seed=0, extra=3, width=None, kscale=None, vscale=None, num_blocks=None,
                 low=8.5):
        g = torch.Generator().manual_seed(seed)
        self.g, self.L, self.heads, self.dim, self.block = g, list(L), heads, dim, block
        nb = [(max(n, 0) + block - 1) // block for n in L]
        self.width = width or max(max(nb), 1)
        self.num_blocks = num_blocks or sum(nb) + extra
        perm = torch.randperm(sum(nb) + extra, generator=g).to(torch.int32)
        if num_blocks:                                   # far blocks
            perm = num_blocks - 1 - perm
        self.tables = torch.full((len(L), self.width), -1, dtype=torch.int32)
        self.seq_lens = torch.tensor(L, dtype=torch.int32)
        self.records = {}                                # block id -> [heads, record]
        at = 0
        for b, n in enumerate(nb):
            ids = perm[at:at + n]
            self.tables[b, :n] = ids
            at += n
            codes = torch.randint(0, 16, (2, n, heads, block, dim), generator=g)
            scale = 0.3 * (0.5 + torch.rand((2, n, heads, block, dim // 64), generator=g))
            if kscale is not None:
                scale[0] *= kscale(scale[0].shape, g)
            if vscale is not None:
                scale[1] *= vscale(scale[1].shape, g)
            rec = pack(codes, scale, -scale * (low - torch.rand(scale.shape, generator=g)), block, dim)
            k, v = unpack(rec, block, dim)
            last = int(L[b]) - (n - 1) * block if n else 0
            if n and last < block:
                tail = pack(torch.full((2, heads, block, dim), 15), torch.full((2, heads, block, dim // 64), math.nan),
                            torch.full((2, heads, block, dim // 64), math.nan), block, dim)
                mine = pack(torch.stack((k[0][-1], v[0][-1])), torch.stack((k[1][-1], v[1][-1])).float(),
                            torch.stack((k[2][-1], v[2][-1])).float(), block, dim)
                keep = torch.arange(block) < last
                c, t = unpack(mine, block, dim), unpack(tail, block, dim)
                merged = [[torch.where(keep[:, None], x, y) for x, y in zip(c[i], t[i])] for i in range(2)]
                rec[-1] = pack(torch.stack((merged[0][0], merged[1][0])),
                               torch.stack((merged[0][1], merged[1][1])).float(),
                               torch.stack((merged[0][2], merged[1][2])).float(), block, dim)
            for i, x in enumerate(ids.tolist()):
                self.records[x] = rec[i]

    def randn(self, *shape, scale=1.0):
        return (scale * torch.randn(shape, generator=self.g)).to(torch.bfloat16)

    def on(self, device="cuda"):
        """(kv_cache, tables, seq_lens) on the device."""
        kv = torch.full((self.num_blocks, self.heads, record_bytes(self.block, self.dim)), 0xFF, dtype=torch.uint8,
                        device=device)
        if self.records:
            kv[torch.tensor(list(self.records), device=device).long()] = torch.stack(list(self.records.values())).to(device)
        return kv, self.tables.to(device), self.seq_lens.to(device)

    def rows(self, b, L):
        """Per tensor (K, V) the codes, scales and minima of sequence b's rows, fp64 per element [H, L, d]."""
        n = (L + self.block - 1) // self.block
        rec = torch.stack([self.records[i] for i in self.tables[b, :n].tolist()])
        return rows_of(rec, self.block, self.dim, L)


def rows_of(rec, block, d, L):
    """rec [n, H, bytes] -> for K and V: (codes, scale, min) [H, L, d] in fp64."""
    out = []
    for c, s, m in unpack(rec, block, d):
        part = [x.transpose(0, 1).flatten(1, 2)[:, :L] for x in (c.double(), s, m)]
        part[1], part[2] = (x.repeat_interleave(64, dim=-1) for x in part[1:])
        out.append(part)
    return out


def attention(rows, q, scale, positions, wide=False):
    """Attention of query rows q [n, Hq, d] (bf16) at `positions` [n] over one
    sequence's rows, and how far a kernel may be off.

    Per output element, with w the exact weights: the output's own rounding
    2^-8 |out|; the fp16 rounding of weight * scale, 2^-11 sum w (scale code);
    the scores' fp32 sums, each of 64 products cut by at most 2^-24 of the
    largest partial sum, 2^-18 of S_abs = |scale| sum |q| |K|-terms, doubled for
    the products with scale and min, which moves every weight by at most that
    (natural units) and the normalised sum by twice that times sum w |V|; the
    exponential, 2^-22, likewise; the fp32 sums over tokens, 2^-14 of
    sum w (scale code + |min|) for up to 2^14 steps of 2^-24 each and their ten
    joins; half a step of the smallest fp16 (2^-30 of the largest product, times
    15 for its code) per token.

    ``wide``: keys and values enter the products as fp16 numbers (2^-11 of their
    value), the weight alone as one: 2^-11 of S_abs in the scores, of sum w |V|
    twice in the sum.  A weight is p = w 2^E M, E the exponent that brings the 128 rows'
    largest |V|, top, into [2^12, 2^13) (-80 at least, as if top were 2^-67), and
    the row's largest p is 2^5 at least: half a step of the smallest fp16, 2^-25, is
    2^-30 of it.  Times |V| / 2^E < 2^13, and with 2^E <= top / 2^12, a token is off by at
    most 2^-29 max(w top).  Half a step of a value, 2^-25 2^E <= 2^-37 top, is less."""
    (kc, ks, km), (vc, vs, vm) = rows
    H, L, d = kc.shape
    n, hq, _ = q.shape
    qq = q.double().view(n, H, hq // H, d)
    K, V = km + ks * kc, vm + vs * vc
    S = torch.einsum("nhgd,htd->nhgt", qq, K) * scale
    Sabs = torch.einsum("nhgd,htd->nhgt", qq.abs(), km.abs() + ks * kc) * abs(scale)
    mask = torch.arange(L) > positions[:, None]
    S = S.masked_fill(mask[:, None, None], -math.inf)
    Sabs = Sabs.masked_fill(mask[:, None, None], 0)
    w = torch.softmax(S, dim=-1)
    out = torch.einsum("nhgt,htd->nhgd", w, V)
    mag = torch.einsum("nhgt,htd->nhgd", w, vs * vc + vm.abs())
    part = torch.einsum("nhgt,htd->nhgd", w, vs * vc)
    # a weight's relative error times what it carries, and the sum's own
    shift = (2.0 ** -17 + (2.0 ** -11 if wide else 0)) * Sabs + 2.0 ** -21
    moved = torch.einsum("nhgt,htd->nhgd", w * shift, vs * vc + vm.abs()) + mag * (w * shift).sum(-1, keepdim=True)
    floor = 2.0 ** -30 * 15 * L * (w[..., None] * vs.amax(-1)[None, :, None, :, None]).amax(dim=3)
    tol = 2.0 ** -8 * out.abs() + 2.0 ** -11 * part + moved + 2.0 ** -14 * mag + floor
    if wide:
        top = (vm.abs() + 15 * vs).amax(-1)
        top = torch.cat([x.amax(1, keepdim=True).expand_as(x) for x in top.split(128, dim=1)], 1).clamp(min=2.0 ** -67)
        tol = tol + 2.0 ** -10 * mag + 2.0 ** -29 * L * (w * top[None, :, None]).amax(-1)[..., None]
    return out.reshape(n, hq, d), tol.reshape(n, hq, d)


def verify(tokens, target, draft, u, start, seq_lens=None):
    """Kept drafts and, per sequence, the range of next tokens that sums off by
    half a unit (2^-45) per weight allow."""
    V = target.shape[1]
    res = []
    for b in range(len(start) - 1):
        r, n = int(start[b]), int(start[b + 1] - start[b])
        kept = []
        for i in range(n - 1):
            x = int(tokens[r + i + 1])
            if not 0 <= x < V:
                break
            q = 1.0 if draft is None else float(draft[r - b + i, x])
            if not float(u[r + i]) * q < float(target[r + i, x]):
                break
            kept.append(x)
        if n == 0:
            res.append(([], None))
            continue
        a = len(kept)
        w = target[r + a].float()
        x = int(tokens[r + a + 1]) if a < n - 1 else -1
        if 0 <= x < V:
            if draft is None:
                less = w.clone()
                less[x] = 0
            else:
                less = w - draft[r - b + a].float()
            less = torch.nan_to_num(less, nan=0.0).clamp(0, 1)
            if float(less.sum()) > 0:
                w = less
        w = torch.nan_to_num(w, nan=0.0).clamp(0, 1).double().numpy()
        total = np.cumsum(w)
        if total[-1] == 0:
            res.append((kept, (V - 1, V - 1)))
            continue
        uu = float(u[r + n - 1])
        uu = min(uu, 1 - 2.0 ** -24) if uu >= 0 else 0.0
        off = V * 2.0 ** -45 + 2.0 ** -50
        goal = uu * total[-1]
        lo = int(np.searchsorted(total, goal - off, side="right"))
        hi = min(int(np.searchsorted(total, goal + off, side="right")), V - 1)
        res.append((kept, (lo, hi)))
    return res
