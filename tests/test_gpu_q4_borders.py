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
