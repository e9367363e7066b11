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
