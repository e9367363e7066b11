"""Refusals of the rotated append at sizes past its counts, without a GPU (nothing
is launched)."""
import pytest

from test_q4_host import ROTARY, ROTARY_Q4, pkv  # noqa: F401


@pytest.mark.parametrize("name,base", [("pagedkv_append_rotary", ROTARY), ("pagedkv_append_rotary_q4", ROTARY_Q4)])
@pytest.mark.parametrize("change", [
    dict(num_q_heads=(1 << 31) - 8, q_stride=1 << 38, q_out_stride=1 << 38),
    dict(num_kv_heads=1 << 30, k_stride=1 << 37, v_stride=1 << 37),
    dict(q=None, q_out=None, num_q_heads=(1 << 31) - 1, num_kv_heads=1 << 30, k_stride=1 << 37, v_stride=1 << 37)])
def test_heads_are_counted_in_32_bits(pkv, name, base, change):
    """A token's rows (heads of q, k and v) are numbered in 32 bits: more are refused."""
    assert getattr(pkv.load(), name)(*dict(base, **change).values()) == pkv.KV_ERR_INVALID_ARG
    assert "heads" in pkv.load().pagedkv_last_error().decode()
