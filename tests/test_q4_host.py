"""The host side of the rotated append, the 4-bit pool and draft verification,
without a GPU: argument refusals (nothing is launched), sizes, and the
reference's own consistency."""
import ctypes

import pytest
import torch

import q4_reference as ref

P16 = ctypes.c_void_p(0x1000)                    # aligned, never dereferenced
P32 = ctypes.c_void_p(0x2000)
ODD = ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_97_gb300 as pkv
    from paged_kv_cache_97_gb300 import _build
    _build.build()
    pkv.load()
    return pkv


def sections(*x):
    return (ctypes.c_int32 * len(x))(*x)


ROTARY = dict(q_out=P16, q_out_stride=512, q=P16, q_stride=512, k=P16, k_stride=128, v=P16, v_stride=128, k_cache=P16,
              v_cache=P16, k_scale=None, v_scale=None, cos_sin=P16, max_position=100, rotary_dim=64, interleaved=0,
              positions=None, num_axes=1, axis_sections=None, block_tables=P16, max_blocks=4, seq_lens=P16,
              query_start=P16, batch=2, num_tokens=6, max_query_len=4, num_q_heads=8, num_kv_heads=2, head_dim=64,
              num_blocks=64, block_size=16, dtype=0, stream=None)
ROTARY_Q4 = {("kv_cache" if k == "k_cache" else k): v for k, v in ROTARY.items()
             if k not in ("v_cache", "k_scale", "v_scale", "dtype")}
READ = dict(k_out=P16, v_out=P16, kv_cache=P16, block_tables=P16, max_blocks=4, seq_lens=P16, query_start=P16, batch=2,
            num_tokens=6, max_query_len=4, num_kv_heads=2, head_dim=64, num_blocks=64, block_size=16, stream=None)
COPY = dict(kv_cache=P16, block_pairs=P16, num_pairs=2, num_blocks=8, block_size=16, num_kv_heads=2, head_dim=64,
            stream=None)
DECODE = dict(out=P16, q=P16, kv_cache=P16, block_tables=P16, max_blocks=64, seq_lens=P16, batch=2, num_q_heads=8,
              num_kv_heads=2, head_dim=64, num_blocks=64, block_size=16, max_seq_len=1000, scale=0.1, workspace=None,
              workspace_bytes=0, stream=None)
MULTI = dict(out=P16, q=P16, kv_cache=P16, block_tables=P16, max_blocks=64, seq_lens=P16, query_start=P16, batch=2,
             num_tokens=6, max_query_len=4, num_q_heads=8, num_kv_heads=2, head_dim=64, num_blocks=64, block_size=16,
             max_seq_len=1000, scale=0.1, workspace=None, workspace_bytes=0, stream=None)
VERIFY = dict(out_tokens=P16, num_accepted=P16, tokens=P32, target=P16, draft=P16, uniform=P16, query_start=P16,
              seq_lens=P16, new_lens=P16, batch=2, num_tokens=6, max_query_len=4, vocab=100, dtype=0, stream=None)

GEOMETRY = [dict(head_dim=96), dict(block_size=8), dict(num_kv_heads=0), dict(num_blocks=0), dict(batch=-1),
            dict(max_blocks=0), dict(block_tables=None), dict(seq_lens=None), dict(num_tokens=-1),
            dict(max_query_len=0)]
TURN = GEOMETRY + [
    dict(q=None), dict(q_out=None), dict(num_q_heads=0), dict(rotary_dim=24), dict(rotary_dim=0), dict(rotary_dim=80),
    dict(max_position=0), dict(num_axes=0), dict(num_axes=5), dict(num_axes=2), dict(num_axes=2, positions=P16),
    dict(num_axes=2, positions=P16, axis_sections=sections(16, 15)),
    dict(num_axes=2, positions=P16, axis_sections=sections(40, -8)), dict(axis_sections=sections(31)), dict(k=None),
    dict(v=None), dict(query_start=None), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(q_out=ODD), dict(cos_sin=ODD),
    dict(q_stride=511), dict(q_stride=504), dict(k_stride=120), dict(v_stride=132), dict(q_out_stride=0),
    dict(q_stride=520)]
REFUSED = (
    [("pagedkv_append_rotary", ROTARY, c) for c in TURN + [
        dict(dtype=3), dict(k_cache=None), dict(v_cache=None), dict(k_cache=ODD), dict(v_cache=ODD), dict(k_scale=P16),
        dict(dtype=1), dict(dtype=2, k_scale=P16)]] +
    [("pagedkv_append_rotary_q4", ROTARY_Q4, c) for c in TURN + [dict(kv_cache=None), dict(kv_cache=ODD)]] +
    [("pagedkv_read_q4", READ, c) for c in GEOMETRY + [
        dict(k_out=None), dict(v_out=None), dict(kv_cache=None), dict(k_out=ODD), dict(kv_cache=ODD),
        dict(query_start=None)]] +
    [("pagedkv_copy_blocks_q4", COPY, c) for c in [
        dict(kv_cache=None), dict(kv_cache=ODD), dict(block_pairs=None), dict(num_pairs=-1), dict(num_pairs=65536),
        dict(num_blocks=0), dict(block_size=8), dict(num_kv_heads=0), dict(head_dim=96)]] +
    [("paged_attention_decode_q4", DECODE, c) for c in [g for g in GEOMETRY if not {"num_tokens", "max_query_len"} & set(g)] + [
        dict(out=None), dict(q=None), dict(kv_cache=None), dict(out=ODD), dict(q=ODD), dict(kv_cache=ODD),
        dict(num_q_heads=7), dict(num_q_heads=18), dict(max_seq_len=0),
        dict(num_q_heads=65536, num_kv_heads=65536)]] +
    [("paged_attention_multi_q4", MULTI, c) for c in GEOMETRY + [
        dict(out=None), dict(q=None), dict(kv_cache=None), dict(out=ODD), dict(q=ODD), dict(kv_cache=ODD),
        dict(num_q_heads=7), dict(num_q_heads=18), dict(max_seq_len=0), dict(query_start=None),
        dict(num_q_heads=65536, num_kv_heads=65536)]] +
    [("pagedkv_verify_drafts", VERIFY, c) for c in [
        dict(batch=-1), dict(num_tokens=-1), dict(max_query_len=0), dict(vocab=0), dict(vocab=1 << 19), dict(dtype=3),
        dict(dtype=-1), dict(out_tokens=None), dict(num_accepted=None), dict(tokens=None), dict(target=None),
        dict(uniform=None), dict(query_start=None), dict(seq_lens=None), dict(new_lens=None), dict(num_tokens=1),
        dict(target=ctypes.c_void_p(0x1002)), dict(draft=ctypes.c_void_p(0x1001), dtype=1), dict(tokens=P16)]])


@pytest.mark.parametrize("i", range(len(REFUSED)), ids=lambda i: f"{REFUSED[i][0]}-{'-'.join(REFUSED[i][2])}-{i}")
def test_refused(pkv, i):
    name, base, change = REFUSED[i]
    args = dict(base, **change)
    assert set(args) == set(base)
    assert getattr(pkv.load(), name)(*args.values()) == pkv.KV_ERR_INVALID_ARG
    assert name in pkv.load().pagedkv_last_error().decode()


@pytest.mark.parametrize("name,base", [("pagedkv_append_rotary", ROTARY), ("pagedkv_append_rotary_q4", ROTARY_Q4),
                                       ("pagedkv_read_q4", READ), ("paged_attention_decode_q4", DECODE),
                                       ("paged_attention_multi_q4", MULTI), ("pagedkv_verify_drafts", VERIFY)])
def test_empty_batch_is_a_no_op(pkv, name, base):
    args = dict(base, batch=0)
    if "num_tokens" in args:
        args["num_tokens"] = 0
    assert getattr(pkv.load(), name)(*args.values()) == pkv.KV_OK
    assert pkv.load().pagedkv_copy_blocks_q4(*dict(COPY, num_pairs=0).values()) == pkv.KV_OK


def test_packed_calls(pkv):
    """pagedkv_call passes on what the calls themselves get, and counts arguments."""
    import struct
    lib = pkv.load()
    for which, (name, base) in enumerate([("pagedkv_append_rotary", ROTARY), ("pagedkv_append_rotary_q4", ROTARY_Q4),
                                          ("pagedkv_read_q4", READ), ("paged_attention_decode_q4", DECODE),
                                          ("paged_attention_multi_q4", MULTI), ("pagedkv_verify_drafts", VERIFY)]):
        assert pkv._COUNTS[which] == len(base)

        def packed(**change):
            xs = [getattr(x, "value", x) or 0 for x in dict(base, **change).values()]
            return struct.pack(f"{len(xs)}q", *[struct.unpack("I", struct.pack("f", x))[0] if isinstance(x, float) else x
                                                for x in xs])
        empty = dict(batch=0, **({"num_tokens": 0} if "num_tokens" in base else {}))
        assert lib.pagedkv_call(which, packed(**empty), len(base)) == pkv.KV_OK
        assert lib.pagedkv_call(which, packed(batch=-1), len(base)) == pkv.KV_ERR_INVALID_ARG
        assert name in lib.pagedkv_last_error().decode()
        assert lib.pagedkv_call(which, packed(), len(base) - 1) == pkv.KV_ERR_INVALID_ARG
    assert lib.pagedkv_call(6, packed(), 15) == pkv.KV_ERR_INVALID_ARG
    assert lib.pagedkv_call(0, None, 33) == pkv.KV_ERR_INVALID_ARG


def test_sizes(pkv):
    for bs in (16, 32):
        for d in (64, 128):
            assert pkv.q4_record_bytes(bs, d) == ref.record_bytes(bs, d) == bs * 2 * (d // 2 + d // 64 * 4)
            assert pkv.q4_record_bytes(bs, d) % 16 == 0
    assert pkv.q4_record_bytes(8, 64) == 0 and pkv.q4_record_bytes(16, 96) == 0
    assert pkv.q4_workspace_bytes(8, 3, 64) == 0
    sizes = [pkv.q4_workspace_bytes(32, 8, 128, n) for n in (1, 2, 3, 8, 4000)]
    assert sizes[0] == sizes[1] and all(0 < x < 64 << 20 for x in sizes)


def test_reference_packs_what_it_unpacks():
    g = torch.Generator().manual_seed(1)
    for block, d in ((16, 64), (32, 128)):
        codes = torch.randint(0, 16, (2, 3, block, d), generator=g)
        scale, low = (torch.randn((2, 3, block, d // 64), generator=g).to(torch.bfloat16).float() for _ in "ab")
        rec = ref.pack(codes, scale, low, block, d)
        assert rec.shape == (3, ref.record_bytes(block, d))
        for i, (c, s, m) in enumerate(ref.unpack(rec, block, d)):
            assert torch.equal(c, codes[i]) and torch.equal(s, scale[i].double()) and torch.equal(m, low[i].double())


def test_half_a_scale_at_most():
    """The definition's own bound on random rows: half a scale, and the fp32
    steps' 2^-20 of the range."""
    x = torch.randn((400, 128), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    c, s, m = ref.quantise(x)
    value = m.double().repeat_interleave(64, -1) + s.double().repeat_interleave(64, -1) * c
    assert ((value - x.double()).abs() <= s.double().repeat_interleave(64, -1) * (0.5 + 2.0 ** -16)).all()


def test_binding_refuses(pkv):
    bf, i32 = (lambda *s: torch.zeros(s, dtype=torch.bfloat16)), (lambda *s: torch.zeros(s, dtype=torch.int32))
    kv, bt, sl, q = torch.zeros((4, 2, 1152), dtype=torch.uint8), i32(2, 2), i32(2), bf(2, 4, 64)
    cache, rows = bf(4, 16, 2, 64), bf(2, 2, 64)
    probs = torch.zeros((2, 9))
    for call in (lambda: pkv.append_rotary(q, q, rows, rows, cache, cache, torch.zeros((9, 64)), bt, sl),
                 lambda: pkv.append_rotary_q4(q, q, rows, rows, kv, torch.zeros((9, 64)), bt, sl, 16),
                 lambda: pkv.read_q4(rows, rows, kv, bt, sl, 16), lambda: pkv.copy_blocks_q4(kv, i32(1, 2), 16),
                 lambda: pkv.paged_attention_decode_q4(q, q, kv, bt, sl, 16, 32, 1.0),
                 lambda: pkv.paged_attention_multi_q4(q, q, kv, bt, sl, i32(3), 16, 32, 1, 1.0),
                 lambda: pkv.verify_drafts(i32(2), i32(2), i32(2), probs, None, torch.zeros(2), i32(3))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="q4_record_bytes"):
        pkv.read_q4(rows, rows, kv, bt, sl, 32 + 16)
    with pytest.raises(TypeError):
        pkv.paged_attention_decode_q4(q, q, cache, bt, sl, 16, 32, 1.0)
