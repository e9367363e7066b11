"""The host side of the operators around the decode attention, without a GPU:
argument refusals (nothing is launched), workspace sizes, and the block pool's
preparation of an eviction."""
import ctypes

import numpy as np
import pytest
import torch

P16 = ctypes.c_void_p(0x1000)                    # aligned, never dereferenced
ODD = ctypes.c_void_p(0x1008)
BIG = 1 << 40


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_97_gb300 as pkv
    from paged_kv_cache_97_gb300 import _build
    _build.build()
    pkv.load()
    return pkv


WEIGHTS = dict(out=P16, weights=P16, weights_stride=200, q=P16, k_cache=P16, v_cache=P16, k_scale=None,
               v_scale=None, block_tables=P16, max_blocks=13, seq_lens=P16, batch=2, num_q_heads=8,
               num_kv_heads=2, head_dim=64, num_blocks=64, block_size=16, max_seq_len=200, scale=0.125,
               dtype=0, workspace=None, workspace_bytes=0, stream=None)
PROMPT = dict(weights=P16, weights_stride=200, q=P16, k_cache=P16, k_scale=None, block_tables=P16,
              max_blocks=13, seq_lens=P16, query_start=P16, batch=2, num_tokens=6, max_query_len=4,
              num_q_heads=8, num_kv_heads=2, head_dim=64, num_blocks=64, block_size=16, max_seq_len=200,
              scale=0.125, accumulate=1, dtype=0, workspace=None, workspace_bytes=0, stream=None)
SELECT = dict(keep_idx=P16, keep_len=P16, weights=P16, weights_stride=200, seq_lens=P16, batch=2,
              num_kv_heads=2, max_seq_len=200, budget=16, recent=4, stream=None)
EVICT = dict(k_cache=P16, v_cache=P16, k_scale=None, v_scale=None, block_tables=P16, max_blocks=13,
             dst_block_tables=P16, dst_max_blocks=13, seq_lens=P16, keep_idx=P16, keep_len=P16, budget=16,
             weights=P16, weights_stride=200, batch=2, num_blocks=64, block_size=16, num_kv_heads=2,
             head_dim=64, dtype=0, stream=None)
APPEND = dict(new_k=P16, new_v=P16, k_cache=P16, v_cache=P16, k_scale=P16, v_scale=P16, block_tables=P16,
              max_blocks=13, seq_lens=P16, query_start=P16, batch=2, num_tokens=6, max_query_len=4,
              num_blocks=64, block_size=16, num_kv_heads=2, head_dim=64, dtype=1, stream=None)
DIFF = dict(out=P16, q=P16, k_cache=P16, v_cache=P16, k_scale=None, v_scale=None, block_tables=P16,
            max_blocks=13, seq_lens=P16, batch=2, num_heads=4, num_kv_heads=2, head_dim=64, num_blocks=64,
            block_size=16, max_seq_len=200, scale=0.125, lam=P16, norm_weight=P16, eps=1e-5, dtype=0,
            workspace=None, workspace_bytes=0, stream=None)

GEOMETRY = [dict(head_dim=96), dict(block_size=8), dict(num_kv_heads=0), dict(num_blocks=0), dict(batch=-1),
            dict(dtype=3), dict(batch=65536), dict(max_blocks=0), dict(block_tables=None),
            dict(seq_lens=None), dict(k_cache=None), dict(k_cache=ODD)]

REFUSED = (
    [("paged_attention_decode_weights", WEIGHTS, c) for c in GEOMETRY + [
        dict(out=None), dict(weights=None), dict(q=None), dict(q=ODD), dict(v_cache=ODD), dict(out=ODD),
        dict(num_q_heads=7), dict(num_q_heads=18), dict(weights_stride=199), dict(weights_stride=0),
        dict(max_seq_len=0), dict(k_scale=P16), dict(dtype=1), dict(dtype=2, k_scale=P16)]] +
    [("pagedkv_attention_weights", PROMPT, c) for c in GEOMETRY + [
        dict(weights=None), dict(q=None), dict(q=ODD), dict(query_start=None), dict(num_q_heads=7),
        dict(weights_stride=199), dict(max_query_len=0), dict(num_tokens=-1), dict(k_scale=P16),
        dict(dtype=1), dict(max_seq_len=1 << 30, weights_stride=1 << 30),
        dict(max_query_len=1 << 30, num_tokens=1 << 30)]] +
    [("pagedkv_select_tokens", SELECT, c) for c in [
        dict(keep_idx=None), dict(keep_len=None), dict(weights=None), dict(seq_lens=None), dict(batch=-1),
        dict(num_kv_heads=0), dict(max_seq_len=201), dict(max_seq_len=0), dict(weights_stride=0),
        dict(budget=0), dict(recent=-1), dict(recent=17), dict(batch=1 << 30, num_kv_heads=1 << 10)]] +
    [("pagedkv_evict_tokens", EVICT, c) for c in GEOMETRY + [
        dict(v_cache=None), dict(v_cache=ODD), dict(dst_block_tables=None), dict(dst_max_blocks=0),
        dict(keep_idx=None), dict(keep_len=None), dict(budget=0), dict(weights_stride=0),
        dict(k_scale=P16), dict(dtype=1), dict(dtype=2, v_scale=P16)]] +
    [("pagedkv_append_scaled", APPEND, c) for c in [g for g in GEOMETRY if g != dict(batch=65536)] + [
        dict(dtype=0), dict(new_k=None), dict(new_v=None), dict(new_k=ODD), dict(v_cache=ODD),
        dict(k_scale=None), dict(v_scale=None), dict(max_query_len=0), dict(num_tokens=-1),
        dict(query_start=None), dict(batch=1 << 30, num_kv_heads=1 << 10)]] +
    [("paged_diff_attention_decode", DIFF, c) for c in GEOMETRY + [
        dict(out=None), dict(q=None), dict(lam=None), dict(q=ODD), dict(out=ODD), dict(v_cache=ODD),
        dict(num_heads=5), dict(num_heads=0), dict(max_seq_len=0), dict(eps=-1.0), dict(eps=float("nan")),
        dict(k_scale=P16), dict(dtype=1)]])


@pytest.mark.parametrize("name,base,change", REFUSED,
                         ids=[f"{n}-{'-'.join(f'{k}={getattr(v, 'value', v)}' for k, v in c.items())}" for n, _, c in REFUSED])
def test_refused(pkv, name, base, change):
    args = dict(base, **change)
    assert set(args) == set(base)
    st = getattr(pkv.load(), name)(*args.values())
    assert st == pkv.KV_ERR_INVALID_ARG
    assert name in pkv.load().pagedkv_last_error().decode()


@pytest.mark.parametrize("name,base", [("paged_attention_decode_weights", WEIGHTS),
                                       ("pagedkv_attention_weights", PROMPT), ("pagedkv_select_tokens", SELECT),
                                       ("pagedkv_evict_tokens", EVICT), ("pagedkv_append_scaled", APPEND),
                                       ("paged_diff_attention_decode", DIFF)])
def test_empty_batch_is_a_no_op(pkv, name, base):
    args = dict(base, batch=0)
    if "num_tokens" in args:
        args["num_tokens"] = 0
    assert getattr(pkv.load(), name)(*args.values()) == pkv.KV_OK


def test_binding_refuses_host_tensors(pkv):
    bf, i32, f32 = (lambda *s: torch.zeros(s, dtype=torch.bfloat16)), (lambda *s: torch.zeros(s, dtype=torch.int32)), torch.zeros
    cache, bt, sl = bf(4, 16, 2, 64), i32(2, 2), i32(2)
    for call in (lambda: pkv.paged_attention_decode_weights(bf(2, 4, 64), f32(2, 2, 32), bf(2, 4, 64), cache, cache, bt, sl, 32, 1.0, None),
                 lambda: pkv.attention_weights(f32(2, 2, 32), bf(3, 4, 64), cache, bt, sl, i32(3), 32, 2, 1.0, None),
                 lambda: pkv.select_tokens(i32(2, 2, 8), sl, f32(2, 2, 32), sl, 32, 1),
                 lambda: pkv.evict_tokens(cache, cache, bt, sl, i32(2, 2, 8), sl),
                 lambda: pkv.append_scaled(bf(2, 2, 64), bf(2, 2, 64), cache, cache, None, None, bt, sl),
                 lambda: pkv.paged_diff_attention_decode(bf(2, 2, 128), bf(2, 4, 64), cache, cache, bt, sl, 32, 1.0, f32(2))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_workspace_sizes(pkv):
    # decode weights: the scores of every row, (m, l), and partials when a
    # sequence may have several
    one = pkv.weights_workspace_bytes(2, 8, 64, 256, 16)
    assert one >= 2 * 8 * (256 + 2) * 4
    assert pkv.weights_workspace_bytes(2, 8, 64, 257, 16) >= 2 * 8 * (257 + 2 * 2 + 2 * 64) * 4
    assert pkv.attention_weights_workspace_bytes(10, 8, 256) == 10 * 8 * 2 * 4
    assert pkv.attention_weights_workspace_bytes(10, 8, 257) == 10 * 8 * 2 * 2 * 4
    assert pkv.diff_workspace_bytes(2, 4, 64, 256, 16) == 0
    assert pkv.diff_workspace_bytes(2, 4, 64, 257, 16) == 2 * 8 * 2 * (2 + 128) * 4
    for f, args in ((pkv.weights_workspace_bytes, (2, 8, 64, 256, 16)), (pkv.diff_workspace_bytes, (2, 4, 64, 300, 16))):
        for i in range(4):
            bad = list(args)
            bad[i] = 0
            assert f(*bad) == 0
    assert pkv.attention_weights_workspace_bytes(0, 8, 256) == 0


# --------------------------------------------------------------------------
# kv_pool_prepare_evict
# --------------------------------------------------------------------------

def table(rows, width):
    t = np.full((len(rows), width), -1, np.int32)
    for b, r in enumerate(rows):
        t[b, :len(r)] = r
    return t


def test_prepare_evict_in_place(pkv):
    pool = pkv.KVPool(10, 16, 2, 64)
    a, b = pool.alloc(4), pool.alloc(3)
    bt = table([a, b], 5)
    dst = pool.prepare_evict(bt, [60, 40], [20, 40])
    assert dst.tolist() == [a[:2] + [-1] * 3, b + [-1] * 2]   # the second keeps everything
    assert [pool.refcount(i) for i in a] == [1, 1, 0, 0] and [pool.refcount(i) for i in b] == [1] * 3
    assert pool.stats() == (5, 5)
    assert pool.alloc(5)[-2:] == a[2:]                        # released in table order
    assert bt.tolist() == table([a, b], 5).tolist()


def test_prepare_evict_shared_blocks(pkv):
    """A fork's blocks are replaced, whoever of the sharers is evicted; a
    replacement is never a block that the call releases."""
    pool = pkv.KVPool(12, 16, 2, 64)
    a = pool.alloc(4)
    pool.fork(a[:3])
    last = pool.alloc(1)
    bt = table([a, a[:3] + last], 4)
    dst = pool.prepare_evict(bt, [64, 64], [33, 17])
    assert dst.tolist() == [[5, 6, 7, -1], [8, 9, -1, -1]]
    assert all(pool.refcount(i) == 0 for i in a + last)
    assert pool.stats() == (5, 7)
    # one of two sharers: the other's blocks stay as they are
    pool = pkv.KVPool(8, 16, 2, 64)
    a = pool.alloc(3)
    pool.fork(a)
    dst = pool.prepare_evict(table([a], 3), [48], [32])
    assert dst.tolist() == [[3, 4, -1]] and [pool.refcount(i) for i in a] == [1, 1, 1]


def test_prepare_evict_is_all_or_nothing(pkv):
    pool = pkv.KVPool(5, 16, 2, 64)
    a = pool.alloc(3)
    pool.fork(a)
    own = pool.alloc(1)
    bt = table([a, a, own], 3)
    before = [pool.refcount(i) for i in range(5)], pool.stats()
    with pytest.raises(pkv.KVError) as e:
        pool.prepare_evict(bt, [48, 48, 16], [16, 20, 5])     # 1 + 2 blocks, 1 free
    assert e.value.status == pkv.KV_ERR_OUT_OF_BLOCKS
    for lens, keep, t in (([48, 48, 17], [16, 16, 5], bt),    # entry -1
                          ([48, 48, 16], [16, 16, 17], bt),   # keeps more than there is
                          ([48, 48, 16], [16, -1, 5], bt), ([49, 48, 16], [16, 16, 5], bt),
                          ([48, 48, 48], [16, 16, 5], table([a, a, a], 3)),   # listed three times, held twice
                          ([16, 16, 16], [1, 1, 1], table([[4], [3], [3]], 3))):
        with pytest.raises(pkv.KVError) as e:
            pool.prepare_evict(t, lens, keep)
        assert e.value.status == pkv.KV_ERR_INVALID_ARG
    assert ([pool.refcount(i) for i in range(5)], pool.stats()) == before


def test_prepare_evict_and_the_prefix_cache(pkv):
    """A block whose rows change leaves the prefix cache; one that is only
    released stays findable."""
    pool = pkv.KVPool(6, 16, 2, 64)
    tokens = list(range(48))
    a = pool.alloc(3)
    pool.register_prefix(a, tokens)
    assert pool.cached_blocks() == 3
    dst = pool.prepare_evict(table([a], 3), [48], [16])
    assert dst.tolist() == [[a[0], -1, -1]]
    assert pool.cached_blocks() == 2 and pool.match_prefix(tokens) == []
    # keeping everything changes nothing
    pool = pkv.KVPool(6, 16, 2, 64)
    a = pool.alloc(3)
    pool.register_prefix(a, tokens)
    assert pool.prepare_evict(table([a], 3), [48], [48]).tolist() == [a]
    assert pool.match_prefix(tokens) == a
    # nothing kept: every block is released, all still findable
    pool.free(a)
    assert pool.prepare_evict(table([a], 3), [48], [0]).tolist() == [[-1] * 3]
    assert pool.stats() == (0, 6) and pool.match_prefix(tokens) == a


def test_prepare_evict_blocks_reserved_ahead(pkv):
    """Blocks that a row lists beyond its tokens stay the sequence's: behind
    the kept blocks, in their order, with their references."""
    pool = pkv.KVPool(16, 16, 2, 64)
    a, b, c, d = pool.alloc(4), pool.alloc(4), pool.alloc(3), pool.alloc(2)
    bt = table([a, b, c, d], 4)
    dst = pool.prepare_evict(bt, [40, 20, 48, 0], [16, 20, 1, 0])
    assert dst.tolist() == [[a[0], a[3], -1, -1], b, [c[0], -1, -1, -1], d + [-1, -1]]
    assert [pool.refcount(i) for i in a + b + c + d] == [1, 0, 0, 1] + [1] * 4 + [1, 0, 0] + [1, 1]
    assert pool.stats() == (9, 7)
    held = [int(x) for row in dst for x in row if x >= 0]
    pool.free(held)                                            # every reference is in the tables
    assert pool.stats() == (0, 16)
    # a shared block is replaced, the reserved ones follow its replacement
    pool = pkv.KVPool(8, 16, 2, 64)
    a = pool.alloc(5)
    pool.fork(a[:2])
    dst = pool.prepare_evict(table([a], 6), [33], [17])
    assert dst.tolist() == [[5, 6, a[3], a[4], -1, -1]]
    assert [pool.refcount(i) for i in a] == [1, 1, 0, 1, 1]
    # nothing kept: the reserved blocks come first
    pool = pkv.KVPool(4, 16, 2, 64)
    a = pool.alloc(3)
    assert pool.prepare_evict(table([a], 3), [16], [0]).tolist() == [[a[1], a[2], -1]]
    assert pool.stats() == (2, 2)


def test_prepare_evict_allocates_nothing(pkv):
    """In a process that can get no more memory the call works (a C++ exception
    would end it at the C entry)."""
    import subprocess
    import sys
    code = """
import resource, sys
import numpy as np
import paged_kv_cache_97_gb300 as pkv
pool = pkv.KVPool(1 << 22, 16, 2, 64)
ids = pool.alloc(4)
pool.fork(ids[:1])
bt = np.array([ids], np.int32)
pool.prepare_evict(np.full((1, 4), -1, np.int32), [0], [0])
with open("/proc/self/statm") as f:
    now = int(f.read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (now + (4 << 20), resource.RLIM_INFINITY))
dst = pool.prepare_evict(bt, [64], [20])
assert dst.tolist() == [[4, ids[1], -1, -1]], dst
print("done")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(pkv.__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stderr[-500:]


def test_prepare_evict_arguments(pkv):
    pool = pkv.KVPool(4, 16, 2, 64)
    with pytest.raises(TypeError):
        pool.prepare_evict(np.zeros((2, 2), np.int64), [0, 0], [0, 0])
    with pytest.raises(ValueError):
        pool.prepare_evict(np.zeros((2, 2), np.int32), [0, 0], [0])
    t = np.zeros((1, 2), np.int32)
    n = np.zeros(1, np.int32)
    lib = pkv.load()
    for args in ((None, t.ctypes.data, 2, n.ctypes.data, n.ctypes.data, 1, t.ctypes.data + 64),
                 (pool._h, t.ctypes.data, 2, n.ctypes.data, n.ctypes.data, 1, t.ctypes.data),
                 (pool._h, None, 2, n.ctypes.data, n.ctypes.data, 1, t.ctypes.data),
                 (pool._h, t.ctypes.data, 0, n.ctypes.data, n.ctypes.data, 1, t.ctypes.data + 64)):
        assert lib.kv_pool_prepare_evict(*args) == pkv.KV_ERR_INVALID_ARG
    assert pool.prepare_evict(np.zeros((0, 2), np.int32), [], []).shape == (0, 2)
