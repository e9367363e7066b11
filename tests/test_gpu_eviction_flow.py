"""The eviction operators as a serving loop uses them together: prompts
appended into a block pool, their attention weights, decode steps that add to
them, selection, eviction (with forked sequences that share blocks) and decode
again.  Every call is compared with its 64-bit reference on the state that the
calls before it left on the device.  Also: the operators far into a large
pool, on a side stream, in a replayed graph, and their argument checks."""
import numpy as np
import pytest
import torch

import operator_reference as ref
from test_gpu_operators import same_bits, within, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_97_gb300 as pkv
    pkv.load()
    return pkv


class State:
    """What ref's functions read of a pool, from device tensors."""

    def __init__(self, s):
        self.k, self.v = s["k"].cpu(), s["v"].cpu()
        self.k_scale, self.v_scale = (None if s[n] is None else s[n].cpu() for n in ("ks", "vs"))
        self.tables = torch.from_numpy(s["table"].copy())
        self.L, self.heads = list(s["L"]), s["k"].shape[2]
        self.dim, self.block, self.dtype = s["k"].shape[3], s["k"].shape[1], s["dtype"]

    rows = ref.Pool.rows


@pytest.mark.parametrize("dtype", ["bf16", "int8", "fp8"])
def test_serving_loop(pkv, dtype):
    H, G, d, bs, B = 2, 4, 64, 16, 3
    budget, recent, width = 48, 16, 12
    nb = 40
    g = torch.Generator().manual_seed(3)
    pool = pkv.KVPool(nb, bs, H, d)
    torch_dtype = ref.DTYPES[dtype]
    shape = (nb, bs, H, d)
    s = dict(dtype=dtype)
    if dtype == "bf16":
        s["k"] = torch.full(shape, float("nan"), dtype=torch_dtype, device="cuda")
    else:
        s["k"] = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(torch_dtype)
    s["v"] = s["k"].clone()
    scales = dtype != "bf16"
    s["ks"] = torch.full((nb, H), float("nan"), device="cuda") if scales else None
    s["vs"] = s["ks"].clone() if scales else None
    weights = torch.full((B, H, width * bs), float("nan"), device="cuda")
    randn = lambda *sh: torch.randn(sh, generator=g).to(torch.bfloat16)  # noqa: E731

    def put(new_k, new_v, counts):
        """Appends each sequence's last tokens."""
        bt = torch.from_numpy(s["table"]).cuda()
        sl = torch.tensor(s["L"], dtype=torch.int32, device="cuda")
        qs = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        if scales:
            before = State(s)
            pkv.append_scaled(new_k.cuda(), new_v.cuda(), s["k"], s["v"], s["ks"], s["vs"], bt, sl, qs, max(counts))
            for a, b in zip((s["k"], s["ks"], s["v"], s["vs"]), ref.append(before, new_k, new_v, counts)):
                assert same_bits(a, b)
        else:
            pos = torch.tensor([L - n + i for L, n in zip(s["L"], counts) for i in range(n)], dtype=torch.int32)
            seq = torch.tensor([b for b, n in enumerate(counts) for _ in range(n)], dtype=torch.int32)
            slots = torch.empty(len(pos), dtype=torch.int64, device="cuda")
            pkv.token_slot_mapping(bt, pos.cuda(), nb, bs, slots, seq_idx=seq.cuda())
            pkv.reshape_and_cache(new_k.cuda(), new_v.cuda(), s["k"], s["v"], slots)
        return bt, sl, qs

    # prompts; sequence 2 is a fork of sequence 1 (same blocks, full ones)
    s["L"] = [37, 64]
    ids = [pool.alloc(3), pool.alloc(4)]
    s["table"] = np.full((2, width), -1, np.int32)
    for b, x in enumerate(ids):
        s["table"][b, :len(x)] = x
    T = sum(s["L"])
    put(randn(T, H, d), randn(T, H, d), s["L"])
    pool.fork(ids[1])
    s["table"] = np.concatenate([s["table"], s["table"][1:2]])
    s["L"] = [37, 64, 64]
    counts = [37, 64, 5]                                      # the fork scores its last tokens alone
    q = randn(sum(counts), H * G, d) * 2
    bt, sl = torch.from_numpy(s["table"]).cuda(), torch.tensor(s["L"], dtype=torch.int32, device="cuda")
    qs = torch.tensor([0, 37, 101, 106], dtype=torch.int32, device="cuda")
    want, tol = ref.prompt_weights(State(s), q, counts, torch.zeros(B, H, width * bs), d ** -0.5, False)
    pkv.attention_weights(weights, q.cuda(), s["k"], bt, sl, qs, 64, 64, d ** -0.5,
                          workspace(pkv.attention_weights_workspace_bytes(106, H * G, 64)),
                          accumulate=False, k_scale=s["ks"])
    for b, L in enumerate(s["L"]):
        within(weights[b, :, :L], want[b, :, :L], tol[b, :, :L])
    evictions = 0
    ws = workspace(pkv.weights_workspace_bytes(B, H * G, d, width * bs, bs))
    for step in range(14):
        # one decode step: blocks, append, attention with weights
        s["L"] = [n + 1 for n in s["L"]]
        pairs = pool.prepare_append(s["table"], s["L"])
        if len(pairs):
            pkv.copy_blocks(s["k"], s["v"], torch.from_numpy(pairs).cuda(), s["ks"], s["vs"])
        bt, sl, _ = put(randn(B, H, d), randn(B, H, d), [1] * B)
        st = State(s)
        q = randn(B, H * G, d) * 2
        before = weights.cpu()
        for b, L in enumerate(s["L"]):
            before[b, :, L - 1] = 0                            # may hold anything
        want, tol, ww, wtol = ref.decode_weights(st, q, torch.nan_to_num(before), d ** -0.5)
        out = torch.empty((B, H * G, d), dtype=torch.bfloat16, device="cuda")
        pkv.paged_attention_decode_weights(out, weights, q.cuda(), s["k"], s["v"], bt, sl, width * bs,
                                           d ** -0.5, ws, k_scale=s["ks"], v_scale=s["vs"])
        within(out, want, tol)
        for b, L in enumerate(s["L"]):
            within(weights[b, :, :L], ww[b, :, :L], wtol[b, :, :L])
        if step % 5 == 4 and max(s["L"]) > budget:
            idx = torch.empty((B, H, budget), dtype=torch.int32, device="cuda")
            num = torch.empty(B, dtype=torch.int32, device="cuda")
            pkv.select_tokens(idx, num, weights, sl, width * bs, recent)
            wi, wn = ref.select(weights.cpu(), s["L"], budget, recent)
            assert torch.equal(idx.cpu(), wi) and torch.equal(num.cpu(), wn)
            keep = num.cpu().numpy()
            dst = pool.prepare_evict(s["table"], s["L"], keep)
            shared = {int(x) for r in s["table"] for x in r if x >= 0 and pool.refcount(int(x)) > 1}
            assert not shared & {int(x) for r, n, m in zip(dst, s["L"], keep) if m < n for x in r}
            before, w0 = State(s), weights.cpu()
            pkv.evict_tokens(s["k"], s["v"], bt, sl, idx, num, dst_block_tables=torch.from_numpy(dst).cuda(),
                             weights=weights, k_scale=s["ks"], v_scale=s["vs"])
            got = (s["k"], s["v"], s["ks"], s["vs"], weights)
            for a, b in zip(got, ref.evict(before, wi, wn, torch.from_numpy(dst), w0)):
                if a is not None:
                    assert same_bits(a, b)
            s["table"], s["L"] = dst, keep.tolist()
            evictions += 1
    assert evictions == 2
    assert pkv.get_status()[1] == 0


def test_far_into_a_large_pool(pkv):
    """Offsets past 32 bits: the same blocks at the start of a small pool and at
    the end of one of more than 2^31 elements give the same bits."""
    H, d, bs, G = 8, 128, 32, 4
    nb = 2 ** 31 // (H * d * bs) + 200
    L = [100, 33]
    for dtype in ("int8", "bf16"):
        small = ref.Pool(L, H, d, bs, dtype, seed=1, extra=10)
        far = nb - small.num_blocks
        k, v, sc, bt, sl = small.on()
        big = {}
        for n, x in (("k", k), ("v", v)):
            big[n] = torch.empty((nb, bs, H, d), dtype=x.dtype, device="cuda")
            big[n][far:] = x
        bsc = {n: None if x is None else torch.cat([torch.zeros(far, H, device="cuda"), x]) for n, x in sc.items()}
        bbt = torch.where(bt >= 0, bt + far, bt)
        q = small.randn(2, H * G, d, scale=2.0).cuda()
        w = [torch.rand((2, H, 128), device="cuda")]
        w.append(w[0].clone())
        idx = torch.stack([torch.arange(1, 33)[None].expand(H, 32), torch.arange(1, 33)[None].expand(H, 32)])
        idx = idx.to(torch.int32).contiguous().cuda()
        num = torch.tensor([32, 32], dtype=torch.int32, device="cuda")
        qd = small.randn(2, H, d, scale=2.0).cuda()
        lam = torch.full((H // 2,), 0.5, device="cuda")
        new = small.randn(2, H, d).cuda(), small.randn(2, H, d).cuda()
        qs = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
        results = []
        for (kc, vc, scales, tab), wt in zip(((k, v, sc, bt), (big["k"], big["v"], bsc, bbt)), w):
            out = torch.empty((2, H * G, d), dtype=torch.bfloat16, device="cuda")
            od = torch.empty((2, H // 2, 2 * d), dtype=torch.bfloat16, device="cuda")
            pkv.paged_attention_decode_weights(out, wt, q, kc, vc, tab, sl, 128, 0.1,
                                               workspace(pkv.weights_workspace_bytes(2, H * G, d, 128, bs)), **scales)
            pkv.attention_weights(wt, q, kc, tab, sl, qs, 128, 1, 0.1, workspace(1 << 16), k_scale=scales["k_scale"])
            pkv.paged_diff_attention_decode(od, qd, kc, vc, tab, sl, 128, 0.1, lam, None, **scales)
            if dtype == "int8":
                pkv.append_scaled(*new, kc, vc, scales["k_scale"], scales["v_scale"], tab, sl)
            pkv.evict_tokens(kc, vc, tab, sl, idx, num, weights=wt, **scales)
            n = small.num_blocks
            results.append([out, od, wt, kc[-n:], vc[-n:]] + [x[-n:] for x in scales.values() if x is not None])
        for a, b in zip(*results):
            assert same_bits(a, b.cpu())
        del big, results
        torch.cuda.empty_cache()
    assert pkv.get_status()[1] == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_graph_of_every_operator(pkv, dtype):
    """One graph with all of them, captured on a side stream, replayed on
    restored state: the bits of the eager calls."""
    H, d, bs, G, L = 2, 64, 16, 2, [200, 60]
    pool = ref.Pool(L, H, d, bs, dtype, seed=2, width=14)
    k, v, sc, bt, sl = pool.on()
    q, qd = pool.randn(2, H * G, d, scale=2.0).cuda(), pool.randn(2, 2, d, scale=2.0).cuda()
    qp = pool.randn(90, H * G, d, scale=2.0).cuda()
    qs = torch.tensor([0, 80, 90], dtype=torch.int32, device="cuda")
    new = pool.randn(2, H, d, scale=3.0).cuda(), pool.randn(2, H, d, scale=3.0).cuda()
    lam = torch.full((1,), 0.4, device="cuda")
    w = torch.rand((2, H, 224), generator=pool.g).cuda()
    idx = torch.empty((2, H, 64), dtype=torch.int32, device="cuda")
    num = torch.empty(2, dtype=torch.int32, device="cuda")
    out = torch.empty((2, H * G, d), dtype=torch.bfloat16, device="cuda")
    od = torch.empty((2, 1, 2 * d), dtype=torch.bfloat16, device="cuda")
    ws = [workspace(n) for n in (pkv.weights_workspace_bytes(2, H * G, d, 224, bs),
                                 pkv.attention_weights_workspace_bytes(90, H * G, 224),
                                 pkv.diff_workspace_bytes(2, 1, d, 224, bs))]
    state = [x for x in (k, v, sc["k_scale"], sc["v_scale"], w) if x is not None]
    saved = [x.clone() for x in state]

    def run():
        if dtype == "fp8":
            pkv.append_scaled(*new, k, v, sc["k_scale"], sc["v_scale"], bt, sl)
        pkv.attention_weights(w, qp, k, bt, sl, qs, 224, 80, 0.125, ws[1], k_scale=sc["k_scale"])
        pkv.paged_attention_decode_weights(out, w, q, k, v, bt, sl, 224, 0.125, ws[0], **sc)
        pkv.paged_diff_attention_decode(od, qd, k, v, bt, sl, 224, 0.125, lam, None, workspace=ws[2], **sc)
        pkv.select_tokens(idx, num, w, sl, 224, 8)
        pkv.evict_tokens(k, v, bt, sl, idx, num, weights=w, **sc)

    def results():
        torch.cuda.synchronize()
        return [x.cpu().clone() for x in state + [idx, num, out, od]]

    def restore():
        for x, y in zip(state, saved):
            x.copy_(y)
        torch.cuda.synchronize()

    run()
    eager = results()
    restore()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    for a, b in zip(results(), eager):
        assert same_bits(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    for _ in range(2):
        restore()
        graph.replay()
        for a, b in zip(results(), eager):
            assert same_bits(a, b)
    assert pkv.get_status()[1] == 0


@pytest.mark.parametrize("dtype", ["bf16", "int8"])
def test_overlapping_calls(pkv, dtype):
    """Every operator on two streams at once, each with a state of its own, in
    small batches (clusters of CTAs side by side): the bits of the calls alone."""
    H, d, bs, G, L = 2, 64, 16, 2, [2000, 700]

    def state(seed):
        pool = ref.Pool(L, H, d, bs, dtype, seed=seed)
        k, v, sc, bt, sl = pool.on()
        i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
        bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        return dict(k=k, v=v, sc=sc, bt=bt, sl=sl, q=pool.randn(2, H * G, d, scale=2.0).cuda(),
                    few=pool.randn(7, H * G, d, scale=2.0).cuda(), many=pool.randn(300, H * G, d, scale=2.0).cuda(),
                    fs=torch.tensor([0, 4, 7], dtype=torch.int32, device="cuda"),
                    ms=torch.tensor([0, 180, 300], dtype=torch.int32, device="cuda"),
                    new=[pool.randn(2, H, d, scale=2.0).cuda() for _ in range(2)],
                    lam=torch.full((1,), 0.4, device="cuda"), qd=pool.randn(2, 2, d, scale=2.0).cuda(),
                    w=torch.rand((2, H, 2000), generator=pool.g).cuda(), idx=i32(2, H, 600), num=i32(2),
                    out=bf(2, H * G, d), od=bf(2, 1, 2 * d),
                    ws=[workspace(n) for n in (pkv.weights_workspace_bytes(2, H * G, d, 2000, bs),
                                               pkv.attention_weights_workspace_bytes(300, H * G, 2000),
                                               pkv.diff_workspace_bytes(2, 1, d, 2000, bs))])

    def run(s, stream):
        k, v, bt, sl, sc, w = (s[n] for n in ("k", "v", "bt", "sl", "sc", "w"))
        if dtype != "bf16":
            pkv.append_scaled(*s["new"], k, v, sc["k_scale"], sc["v_scale"], bt, sl, stream=stream)
        for q, qs, n in ((s["few"], s["fs"], 4), (s["many"], s["ms"], 180)):
            pkv.attention_weights(w, q, k, bt, sl, qs, 2000, n, 0.125, s["ws"][1], k_scale=sc["k_scale"], stream=stream)
        pkv.paged_attention_decode_weights(s["out"], w, s["q"], k, v, bt, sl, 2000, 0.125, s["ws"][0], stream=stream, **sc)
        pkv.paged_diff_attention_decode(s["od"], s["qd"], k, v, bt, sl, 2000, 0.125, s["lam"], None,
                                        workspace=s["ws"][2], stream=stream, **sc)
        pkv.select_tokens(s["idx"], s["num"], w, sl, 2000, 100, stream=stream)
        pkv.evict_tokens(k, v, bt, sl, s["idx"], s["num"], weights=w, stream=stream, **sc)

    def results(s):
        torch.cuda.synchronize()
        return [s[n].cpu() for n in ("k", "v", "w", "idx", "num", "out", "od")] + \
            [x.cpu() for x in s["sc"].values() if x is not None]

    alone = []
    for seed in (1, 2):
        s = state(seed)
        run(s, torch.cuda.current_stream().cuda_stream)
        alone.append(results(s))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        both = [state(seed) for seed in (1, 2)]
        torch.cuda.synchronize()
        for s, stream in zip(both, streams):
            run(s, stream.cuda_stream)
        for s, want in zip(both, alone):
            for a, b in zip(results(s), want):
                assert same_bits(a, b)
    assert pkv.get_status()[1] == 0


def test_argument_checks(pkv):
    """Shapes, types and layouts that do not fit are refused before a launch."""
    pool = ref.Pool([40, 20], 2, 64, 16, "int8", seed=1, extra=4)
    k, v, sc, bt, sl = pool.on()
    f32 = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    ws = workspace(1 << 16)
    bad = [
        (ValueError, lambda: pkv.select_tokens(i32(2, 2, 8), i32(3), f32(2, 2, 64), sl, 64, 1)),
        (ValueError, lambda: pkv.select_tokens(i32(2, 2, 8), i32(2), f32(2, 3, 64), sl, 64, 1)),
        (ValueError, lambda: pkv.select_tokens(i32(2, 8, 2).transpose(1, 2), i32(2), f32(2, 2, 64), sl, 64, 1)),
        (TypeError, lambda: pkv.select_tokens(i32(2, 2, 8), i32(2), f32(2, 2, 64).double(), sl, 64, 1)),
        (pkv.KVError, lambda: pkv.select_tokens(i32(2, 2, 8), i32(2), f32(2, 2, 64), sl, 65, 1)),
        (pkv.KVError, lambda: pkv.select_tokens(i32(2, 2, 8), i32(2), f32(2, 2, 64), sl, 64, 9)),
        (pkv.KVError, lambda: pkv.select_tokens(i32(2, 2, 0), i32(2), f32(2, 2, 64), sl, 64, 0)),
        (ValueError, lambda: pkv.evict_tokens(k, v, bt, sl, i32(2, 2, 8), i32(2))),                # no scales
        (ValueError, lambda: pkv.evict_tokens(k, v[:-1], bt, sl, i32(2, 2, 8), i32(2), **sc)),
        (ValueError, lambda: pkv.evict_tokens(k, v, bt, sl, i32(2, 1, 8), i32(2), **sc)),
        (ValueError, lambda: pkv.evict_tokens(k, v, bt, sl, i32(2, 2, 8), i32(2), dst_block_tables=i32(1, 3), **sc)),
        (ValueError, lambda: pkv.evict_tokens(k, v, bt, sl, i32(2, 2, 8), i32(2), weights=f32(2, 1, 64), **sc)),
        (ValueError, lambda: pkv.evict_tokens(k, v, bt, sl, i32(2, 2, 8), i32(2), k_scale=f32(3, 2), v_scale=sc["v_scale"])),
        (ValueError, lambda: pkv.append_scaled(bf(3, 2, 64), bf(3, 2, 64), k, v, **sc, block_tables=bt, seq_lens=sl)),
        (ValueError, lambda: pkv.append_scaled(bf(2, 2, 64), bf(2, 2, 32), k, v, **sc, block_tables=bt, seq_lens=sl)),
        (ValueError, lambda: pkv.append_scaled(bf(2, 2, 64), bf(2, 2, 64), k, v, **sc, block_tables=bt, seq_lens=sl, query_start=i32(2))),
        (TypeError, lambda: pkv.append_scaled(f32(2, 2, 64), bf(2, 2, 64), k, v, **sc, block_tables=bt, seq_lens=sl)),
        (TypeError, lambda: pkv.append_scaled(bf(2, 2, 64), bf(2, 2, 64), bf(4, 16, 2, 64), bf(4, 16, 2, 64), None, None, bt, sl)),
        (ValueError, lambda: pkv.paged_attention_decode_weights(bf(2, 4, 64), f32(2, 2, 64), bf(2, 4, 32), k, v, bt, sl, 64, 1.0, ws, **sc)),
        (ValueError, lambda: pkv.paged_attention_decode_weights(bf(2, 4, 64), f32(1, 2, 64), bf(2, 4, 64), k, v, bt, sl, 64, 1.0, ws, **sc)),
        (pkv.KVError, lambda: pkv.paged_attention_decode_weights(bf(2, 4, 64), f32(2, 2, 63), bf(2, 4, 64), k, v, bt, sl, 64, 1.0, ws, **sc)),
        (pkv.KVError, lambda: pkv.paged_attention_decode_weights(bf(2, 4, 64), f32(2, 2, 64), bf(2, 4, 64), k, v, bt, sl, 64, 1.0, None, **sc)),
        (pkv.KVError, lambda: pkv.paged_attention_decode_weights(bf(2, 4, 64), f32(2, 2, 64), bf(2, 4, 64), k, v, bt, sl, 64, 1.0, ws[:64], **sc)),
        (ValueError, lambda: pkv.attention_weights(f32(2, 2, 64), bf(3, 4, 64), k, bt, sl, i32(4), 64, 2, 1.0, ws, k_scale=sc["k_scale"])),
        (ValueError, lambda: pkv.attention_weights(f32(2, 2, 64), bf(3, 4, 64), k, bt, sl, i32(3), 64, 2, 1.0, ws)),
        (pkv.KVError, lambda: pkv.attention_weights(f32(2, 2, 64), bf(3, 4, 64), k, bt, sl, i32(3), 64, 2, 1.0, None, k_scale=sc["k_scale"])),
        (ValueError, lambda: pkv.paged_diff_attention_decode(bf(2, 2, 64), bf(2, 4, 64), k, v, bt, sl, 64, 1.0, f32(2), **sc)),
        (ValueError, lambda: pkv.paged_diff_attention_decode(bf(2, 2, 128), bf(2, 4, 64), k, v, bt, sl, 64, 1.0, f32(3), **sc)),
        (ValueError, lambda: pkv.paged_diff_attention_decode(bf(2, 2, 128), bf(2, 4, 64), k, v, bt, sl, 64, 1.0, f32(2), norm_weight=f32(64), **sc)),
        (pkv.KVError, lambda: pkv.paged_diff_attention_decode(bf(2, 2, 128), bf(2, 4, 64), k, v, bt, sl, 600, 1.0, f32(2), **sc)),
    ]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was taken")
    torch.cuda.synchronize()
    assert pkv.get_status()[1] == 0
    assert torch.equal(k.cpu(), pool.k) and torch.equal(sc["k_scale"].cpu(), pool.k_scale)


def test_empty_batch(pkv):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    k = bf(4, 16, 2, 64)
    k8, sc = k.to(torch.int8), f32(4, 2)
    pkv.select_tokens(i32(0, 2, 8), i32(0), f32(0, 2, 64), i32(0), 64, 1)
    pkv.evict_tokens(k, k, i32(0, 2), i32(0), i32(0, 2, 8), i32(0))
    pkv.append_scaled(bf(0, 2, 64), bf(0, 2, 64), k8, k8, sc, sc, i32(0, 2), i32(0))
    pkv.append_scaled(bf(0, 2, 64), bf(0, 2, 64), k8, k8, sc, sc, i32(3, 2), i32(3), i32(4), 1)
    pkv.paged_attention_decode_weights(bf(0, 4, 64), f32(0, 2, 64), bf(0, 4, 64), k, k, i32(0, 2), i32(0), 32, 1.0, None)
    pkv.attention_weights(f32(0, 2, 64), bf(0, 4, 64), k, i32(0, 2), i32(0), i32(1), 32, 1, 1.0, None)
    pkv.paged_diff_attention_decode(bf(0, 2, 128), bf(0, 4, 64), k, k, i32(0, 2), i32(0), 32, 1.0, f32(2))
    assert pkv.get_status()[1] == 0
