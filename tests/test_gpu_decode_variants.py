"""The variants of the decoding-step kernels that the calls choose by their sizes (each is run, and what was chosen is read
from a captured launch), several calls at once, and faults in one expert or token beside sound ones. Bounds as
tests/test_gpu_decode.py derives them."""
import ctypes

import pytest
import torch

from tests.test_gpu_decode import U, _close, _decode_state, _decode_step, _gen, _layer, _norm_case, _run_gemv, _run_norm, _x

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_res", [True, False])
@pytest.mark.parametrize("M,K", [(3, 8448), (130, 9472), (1, 16128), (2, 16640), (5, 31232), (9, 8192), (2, 8704), (593, 8960),
                                 (600, 16640)])
def test_norm_steps_per_thread(osc, M, K, with_res):
    """One, two and four steps of a thread, the last one whole or not for all threads, few rows and many."""
    X, res, gamma = _norm_case(M, K, M + K)
    _run_norm(osc, X, res if with_res else None, gamma, 1e-6)


# ---- what a call launches -----------------------------------------------------------------------

def _launched(call):
    """(CTAs, threads of one, CTAs of a cluster) of each kernel that the call launches, from a captured graph."""
    cuda = ctypes.CDLL("libcuda.so.1")
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    raw, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cuda.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cuda.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        kind, params, attr = ctypes.c_int(-1), (ctypes.c_uint32 * 64)(), (ctypes.c_uint32 * 32)()
        assert cuda.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0 and kind.value == 0   # a kernel
        assert cuda.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), params) == 0   # func (8 bytes), grid, block
        assert cuda.cuGraphKernelNodeGetAttribute(ctypes.c_void_p(node), 4, attr) == 0   # the cluster's dimensions
        out.append((params[2], params[5], max(1, attr[0])))
    return out


def _gemv_launch(osc, M, N, K, G, share=0.0):
    X, Y = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda"), torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    QW = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    SW = torch.zeros(osc.osc_scale_bytes(N, K, G), dtype=torch.uint8, device="cuda")
    L, K_L, WL = None, 0, None
    if share:
        L = torch.full((K // G,), -1, dtype=torch.int8, device="cuda")
        L[:int(share * (K // G))] = 0
        K_L = (int(share * (K // G)) + 15) // 16 * 16
        WL = torch.zeros((N, K_L), dtype=torch.bfloat16, device="cuda")
    got = _launched(lambda: osc.osc_gemv(X, G, L, K_L, QW, SW, WL, N, Y))
    assert len(got) == 1
    return got[0]


def test_products_take_the_variants_that_the_tests_name(osc):
    """The shapes that test_gemv_splits and test_gemv_longest_k run are split over clusters, into several numbers of
    parts, with one unit to a cluster and with more; short ones run with few warps, those of more rows in
    passes on every SM."""
    parts = {}
    for M, N, K, G in [(1, 544, 6144, 32), (3, 1376, 12288, 32), (2, 1440, 12288, 16), (1, 2560, 32768, 64),
                       (5, 1536, 16384, 16), (12, 2576, 16384, 32), (16, 1184, 16384, 64), (8, 672, 12288, 32)]:
        ctas, threads, S = _gemv_launch(osc, M, N, K, G, 0.02)
        assert S > 1 and ctas % S == 0 and threads in (256, 512), (M, N, K, G)
        parts.setdefault(S, []).append((N + 31) // 32 > ctas // S)
    assert len(parts) >= 4 and any(any(v) for v in parts.values()) and not all(all(v) for v in parts.values())
    for M, K, G in [(1, 262144, 32), (3, 262144, 64), (9, 131072, 16), (17, 65536, 32)]:
        assert _gemv_launch(osc, M, 32, K, G)[2] == 8
    assert _gemv_launch(osc, 1, 2048, 2048, 32)[1:] == (256, 1)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert _gemv_launch(osc, 1, 24576, 4096, 32) == (sms, 512, 1)
    assert _gemv_launch(osc, 16, 24576, 4096, 32) == (sms, 256, 1)
    assert _gemv_launch(osc, 333, 4096, 768, 32) == (sms, 256, 1)


@pytest.mark.parametrize("M,N,K,G", [(1, 128, 8192, 32), (2, 128, 10240, 16), (1, 128, 12288, 32), (5, 128, 14336, 64),
                                     (4, 256, 16384, 32)])
def test_gemv_every_number_of_parts(osc, M, N, K, G):
    """Four units or eight in as many parts as give a warp its item: 4, 5, 6, 7 and 8."""
    assert _gemv_launch(osc, M, N, K, G, 0.02)[2] == min(8, K // 256 // 8)
    w = _layer(osc, 1, N, K, G, 1, 0.02, K)
    _run_gemv(osc, w, _x(M, K, N))


# ---- one bad expert, one bad token --------------------------------------------------------------

def _routed(osc, E=6, N=272, K=768, G=32, rows=70, seed=3):
    w = _layer(osc, E, N, K, G, 1, 0.4, 91)
    ids = torch.randint(0, E, (rows,), generator=_gen(seed), device="cuda", dtype=torch.int32)
    return w, _x(rows, K, seed), ids


def _grouped(osc, w, X, ids, fan=1, L=None):
    Y = torch.empty((ids.numel(), w["N"]), dtype=torch.bfloat16, device="cuda")
    Yf = torch.empty((ids.numel(), w["N"]), device="cuda")
    osc.osc_gemv_grouped(X, fan, ids, w["E"], w["G"], w["L"] if L is None else L, w["K_L"], w["QW"], w["SW"], w["WL"], w["N"], Y, Yf)
    return Y, Yf


@pytest.mark.parametrize("rows", [6, 30, 70, 300])
@pytest.mark.parametrize("fault", ["entry", "many"])
def test_grouped_bad_table_of_one_expert(osc, rows, fault):
    """An entry past the group, or more entries than columns, is reported when a row chooses that expert, and the
    other experts' rows come out as before."""
    w, X, ids = _routed(osc, rows=rows)
    ids[0], ids[-1] = 4, 1
    Y, Yf = _grouped(osc, w, X, ids)
    assert osc.osc_status() == (0, 0)
    bad = w["L"].clone()
    if fault == "entry":
        bad.view(6, -1)[4, 11] = w["G"]
    else:
        bad[4] = 5                               # 24 entries, K_L = 16
        assert w["K_L"] < bad[4].numel()
    Z, Zf = _grouped(osc, w, X, ids, L=bad)
    assert osc.osc_status()[0] == -6
    keep = ids != 4
    assert torch.equal(Yf[keep], Zf[keep]) and torch.equal(Y[keep], Z[keep])
    ids[ids == 4] = 2                            # nobody reads that table
    Z, Zf = _grouped(osc, w, X, ids, L=bad)
    assert osc.osc_status() == (0, 0)
    for e in range(6):
        r = (ids == e).nonzero()[:, 0]
        _close(Z[r], Zf[r], X[r].double(), w["W64"][e])


@pytest.mark.parametrize("rows", [1, 6, 30, 70, 300])
@pytest.mark.parametrize("fan", [1, 3])
def test_grouped_nan_and_infinity_stay_in_their_tokens(osc, rows, fan):
    w, X, ids = _routed(osc, rows=rows)
    X = X[:(rows + fan - 1) // fan].contiguous()
    Y, Yf = _grouped(osc, w, X, ids, fan)
    token = X.shape[0] // 2
    hit = torch.arange(rows, device="cuda") // fan == token
    entry = int(w["L"].view(6, -1)[int(ids[token * fan]), 9])
    for c in (5, 9 * 32 + max(entry, 0)):        # a channel of the 4-bit weights (or the table's), one of the table
        for bad in (float("nan"), float("inf")):
            X2 = X.clone()
            X2[token, c] = bad
            Z, Zf = _grouped(osc, w, X2, ids, fan)
            assert torch.equal(Zf[~hit], Yf[~hit]) and torch.equal(Z[~hit], Y[~hit])
            for r in hit.nonzero()[:, 0].tolist():
                ref = X2[token].double() @ w["W64"][int(ids[r])].t()     # infinity times a zero weight: NaN
                assert bool(torch.where(ref.isnan(), Zf[r].isnan(), Zf[r].double() == ref).all())
    assert osc.osc_status() == (0, 0)


def test_grouped_same_expert_twice_for_a_token(osc):
    """The two rows may lie in passes of different sizes, whose fp32 sums run in another order: equal within the bound, not
    in bits."""
    w, X, ids = _routed(osc, rows=40)
    ids = ids.view(20, 2).clone()
    ids[::3, 1] = ids[::3, 0]
    Y, Yf = _grouped(osc, w, X[:20].contiguous(), ids.view(-1), 2)
    Yf = Yf.view(20, 2, -1)
    for t in range(20):
        for j in range(2):
            ref, A = (f(w["W64"][int(ids[t, j])]) @ f(X[t].double()) for f in (lambda v: v, torch.abs))
            assert bool(((Yf[t, j].double() - ref).abs() <= 240 * U * A + 1e-37).all())


# ---- several at once -----------------------------------------------------------------------------

OUT = ("h", "y", "q8", "s8", "z", "u", "f")


def _states(osc):
    """Two decoding steps that share nothing and take different variants, with what each gives alone."""
    a, b = _decode_state(osc, 3, 1024), _decode_state(osc, 2, 2048)
    b["qkv"] = _layer(osc, 1, 400, 2048, 16, 2, 0.4, 73)
    b["up"] = _layer(osc, 8, 96, 2048, 32, 1, 0.0, 74)
    b["ids"] = torch.tensor([1, 6, 6, 3], dtype=torch.int32, device="cuda")
    want = []
    for s in (a, b):
        s["h"].copy_(s["res"])
        _decode_step(osc, s)
        torch.cuda.synchronize()
        want.append([s[k].clone() for k in OUT])
    return (a, b), want


def _same(states, want):
    for s, w in zip(states, want):
        for k, v in zip(OUT, w):
            assert torch.equal(s[k], v), k


def test_different_calls_on_two_streams_at_once(osc):
    states, want = _states(osc)
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(5):
        for s in states:
            for k in OUT:
                s[k].zero_()
        torch.cuda.synchronize()
        for _ in range(10):
            for s, st in zip(states, streams):
                with torch.cuda.stream(st):
                    s["h"].copy_(s["res"])
                    _decode_step(osc, s)
        torch.cuda.synchronize()
        _same(states, want)
    assert osc.osc_status() == (0, 0)


def test_two_captured_graphs_at_once(osc):
    states, want = _states(osc)
    graphs, streams = [], [torch.cuda.Stream() for _ in states]
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(4):
                s["h"].copy_(s["res"])
                _decode_step(osc, s)
        graphs.append(g)
    for s in states:
        for k in OUT:
            s[k].zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    _same(states, want)
    assert osc.osc_status() == (0, 0)
