"""The matrix-vector products on tokens whose values span many binades: the weights of a row are zero wherever the
token is large, so that the small values are all that its output has. Against the definition in 64 bits, with the
bound that tests/test_gpu_decode.py derives (240 u A with A = sum |x| |w| over the row's own channels; products that
stay normal in fp32 carry no other error, whatever stands beside them)."""
import numpy as np
import pytest
import torch

from tests._layout import scale_offsets
from tests.test_gpu_decode import E2M1, Guarded, _close, _gen

pytestmark = pytest.mark.gpu
CLASSES = 4


def _class_layer(osc, E, N, K, G, R, share, seed):
    """E prepared weights whose row n has weights in the channels k with k % 4 == n % 4 alone, with tables of R
    slots, and the weights they stand for in 64 bits."""
    rng = np.random.default_rng(seed)
    g = _gen(seed)
    L = rng.integers(0, G, (E, K // G, R)).astype(np.int8)
    L[rng.random(L.shape) >= share] = -1
    K_L = (max(int((L[e] >= 0).sum()) for e in range(E)) + 15) // 16 * 16
    Ld = torch.from_numpy(L).cuda() if K_L else None
    V = 16 if G == 16 else 32
    offs = torch.from_numpy(scale_offsets(N, K, V)).cuda()
    val = torch.from_numpy(E2M1).cuda()
    own = torch.arange(K, device="cuda")[None] % CLASSES == torch.arange(N, device="cuda")[:, None] % CLASSES
    QW, SW, WL, W64 = [], [], [], []
    for e in range(E):
        W = (torch.randn((N, K), generator=g, device="cuda") * 0.02 * own).bfloat16()
        q, s, wl = osc.prepare_weight(W, G, Ld[e] if K_L else None, K_L)
        codes = torch.stack((q & 15, q >> 4), 2).view(N, K).long()
        w = val[codes] * torch.pow(2.0, s[offs].double() - 127).repeat_interleave(V, 1)
        for k, r in zip(*np.nonzero(L[e] >= 0)):
            c = int(k) * G + int(L[e, k, r])
            w[:, c] = W[:, c].double()
        QW.append(q), SW.append(s), WL.append(wl), W64.append(w)
    return dict(E=E, N=N, K=K, G=G, L=Ld, K_L=K_L, QW=torch.stack(QW), SW=torch.stack(SW),
                WL=torch.stack(WL) if K_L else None, W64=torch.stack(W64))


def _class_tokens(M, K, seed, step=35):
    """Rows whose class c of channels is 2^(-step c) of the first. Every third row is of one size; the others have
    runs of 256 channels in the first class alone, so that nothing large stands beside the small classes' sums.
    There are zeros among the values."""
    g = _gen(seed)
    X = torch.randn((M, K), generator=g, device="cuda").double()
    k = torch.arange(K, device="cuda")[None]
    m = torch.arange(M, device="cuda")[:, None]
    span = X * torch.pow(2.0, -step * (k % CLASSES).double())
    if K > 256:
        span = torch.where((k // 256 % 2 == m % 2) & (k % CLASSES > 0), 0.0, span)
    X = torch.where(m % 3 == 2, X, span) * torch.pow(2.0, (m * 7 % 19).double())
    X[:, 11::37] = 0
    return X.bfloat16()


def _dense(osc, w, X, n_terms=240):
    M, N = X.shape[0], w["N"]
    Y, Yf = Guarded((M, N), torch.bfloat16), Guarded((M, N), torch.float32)
    osc.osc_gemv(X, w["G"], w["L"], w["K_L"], w["QW"], w["SW"], w["WL"], N, Y.t, Yf.t)
    torch.cuda.synchronize()
    assert osc.osc_status() == (0, 0)
    Y.check()
    Yf.check()
    _close(Y.t, Yf.t, X.double(), w["W64"][0], n_terms)
    return Y.t, Yf.t


@pytest.mark.parametrize("M", [1, 2, 3, 4, 7, 9, 16, 17])
@pytest.mark.parametrize("down", [32, 39, 60, 130])
def test_a_value_alone_keeps_its_bits(osc, M, down):
    """One value against weights of 1, beside one 2^down larger against zeros."""
    K, N = 512, 32
    W = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    W[:, 64] = 1.0
    QW, SW, _ = osc.prepare_weight(W, 32)
    X = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    X[:, 1] = 2.0 ** 20
    X[:, 64] = 1.9921875 * 2.0 ** (20 - down)
    Y, Yf = torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), torch.empty((M, N), device="cuda")
    osc.osc_gemv(X, 32, None, 0, QW, SW, None, N, Y, Yf)
    assert bool((Y == X[0, 64]).all()) and bool((Yf == X[0, 64].float()).all())
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    osc.osc_gemv_grouped(X, 1, ids, 1, 32, None, 0, QW, SW, None, N, Y, Yf)
    assert bool((Y == X[0, 64]).all()) and bool((Yf == X[0, 64].float()).all())


@pytest.mark.parametrize("G,R,share", [(32, 1, 0.6), (16, 1, 0.0), (64, 2, 0.4), (16, 2, 0.5), (32, 1, 0.0)])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 16, 19])
def test_gemv_spans_of_binades(osc, G, R, share, M):
    w = _class_layer(osc, 1, 144, 1280, G, R, share, 7)
    _dense(osc, w, _class_tokens(M, 1280, M))


@pytest.mark.parametrize("M,N,K,G", [(1, 32, 256, 32), (1, 2048, 2048, 32), (2, 512, 2048, 16), (6, 512, 2048, 64),
                                     (1, 544, 6144, 32), (8, 672, 12288, 32), (3, 1376, 12288, 16), (12, 2576, 16384, 32),
                                     (16, 6144, 4096, 32), (40, 96, 512, 32)])
def test_gemv_spans_of_binades_by_shape(osc, M, N, K, G):
    """Rings of two and three stages, parts of K over clusters, several passes."""
    w = _class_layer(osc, 1, N, K, G, 1, 0.03, N)
    _dense(osc, w, _class_tokens(M, K, K))


@pytest.mark.parametrize("E,N,K,G,rows", [(5, 80, 768, 32, 7), (5, 80, 768, 16, 2), (9, 48, 1024, 64, 90), (2, 32, 20480, 32, 6),
                                          (1, 144, 512, 32, 3)])
def test_grouped_spans_of_binades(osc, E, N, K, G, rows):
    """(K = 20480: up to 17 more additions, a warp's items.)"""
    w = _class_layer(osc, E, N, K, G, 1, 0.03, E + K)
    X = _class_tokens(rows, K, rows)
    ids = torch.randint(-1, E, (rows,), generator=_gen(rows), device="cuda", dtype=torch.int32)
    Y, Yf = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda"), torch.empty((rows, N), device="cuda")
    osc.osc_gemv_grouped(X, 1, ids, E, G, w["L"], w["K_L"], w["QW"], w["SW"], w["WL"], N, Y, Yf)
    assert osc.osc_status() == (0, 0)
    for r, e in enumerate(ids.tolist()):
        if e >= 0:
            _close(Y[r:r + 1], Yf[r:r + 1], X[r:r + 1].double(), w["W64"][e], 257)
        else:
            assert int(Yf[r].count_nonzero()) == 0


@pytest.mark.parametrize("M", [2, 4, 6, 16])
def test_infinities_beside_spans_of_binades(osc, M):
    """An infinity in one token, small values in another's same channels: the other rows keep their bounds."""
    w = _class_layer(osc, 1, 144, 768, 32, 1, 0.5, 9)
    X = _class_tokens(M, 768, 5)
    X[1, 300] = float("inf")
    X[1, 20] = float("nan") if M > 2 else 1.0
    Y, Yf = torch.empty((M, 144), dtype=torch.bfloat16, device="cuda"), torch.empty((M, 144), device="cuda")
    osc.osc_gemv(X, 32, w["L"], w["K_L"], w["QW"], w["SW"], w["WL"], 144, Y, Yf)
    keep = [m for m in range(M) if m != 1]
    _close(Y[keep], Yf[keep], X[keep].double(), w["W64"][0])
    assert not bool(torch.isfinite(Yf[1]).any())


@pytest.mark.parametrize("G,R,share", [(32, 1, 0.5), (16, 2, 0.4), (64, 1, 0.0)])
@pytest.mark.parametrize("rows,fan", [(8, 8), (12, 3), (31, 2), (100, 4)])
def test_grouped_spans_of_binades_shared_rows(osc, G, R, share, rows, fan):
    """Rows that share an X row, per expert."""
    E, N, K = 7, 112, 768
    w = _class_layer(osc, E, N, K, G, R, share, 5)
    X = _class_tokens((rows + fan - 1) // fan, K, rows)
    ids = torch.randint(0, E, (rows,), generator=_gen(fan), device="cuda", dtype=torch.int32)
    Y, Yf = Guarded((rows, N), torch.bfloat16), Guarded((rows, N), torch.float32)
    osc.osc_gemv_grouped(X, fan, ids, E, G, w["L"], w["K_L"], w["QW"], w["SW"], w["WL"], N, Y.t, Yf.t)
    assert osc.osc_status() == (0, 0)
    Y.check()
    Yf.check()
    for r, e in enumerate(ids.tolist()):
        _close(Y.t[r:r + 1], Yf.t[r:r + 1], X[r // fan:r // fan + 1].double(), w["W64"][e])


@pytest.mark.parametrize("M", [1, 2, 4, 7, 16, 20])
@pytest.mark.parametrize("where", ["one", "some", "padding"])
def test_zeros_among_the_tokens(osc, M, where):
    """Zeros are no small values: with zeros in the weights' place instead, the bits are the same."""
    N, K = 144, 1536
    g = _gen(M)
    W = (torch.randn((N, K), generator=g, device="cuda") * 0.02).bfloat16()
    at = {"one": [777], "some": list(range(5, K, 50)), "padding": list(range(K - 300, K))}[where]
    X = torch.randn((M, K), generator=g, device="cuda").clamp(-3.9, 3.9).bfloat16()
    X[X.abs() < 2.0 ** -20] = 1.0
    X[:, ::256] = 4.0                            # the largest of each run of 256 channels, left alone
    at = [k for k in at if k % 256]
    X0 = X.clone()
    X0[:, at] = 0
    W[:, at] = 0
    QW, SW, _ = osc.prepare_weight(W, 32)
    out = []
    for x in (X, X0):
        Y, Yf = torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), torch.empty((M, N), device="cuda")
        osc.osc_gemv(x, 32, None, 0, QW, SW, None, N, Y, Yf)
        out.append((Y, Yf))
    assert torch.equal(out[0][1], out[1][1]) and torch.equal(out[0][0], out[1][0])
    assert osc.osc_status() == (0, 0)


def test_no_rows(osc):
    """Calls on no rows do nothing, whatever their outputs hold."""
    w = _class_layer(osc, 1, 32, 256, 32, 1, 0.5, 3)
    e = lambda *n, d=torch.bfloat16: torch.empty(n, dtype=d, device="cuda")  # noqa: E731
    osc.osc_gemv(e(0, 256), 32, w["L"], w["K_L"], w["QW"], w["SW"], w["WL"], 32, e(0, 32), e(0, 32, d=torch.float32))
    osc.osc_gemv_grouped(e(0, 256), 4, e(0, d=torch.int32), 1, 32, w["L"], w["K_L"], w["QW"], w["SW"], w["WL"], 32, e(0, 32))
    osc.osc_add_rmsnorm_quantize_fp8(e(0, 256), e(0, 256), e(256), 1e-6, e(0, 256), e(0, 256), e(0, 256, d=torch.uint8),
                                     e(0, d=torch.uint8))
    torch.cuda.synchronize()
    assert osc.osc_status() == (0, 0)
