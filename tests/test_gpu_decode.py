"""GPU parity of the decoding-step operators against their definitions in 64 bits:
osc_add_rmsnorm_quantize_fp8, osc_gemv and osc_gemv_grouped, and the three run together.

Tolerances, with u = 2^-24 (half a step of fp32):

Norm. h is one fp32 addition (relative error u). The sum of squares passes at most 32 fused steps
in a thread, 5 shuffles and 32 warps: relative error below 70 u, so below 35 u after the root;
division, root and the two products add 5 u. y is within DY = 48 u of the definition, H within a
bf16 half step (2^-8) more of h, Y of y, and a code's value within half a step of E4M3
(2^-4 relative, 2^-10 of the scale near zero) of y cut at 448 of the scale. The exponent follows
from the largest |y| unless that lies within DY of a power of two.

Products. With A = sum |x| |w| over everything an output sums: each mma adds 17 terms with an error of at
most 17 u of the largest (truncated alignment). They run in chains of eight over four scale blocks (up to 2
rows), four over two (up to 4 rows) or two over one, so a chain errs by at most 8 * 17 u = 136 u of
its own share of A and all chains by 136 u A. The fp32 additions that follow err by u A each at most: 4 over
an item's steps (16 with one scale block of 16 a step, whose chains are single mma's), 20 over a warp's items
for K up to 16384, 16 over the warps, 8 over a cluster. W_L's mma's run in one chain, up to 48 of 17 u each,
on at most 6 % of A here: 49 u A. Token values below 2^-31 of their run's maximum add at most 2^-39 of it
each. Together below (136 + 4 + 20 + 16 + 8 + 49 + 1) u A < 240 u A, which is used. The bf16 output equals the
fp32 one rounded."""
import numpy as np
import pytest
import torch

from tests._layout import pad_rows_zero, scale_offsets, unswizzle_scales

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DY = 48 * U
GUARD = 64


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


class Guarded:
    """An output buffer of a size with filled guards around it, which have to stay as they were."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape))
        self.all = torch.full((n + 2 * GUARD,), 77, dtype=torch.uint8, device="cuda").to(dtype) if dtype == torch.uint8 \
            else torch.full((n + 2 * GUARD,), 77.0, dtype=dtype, device="cuda")
        self.t = self.all[GUARD:GUARD + n].view(shape)

    def check(self):
        assert bool((self.all[:GUARD] == 77).all()) and bool((self.all[-GUARD:] == 77).all())


# ---- residual, norm, MXFP8 --------------------------------------------------------------------

def _norm_case(M, K, seed, scale=1.0):
    g = _gen(seed)
    X = (torch.randn((M, K), generator=g, device="cuda") * scale).bfloat16()
    X[:, 5] *= 40
    res = (torch.randn((M, K), generator=g, device="cuda") * 3 * scale).bfloat16()
    gamma = (1 + 0.3 * torch.randn(K, generator=g, device="cuda")).bfloat16()
    return X, res, gamma


def _check_norm(X, res, gamma, eps, H, Y, Q, S):
    M, K = X.shape
    h = X.double() + (res.double() if res is not None else 0)
    y = h * gamma.double() / torch.sqrt(h.square().mean(1, keepdim=True) + eps) if eps > 0 else \
        torch.nan_to_num(h * gamma.double() / torch.sqrt(h.square().mean(1, keepdim=True)))
    if H is not None:
        assert bool(((H.double() - h).abs() <= h.abs() * (2.0 ** -8 + 4 * U)).all())
    if Y is not None:
        assert bool(((Y.double() - y).abs() <= y.abs() * (2.0 ** -8 + DY) + 2.0 ** -134).all())
    s = S.cpu().numpy()
    assert pad_rows_zero(s, M, K, 32)
    e = unswizzle_scales(s, M, K, 32).astype(np.int64)
    amax = y.abs().view(M, K // 32, 32).amax(2).cpu().numpy()

    def exponent(a):
        return np.where(a > 0, np.maximum(np.floor(np.log2(np.maximum(a, 1e-300))) - 8, -127), -127)
    lo, hi = exponent(amax * (1 - DY)), exponent(amax * (1 + DY))
    assert np.all((e == lo) | (e == hi))
    two = torch.from_numpy(2.0 ** e.astype(np.float64)).cuda().repeat_interleave(32, 1)
    q = Q.view(torch.float8_e4m3fn).view(M, K).double()
    assert bool(torch.isfinite(q).all())
    cut = torch.minimum(y.abs(), 448 * two) * torch.sign(y)
    off = (q * two - cut).abs()
    assert bool((off <= cut.abs() * (2.0 ** -4 + DY) + y.abs() * DY + two * 2.0 ** -10).all())
    # and nearly every code is the nearest one: only values within DY of a tie may fall to the other side
    near = (cut / two).to(torch.float32).to(torch.float8_e4m3fn).double()
    assert (near != q).double().mean().item() <= 1e-3


def _run_norm(osc, X, res, gamma, eps, want_h=True, want_y=True, inplace=None):
    M, K = X.shape
    Q, S = Guarded((M, K), torch.uint8), Guarded(((M + 127) // 128 * 128 * K // 32,), torch.uint8)
    H = Guarded((M, K), torch.bfloat16) if want_h else None
    Y = Guarded((M, K), torch.bfloat16) if want_y else None
    x, r = X.clone(), None if res is None else res.clone()
    h = H.t if H is not None else None
    if inplace == "X":
        h = x
    elif inplace == "res":
        h = r
    osc.osc_add_rmsnorm_quantize_fp8(x, r, gamma, eps, h, Y.t if Y is not None else None, Q.t, S.t)
    torch.cuda.synchronize()
    for b in (Q, S, H, Y):
        if b is not None:
            b.check()
    if inplace != "X":
        assert torch.equal(x, X)
    if res is not None and inplace != "res":
        assert torch.equal(r, res)
    _check_norm(X, res, gamma, eps, h, Y.t if Y is not None else None, Q.t, S.t)
    return h, Y.t if Y is not None else None, Q.t, S.t


@pytest.mark.parametrize("M,K", [(1, 256), (1, 4096), (2, 512), (3, 768), (5, 8192), (7, 12288), (1, 32768), (2, 20480),
                                 (127, 1280), (128, 2048), (129, 2304), (600, 256), (601, 4096), (700, 6144),
                                 (595, 8448), (593, 32768)])
def test_norm_shapes(osc, M, K):
    X, res, gamma = _norm_case(M, K, 100 + M + K)
    _run_norm(osc, X, res, gamma, 1e-6)


@pytest.mark.parametrize("M", [3, 640])
@pytest.mark.parametrize("want", [(False, False, False), (False, True, False), (True, False, False), (True, False, True),
                                  (False, False, True)])
def test_norm_optional_arguments(osc, M, want):
    has_res, want_h, want_y = want
    X, res, gamma = _norm_case(M, 1536, 7)
    _run_norm(osc, X, res if has_res else None, gamma, 1e-5, want_h, want_y)


@pytest.mark.parametrize("where", ["X", "res"])
@pytest.mark.parametrize("M", [2, 900])
def test_norm_stream_updated_in_place(osc, where, M):
    X, res, gamma = _norm_case(M, 2048, 8)
    a = _run_norm(osc, X, res, gamma, 1e-6, want_h=False, inplace=where)
    b = _run_norm(osc, X, res, gamma, 1e-6)
    for s, t in zip(a, b):
        assert torch.equal(s, t)


def test_norm_edge_rows(osc):
    K = 1024
    X, res, gamma = _norm_case(8, K, 9)
    X[0] = 0
    res[0] = 0                                   # an all-zero row
    X[1] = -res[1]                               # a row that cancels
    X[2] = 1e-30
    res[2] = 0                                   # far below eps
    X[3] *= 1e14
    res[3] *= 1e14                               # large
    X[4, 32:64] = 0
    res[4, 32:64] = 0                            # an empty block
    X[5, 1:] = 0
    res[5, 1:] = 0                               # one value in the row
    res[6] = X[6] * 2.0 ** -12                   # bits of the smaller summand beyond bf16
    for eps in (1e-6, 1.0):
        _run_norm(osc, X, res, gamma, eps)
    _run_norm(osc, X[:2].contiguous(), res[:2].contiguous(), gamma, 0.0)
    Q = torch.full((2, K), 9, dtype=torch.uint8, device="cuda")
    S = torch.full((128 * K // 32,), 9, dtype=torch.uint8, device="cuda")
    osc.osc_add_rmsnorm_quantize_fp8(X[:2].contiguous(), res[:2].contiguous(), gamma, 0.0, None, None, Q, S)
    assert int((Q & 0x7F).count_nonzero()) == 0 and int(S.count_nonzero()) == 0


@pytest.mark.parametrize("M,K", [(5, 256), (3, 4096), (700, 512)])
def test_norm_nan_and_infinity_stay_in_their_rows(osc, M, K):
    X, res, gamma = _norm_case(M, K, 10)
    Y, Q = torch.empty((2, M, K), dtype=torch.bfloat16, device="cuda"), torch.empty((2, M, K), dtype=torch.uint8, device="cuda")
    S = torch.empty((2, (M + 127) // 128 * 128 * K // 32), dtype=torch.uint8, device="cuda")
    osc.osc_add_rmsnorm_quantize_fp8(X, res, gamma, 1e-6, None, Y[0], Q[0], S[0])
    X[0, 33] = float("nan")
    res[2, 7] = float("-inf")
    osc.osc_add_rmsnorm_quantize_fp8(X, res, gamma, 1e-6, None, Y[1], Q[1], S[1])
    keep = [i for i in range(M) if i not in (0, 2)]
    assert torch.equal(Y[0, keep], Y[1, keep]) and torch.equal(Q[0, keep], Q[1, keep])
    assert bool(Y[1, 0].isnan().all()) and bool((Q[1, 0] & 0x7F == 0x7F).all())
    # 1 / sqrt(infinity) = 0: the infinity's own product is NaN, the others are zeros
    at = torch.arange(K, device="cuda") == 7
    assert torch.equal(Y[1, 2].isnan(), at) and torch.equal(Q[1, 2] & 0x7F == 0x7F, at)
    assert int(Q[1, 2][~at].bitwise_and(0x7F).count_nonzero()) == 0


def test_norm_agrees_with_the_fp8_quantize_of_exact_rows(osc):
    """Rows whose norm is 1 and whose normed values are bf16: both quantizes see the same values."""
    K = 512
    X = torch.where(torch.rand((40, K), generator=_gen(3), device="cuda") < 0.5, -1.0, 1.0).bfloat16()
    gamma = (torch.randn(K, generator=_gen(4), device="cuda") * 5).bfloat16()
    _, _, Q, S = _run_norm(osc, X, None, gamma, 0.0)
    Q2, S2 = torch.empty_like(Q), torch.empty_like(S)
    osc.osc_quantize_fp8(X * gamma, Q2, S2)
    assert torch.equal(Q, Q2) and torch.equal(S, S2)


# ---- the products -----------------------------------------------------------------------------

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def _layer(osc, E, N, K, G, R, share, seed, sd=0.02, K_L=None):
    """E prepared weights with tables of R slots (a share of the entries set; a repeated channel and
    channels 0 and G - 1 among them), and the weights they stand for in 64 bits."""
    rng = np.random.default_rng(seed)
    g = _gen(seed)
    L = rng.integers(0, G, (E, K // G, R)).astype(np.int8)
    L[rng.random(L.shape) >= share] = -1
    if share > 0:
        L[:, 0, 0] = 0
        L[:, -1, 0] = G - 1
        if R > 1:
            L[:, 1, :2] = 3
    n = [int((L[e] >= 0).sum()) for e in range(E)]
    K_L = K_L if K_L is not None else (max(n) + 15) // 16 * 16
    QW = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    V = 16 if G == 16 else 32
    nb = (N + 127) // 128 * 128 * (K // V)
    SW = torch.empty((E, nb), dtype=torch.uint8, device="cuda")
    WL = torch.empty((E, N, K_L), dtype=torch.int16, device="cuda") if K_L else None
    Ld = torch.from_numpy(L).cuda() if share > 0 else None
    offs = torch.from_numpy(scale_offsets(N, K, V)).cuda()
    val = torch.from_numpy(E2M1).cuda()
    W64 = torch.empty((E, N, K), dtype=torch.float64, device="cuda")
    for e in range(E):
        W = (torch.randn((N, K), generator=g, device="cuda") * sd).bfloat16()
        W[0] = 0
        q, s, wl = osc.prepare_weight(W, G, Ld[e] if Ld is not None else None, K_L)
        QW[e], SW[e] = q, s
        codes = torch.stack((q & 15, q >> 4), 2).view(N, K).long()
        two = torch.pow(2.0, s[offs].double() - 127).repeat_interleave(V, 1)
        W64[e] = val[codes] * two
        if K_L:
            WL[e] = wl
            seen = set()
            for k in range(K // G):
                for r in range(R):
                    c = int(L[e, k, r])
                    if share > 0 and c >= 0 and (k, c) not in seen:
                        seen.add((k, c))
                        W64[e, :, k * G + c] = W[:, k * G + c].double()
    return dict(E=E, N=N, K=K, G=G, R=R, L=Ld, K_L=K_L, QW=QW, SW=SW, WL=WL, W64=W64)


def _x(M, K, seed, scale=1.0):
    X = torch.randn((M, K), generator=_gen(seed), device="cuda") * scale
    X[:, 7::96] *= 50
    return X.bfloat16()


def _close(Y, Yf, X64, W64, n_terms=240):
    ref = X64 @ W64.t()
    A = X64.abs() @ W64.abs().t()
    off = (Yf.double() - ref).abs()
    assert bool((off <= n_terms * U * A + 1e-37).all()), (off / A.clamp_min(1e-300)).max().item() / U
    assert torch.equal(Yf.bfloat16(), Y)


def _run_gemv(osc, w, X):
    M, N = X.shape[0], w["N"]
    Y, Yf = Guarded((M, N), torch.bfloat16), Guarded((M, N), torch.float32)
    args = (X, w["G"], w["L"], w["K_L"], w["QW"], w["SW"], w["WL"], N)
    osc.osc_gemv(*args, Y.t, Yf.t)
    Y2 = torch.empty_like(Y.t)
    osc.osc_gemv(*args, Y2)
    torch.cuda.synchronize()
    assert osc.osc_status() == (0, 0)
    Y.check()
    Yf.check()
    assert torch.equal(Y2.view(torch.int16), Y.t.view(torch.int16))
    _close(Y.t, Yf.t, X.double(), w["W64"][0])
    return Y.t, Yf.t


@pytest.mark.parametrize("G,R,share", [(32, 1, 0.7), (16, 1, 0.5), (64, 1, 0.9), (32, 3, 0.6), (16, 2, 0.3), (64, 2, 0.4),
                                       (32, 1, 0.0), (16, 1, 0.0)])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 33])
def test_gemv_rows_and_tables(osc, G, R, share, M):
    w = _layer(osc, 1, 272, 1280, G, R, share, 11)
    _run_gemv(osc, w, _x(M, 1280, M))


@pytest.mark.parametrize("N,K", [(16, 256), (48, 256), (128, 512), (144, 768), (112, 4096), (640, 4352), (80, 8192),
                                 (32, 12288), (256, 16384), (16, 33024)])
@pytest.mark.parametrize("M,G", [(1, 32), (5, 16), (12, 64)])
def test_gemv_shapes(osc, N, K, M, G):
    w = _layer(osc, 1, N, K, G, 1, 0.5 if K // G <= 4096 and K <= 8192 else 0.02, N + K)
    X = _x(M, K, N)
    if K <= 16384:
        _run_gemv(osc, w, X)
    else:                                        # up to 17 more additions: a warp's items
        Y, Yf = torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), torch.empty((M, N), device="cuda")
        osc.osc_gemv(X, G, w["L"], w["K_L"], w["QW"], w["SW"], w["WL"], N, Y, Yf)
        _close(Y, Yf, X.double(), w["W64"][0], 257)


@pytest.mark.parametrize("M,K,G", [(1, 262144, 32), (3, 262144, 64), (9, 131072, 16), (16, 16384, 16), (17, 65536, 32)])
def test_gemv_longest_k(osc, M, K, G):
    """K in parts over a cluster, fewer tokens a pass where they do not fit. Up to 64 more additions (a
    warp's items)."""
    N = 32
    W = (torch.randn((N, K), generator=_gen(71), device="cuda") * 0.02).bfloat16()
    QW, SW, _ = osc.prepare_weight(W, G)
    V = 16 if G == 16 else 32
    offs = torch.from_numpy(scale_offsets(N, K, V)).cuda()
    codes = torch.stack((QW & 15, QW >> 4), 2).view(N, K).long()
    W64 = torch.from_numpy(E2M1).cuda()[codes] * torch.pow(2.0, SW[offs].double() - 127).repeat_interleave(V, 1)
    X = _x(M, K, 72)
    Y, Yf = torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), torch.empty((M, N), device="cuda")
    osc.osc_gemv(X, G, None, 0, QW, SW, None, N, Y, Yf)
    _close(Y, Yf, X.double(), W64, 304)
    assert osc.osc_status() == (0, 0)


@pytest.mark.parametrize("M,N,K,G", [(1, 544, 6144, 32), (3, 1376, 12288, 32), (2, 1440, 12288, 16), (1, 2560, 32768, 64),
                                     (5, 1536, 16384, 16), (12, 2576, 16384, 32), (16, 1184, 16384, 64), (8, 672, 12288, 32)])
def test_gemv_splits(osc, M, N, K, G):
    """Parts of K over clusters of 2 to 8, with one unit and with several to a cluster, with a table
    (K = 32768: up to 17 more additions, a warp's items)."""
    w = _layer(osc, 1, N, K, G, 1, 0.02, N + K + M)
    X = _x(M, K, N)
    if K <= 16384:
        _run_gemv(osc, w, X)
    else:
        Y, Yf = torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), torch.empty((M, N), device="cuda")
        osc.osc_gemv(X, G, w["L"], w["K_L"], w["QW"], w["SW"], w["WL"], N, Y, Yf)
        _close(Y, Yf, X.double(), w["W64"][0], 257)


@pytest.mark.parametrize("M,N,K", [(17, 16, 256), (40, 16, 512), (1000, 16, 256), (333, 80, 768), (100, 4112, 256)])
def test_gemv_many_passes(osc, M, N, K):
    """Passes of one to many units, and fewer units than CTAs."""
    w = _layer(osc, 1, N, K, 32, 1, 0.5, M + N)
    _run_gemv(osc, w, _x(M, K, M))


@pytest.mark.parametrize("E,N,K,rows", [(300, 16, 256, 500), (40, 48, 512, 31), (3, 4112, 256, 100), (1, 32, 256, 2000)])
def test_grouped_many_passes(osc, E, N, K, rows):
    w = _layer(osc, E, N, K, 32, 1, 0.5, E)
    ids = torch.randint(-1, E, (rows,), generator=_gen(rows), device="cuda", dtype=torch.int32)
    _run_grouped(osc, w, _x(rows, K, E), 1, ids)
    assert osc.osc_status() == (0, 0)


def test_gemv_wide_w_l_and_extremes(osc):
    """K_L wider than the table; tokens of very different and of extreme sizes; weights from 1e-30
    to 1e25; an all-zero token."""
    for sd in (1e-30, 1.0, 1e25):
        w = _layer(osc, 1, 128, 512, 32, 1, 0.7, 5, sd=sd, K_L=64)
        X = _x(9, 512, 1)
        X[0] = 0
        X[1] *= 1e-36
        X[2] *= 1e10 if sd > 1e20 else 1e35
        X[3, ::2] *= 1e-9                        # 2^-30 of its neighbours, still exact
        X[4, 3:] = 0
        _run_gemv(osc, w, X)


def test_gemv_small_values_beside_large_ones(osc):
    """A value 2^-31 of its run's largest, alone against weights that are zero elsewhere, keeps its bits."""
    K, N = 256, 16
    W = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    W[:, 64] = 1.0
    QW, SW, _ = osc.prepare_weight(W, 32)
    X = torch.zeros((1, K), dtype=torch.bfloat16, device="cuda")
    X[0, 1] = 2.0 ** 20
    X[0, 64] = 1.9921875 * 2.0 ** -11
    Y = torch.empty((1, N), dtype=torch.bfloat16, device="cuda")
    osc.osc_gemv(X, 32, None, 0, QW, SW, None, N, Y)
    assert bool((Y == X[0, 64]).all())


@pytest.mark.parametrize("M", [1, 2, 4, 8, 9, 16, 19])
@pytest.mark.parametrize("where", [7, 300, 301])
def test_gemv_nan_and_infinity_stay_in_their_rows(osc, M, where):
    """In a channel of the 4-bit weights, in one of the table."""
    N, K = 144, 768
    w = _layer(osc, 1, N, K, 32, 1, 0.7, 6)
    X = _x(M, K, 3)
    Y, Yf = _run_gemv(osc, w, X)
    table = w["L"].view(-1).tolist()
    c = where // 32 * 32 + table[where // 32] if where == 300 and table[where // 32] >= 0 else where
    for bad in (float("nan"), float("inf")):
        X2 = X.clone()
        X2[M // 2, c] = bad
        Y2, Yf2 = torch.empty_like(Y), torch.empty_like(Yf)
        osc.osc_gemv(X2, 32, w["L"], w["K_L"], w["QW"], w["SW"], w["WL"], N, Y2, Yf2)
        keep = [i for i in range(M) if i != M // 2]
        assert torch.equal(Yf2[keep], Yf[keep]) and torch.equal(Y2[keep], Y[keep])
        ref = X2[M // 2].double() @ w["W64"][0].t()      # infinity times a zero weight: NaN
        assert bool(torch.where(ref.isnan(), Yf2[M // 2].isnan(), Yf2[M // 2].double() == ref).all())


@pytest.mark.parametrize("M", [1, 5, 16])
def test_gemv_table_without_channels(osc, M):
    """A table with no entry set has no W_L columns (K_L = 0): the 4-bit weights alone, and an entry
    set all the same is reported and left out."""
    w = _layer(osc, 1, 80, 512, 32, 1, 0.0, 8)
    X = _x(M, 512, 4)
    Y, Yf = _run_gemv(osc, w, X)
    table = torch.full((1, 16, 1), -1, dtype=torch.int8, device="cuda")
    Y2, Yf2 = torch.empty_like(Y), torch.empty_like(Yf)
    osc.osc_gemv(X, 32, table, 0, w["QW"], w["SW"], None, 80, Y2, Yf2)
    assert osc.osc_status() == (0, 0) and torch.equal(Yf, Yf2)
    Yg = torch.empty_like(Y)
    osc.osc_gemv_grouped(X, 1, torch.zeros(M, dtype=torch.int32, device="cuda"), 1, 32, table, 0, w["QW"], w["SW"],
                         None, 80, Yg, Yf2)
    assert osc.osc_status() == (0, 0)
    _close(Yg, Yf2, X.double(), w["W64"][0])
    table[0, 5, 0] = 9
    osc.osc_gemv(X, 32, table, 0, w["QW"], w["SW"], None, 80, Y2, Yf2)
    assert osc.osc_status()[0] == -6 and torch.equal(Yf, Yf2)


def test_gemv_bad_table_is_reported(osc):
    w = _layer(osc, 1, 128, 512, 32, 1, 0.7, 5)
    X, Y = _x(2, 512, 1), torch.empty((2, 128), dtype=torch.bfloat16, device="cuda")
    bad = w["L"].clone()
    bad.view(-1)[3] = 32
    osc.osc_gemv(X, 32, bad, w["K_L"], w["QW"], w["SW"], w["WL"], 128, Y)
    assert osc.osc_status()[0] == -6
    many = torch.zeros_like(w["L"])                              # 16 entries, no column for them
    osc.osc_gemv(X, 32, many, 0, w["QW"], w["SW"], None, 128, Y)
    assert osc.osc_status()[0] == -6
    osc.osc_gemv(X, 32, w["L"], w["K_L"], w["QW"], w["SW"], w["WL"], 128, Y)
    assert osc.osc_status() == (0, 0)


def _run_grouped(osc, w, X, fan, ids):
    rows, N = ids.numel(), w["N"]
    Y, Yf = Guarded((rows, N), torch.bfloat16), Guarded((rows, N), torch.float32)
    args = (X, fan, ids, w["E"], w["G"], w["L"], w["K_L"], w["QW"], w["SW"], w["WL"], N)
    osc.osc_gemv_grouped(*args, Y.t, Yf.t)
    Y2 = torch.empty_like(Y.t)
    osc.osc_gemv_grouped(*args, Y2)
    torch.cuda.synchronize()
    Y.check()
    Yf.check()
    assert torch.equal(Y2.view(torch.int16), Y.t.view(torch.int16))
    host = ids.cpu().tolist()
    for e in sorted(set(host)):
        r = [i for i, x in enumerate(host) if x == e]
        if 0 <= e < w["E"]:
            _close(Y.t[r], Yf.t[r], X[[i // fan for i in r]].double(), w["W64"][e])
        else:
            assert int(Y.t[r].view(torch.int16).count_nonzero()) == 0 and int(Yf.t[r].count_nonzero()) == 0
    return Y.t


@pytest.mark.parametrize("G,R,share", [(32, 1, 0.7), (16, 1, 0.5), (64, 2, 0.4), (32, 1, 0.0)])
@pytest.mark.parametrize("T,top", [(1, 1), (1, 8), (3, 2), (7, 8), (33, 8), (40, 2)])
def test_grouped(osc, G, R, share, T, top):
    w = _layer(osc, 9, 144, 768, G, R, share, 21)
    g = _gen(T * 10 + top)
    ids = torch.rand((T, 9), generator=g, device="cuda").argsort(1)[:, :top].reshape(-1).to(torch.int32).contiguous()
    _run_grouped(osc, w, _x(T, 768, T), top, ids)
    _run_grouped(osc, w, _x(T * top, 768, T), 1, ids)
    assert osc.osc_status() == (0, 0)


@pytest.mark.parametrize("rows", [1, 5, 17, 70, 333, 4096])
def test_grouped_id_patterns(osc, rows):
    """One expert for all rows, unused rows, nothing but unused rows, the last expert alone, long
    runs that end at the tile sizes."""
    w = _layer(osc, 40, 48, 256, 32, 1, 0.5, 31)
    X = _x(rows, 256, rows)
    i = torch.arange(rows, device="cuda")
    for ids in (torch.full_like(i, 39), torch.where(i % 3 == 0, -1, i % 40), torch.full_like(i, -5), i // 16 % 40,
                i // 8 % 40, (i * 7) % 40, torch.where(i == rows - 1, 38, -1), torch.where(i % 33 < 2, 4, 11)):
        _run_grouped(osc, w, X, 1, ids.to(torch.int32))
    assert osc.osc_status() == (0, 0)


@pytest.mark.parametrize("E,N,K,rows", [(4096, 16, 256, 4096), (2, 16, 32768, 40), (3, 32, 20480, 9), (600, 48, 512, 90)])
def test_grouped_limits(osc, E, N, K, rows):
    """The most experts and rows, the longest K (64 more additions there), more experts than threads."""
    g = _gen(E + K)
    W = (torch.randn((E, N, K), generator=g, device="cuda") * 0.02).bfloat16()
    QW = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    SW = torch.empty((E, 128 * K // 32), dtype=torch.uint8, device="cuda")
    for e in range(E):
        QW[e], SW[e], _ = osc.prepare_weight(W[e], 32)
    ids = torch.randint(0, E, (rows,), generator=g, device="cuda").to(torch.int32)
    X = _x(rows, K, 5)
    Y, Yf = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda"), torch.empty((rows, N), device="cuda")
    osc.osc_gemv_grouped(X, 1, ids, E, 32, None, 0, QW, SW, None, N, Y, Yf)
    offs = torch.from_numpy(scale_offsets(N, K, 32)).cuda()
    val = torch.from_numpy(E2M1).cuda()
    for r in range(0, rows, max(1, rows // 64)):
        q = QW[int(ids[r])]
        w = val[torch.stack((q & 15, q >> 4), 2).view(N, K).long()]
        w = w * torch.pow(2.0, SW[int(ids[r])][offs].double() - 127).repeat_interleave(32, 1)
        _close(Y[r:r + 1], Yf[r:r + 1], X[r:r + 1].double(), w, 304)
    assert osc.osc_status() == (0, 0)


def test_grouped_id_out_of_range_is_reported(osc):
    w = _layer(osc, 5, 128, 512, 32, 1, 0.7, 41)
    ids = torch.tensor([0, 5, 4, 2**31 - 1, -2**31, 4], dtype=torch.int32, device="cuda")
    _run_grouped(osc, w, _x(6, 512, 1), 1, ids)
    assert osc.osc_status()[0] == -6
    _run_grouped(osc, w, _x(2, 512, 1), 3, ids.clamp(0, 4))
    assert osc.osc_status() == (0, 0)


def test_grouped_rows_not_a_multiple_of_fan(osc):
    w = _layer(osc, 4, 64, 256, 64, 1, 0.5, 42)
    ids = torch.tensor([3, 1, 2, 2, 0, 3, 3], dtype=torch.int32, device="cuda")
    _run_grouped(osc, w, _x(3, 256, 1), 3, ids)


def test_grouped_equals_the_dense_product(osc):
    """One expert in the grouped form gives the dense form's bits."""
    w = _layer(osc, 1, 272, 1280, 32, 1, 0.7, 51)
    X = _x(6, 1280, 3)
    Y, _ = _run_gemv(osc, w, X)
    Z = _run_grouped(osc, w, X, 1, torch.zeros(6, dtype=torch.int32, device="cuda"))
    assert torch.equal(Y, Z)


def test_weights_past_2_to_the_31_bytes(osc):
    """The last expert's weights lie past 2^32 codes and 2^31 bytes."""
    E, N, K, G = 300, 4096, 4096, 32
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    QW = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    SW = torch.zeros((E, N * K // 32), dtype=torch.uint8, device="cuda")
    W = (torch.randn((N, K), generator=_gen(1), device="cuda") * 0.02).bfloat16()
    QW[-1], SW[-1], _ = osc.prepare_weight(W, G)
    X = _x(1, K, 2)
    Y, Z = (torch.empty((1, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    osc.osc_gemv_grouped(X, 1, torch.tensor([E - 1], dtype=torch.int32, device="cuda"), E, G, None, 0, QW, SW, None, N, Y)
    osc.osc_gemv(X, G, None, 0, QW[-1].clone(), SW[-1].clone(), None, N, Z)
    assert torch.equal(Y, Z) and int(Y.count_nonzero()) > N // 2


# ---- together ---------------------------------------------------------------------------------

def _decode_step(osc, s):
    """One layer's linears of a decoding step on fixed buffers: the residual's norm, the attention
    projection on the normed rows, an expert layer on a second norm, an FP8 module on its codes."""
    osc.osc_add_rmsnorm_quantize_fp8(s["x"], s["h"], s["gamma"], 1e-6, s["h"], s["y"], s["q8"], s["s8"])
    a, b = s["qkv"], s["up"]
    osc.osc_gemv(s["y"], a["G"], a["L"], a["K_L"], a["QW"], a["SW"], a["WL"], a["N"], s["z"])
    osc.osc_gemv_grouped(s["y"], 2, s["ids"], b["E"], b["G"], b["L"], b["K_L"], b["QW"], b["SW"], b["WL"], b["N"], s["u"])
    osc.osc_linear_fp8_fallback(s["q8"], s["s8"], s["w8"], s["sw8"], s["x"].shape[0], 256, s["x"].shape[1], s["f"])


def _decode_state(osc, M=3, K=1024):
    X, res, gamma = _norm_case(M, K, 61)
    W = (torch.randn((256, K), generator=_gen(62), device="cuda") * 0.02).bfloat16()
    w8 = torch.empty((256, K), dtype=torch.uint8, device="cuda")
    sw8 = torch.empty(osc.osc_scale_bytes(256, K, 0), dtype=torch.uint8, device="cuda")
    osc.osc_quantize_fp8(W, w8, sw8)
    e = lambda n, d=torch.bfloat16: torch.empty(n, dtype=d, device="cuda")  # noqa: E731
    return dict(x=X, h=res.clone(), res=res, gamma=gamma, y=e((M, K)), q8=e((M, K), torch.uint8),
                s8=e(128 * K // 32, torch.uint8), qkv=_layer(osc, 1, 400, K, 32, 1, 0.7, 63),
                up=_layer(osc, 8, 96, K, 16, 1, 0.4, 64), z=e((M, 400)), u=e((2 * M, 96)), f=e((M, 256)), W=W, w8=w8, sw8=sw8,
                ids=torch.tensor([5, 2, 0, 7, 2, 5][:2 * M], dtype=torch.int32, device="cuda"))


def _check_step(s, M=3):
    h = s["x"].double() + s["res"].double()
    y = h * s["gamma"].double() / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6)
    # each product against its own input as it was rounded (bf16 rows, 8-bit codes), in 64 bits
    ref = s["y"].double() @ s["qkv"]["W64"][0].t()
    A = s["y"].double().abs() @ s["qkv"]["W64"][0].abs().t()
    assert bool(((s["z"].double() - ref).abs() <= ref.abs() * 2.0 ** -8 + 241 * U * A).all())
    for r, e in enumerate(s["ids"].tolist()):
        x = s["y"][r // 2].double()
        ref, A = s["up"]["W64"][e] @ x, s["up"]["W64"][e].abs() @ x.abs()
        assert bool(((s["u"][r].double() - ref).abs() <= ref.abs() * 2.0 ** -8 + 241 * U * A).all())
    # and the FP8 module against the unquantized product: half a step of E4M3 on either side,
    # 2^-4 relative each (or 2^-10 of a scale that is at most 2^-8 of the block's maximum: the
    # small values' share, below 2^-10 of the block), the product of both, and bf16
    ref, A = y @ s["W"].double().t(), y.abs() @ s["W"].double().abs().t()
    assert bool(((s["f"].double() - ref).abs() <= A * 0.14 + ref.abs() * 2.0 ** -8).all())
    assert bool(((s["h"].double() - h).abs() <= h.abs() * (2.0 ** -8 + 4 * U)).all())


def test_decode_step_eager_side_stream_and_graph(osc):
    s = _decode_state(osc)
    _decode_step(osc, s)
    torch.cuda.synchronize()
    _check_step(s)
    first = [s[k].clone() for k in ("h", "y", "q8", "s8", "z", "u", "f")]
    side = torch.cuda.Stream()
    s["h"].copy_(s["res"])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _decode_step(osc, s)
    side.synchronize()
    for k, v in zip(("h", "y", "q8", "s8", "z", "u", "f"), first):
        assert torch.equal(s[k], v), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s["h"].copy_(s["res"])
        _decode_step(osc, s)
    for _ in range(3):
        for k in ("h", "y", "q8", "s8", "z", "u", "f"):
            s[k].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in zip(("h", "y", "q8", "s8", "z", "u", "f"), first):
            assert torch.equal(s[k], v), k
    assert osc.osc_status() == (0, 0)


def test_calls_on_two_streams_at_once(osc):
    """Two streams run the products and the norm at the same time on buffers of their own."""
    s, r = _decode_state(osc), _decode_state(osc)
    _decode_step(osc, s)
    torch.cuda.synchronize()
    want = [s[k].clone() for k in ("z", "u", "f")]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for q, st in zip((s, r), streams):
            with torch.cuda.stream(st):
                q["h"].copy_(q["res"])
                _decode_step(osc, q)
    torch.cuda.synchronize()
    for q in (s, r):
        for k, v in zip(("z", "u", "f"), want):
            assert torch.equal(q[k], v), k
