"""Argument checks of the decoding-step operators (osc_add_rmsnorm_quantize_fp8, osc_gemv,
osc_gemv_grouped): every refusal comes back before anything touches a device, from the C ABI as a
code and from the binding as an exception."""
import ctypes

import pytest
import torch

V, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from w4a4_outlier_separated_b200 import build
    return ctypes.CDLL(build.build())


@pytest.fixture(scope="module")
def p16():
    buf = (ctypes.c_uint8 * 4096)()
    p = V((ctypes.addressof(buf) + 15) // 16 * 16)
    p.keep = buf
    return p


def _norm(lib, p, **k):
    a = dict(X=p, res=p, gamma=p, eps=1e-6, M=4, K=256, H=p, Y=p, Q=p, S=p)
    a.update(k)
    f = lib.osc_add_rmsnorm_quantize_fp8
    f.argtypes = [V, V, V, F, I, I, V, V, V, V, V]
    return f(a["X"], a["res"], a["gamma"], a["eps"], a["M"], a["K"], a["H"], a["Y"], a["Q"], a["S"], None)


def _gemv(lib, p, **k):
    a = dict(X=p, M=4, K=256, G=32, L=p, R=1, K_L=16, QW=p, SW=p, WL=p, N=128, Y=p, Yf=None)
    a.update(k)
    f = lib.osc_gemv
    f.argtypes = [V, I, I, I, V, I, I, V, V, V, I, V, V, V]
    return f(*(a[n] for n in ("X", "M", "K", "G", "L", "R", "K_L", "QW", "SW", "WL", "N", "Y", "Yf")), None)


def _grouped(lib, p, **k):
    a = dict(X=p, rows=4, fan=1, expert=p, E=8, K=256, G=32, L=p, R=1, K_L=16, QW=p, SW=p, WL=p, N=128, Y=p, Yf=None)
    a.update(k)
    f = lib.osc_gemv_grouped
    f.argtypes = [V, I, I, V, I, I, I, V, I, I, V, V, V, I, V, V, V]
    return f(*(a[n] for n in ("X", "rows", "fan", "expert", "E", "K", "G", "L", "R", "K_L", "QW", "SW", "WL", "N", "Y",
                              "Yf")), None)


def _off(p):
    return V(p.value + 2)


def test_norm_refusals(lib, p16):
    for k in ("X", "gamma", "Q", "S"):
        assert _norm(lib, p16, **{k: None}) == -1, k
    for k in ("X", "res", "gamma", "H", "Y", "Q", "S"):
        assert _norm(lib, p16, **{k: _off(p16)}) == -2, k
    for eps in (-1e-6, NAN, INF):
        assert _norm(lib, p16, eps=eps) == -1
    assert _norm(lib, p16, K=264) == -2
    assert _norm(lib, p16, K=0) == -1
    assert _norm(lib, p16, K=32768 + 256) == -1
    assert _norm(lib, p16, M=-1) == -1
    assert _norm(lib, p16, M=2**31 - 1, K=256) == -1          # scale positions past 31 bits
    assert _norm(lib, p16, M=0, X=None, res=None, gamma=None, H=None, Y=None, Q=None, S=None) == 0
    assert _norm(lib, p16, M=0, eps=-1.0) == -1


@pytest.mark.parametrize("call", [_gemv, _grouped])
def test_product_refusals(lib, p16, call):
    m = "M" if call is _gemv else "rows"
    for k in ("X", "QW", "SW", "Y"):
        assert call(lib, p16, **{k: None}) == -1, k
    for k in ("X", "QW", "SW", "WL", "Y", "Yf"):
        assert call(lib, p16, **{k: _off(p16)}) == -2, k
    assert call(lib, p16, G=24) == -3
    assert call(lib, p16, K=128) == -2
    assert call(lib, p16, N=8) == -2
    assert call(lib, p16, K_L=8) == -2
    assert call(lib, p16, K_L=-16) == -1
    assert call(lib, p16, K_L=32768) == -1
    assert call(lib, p16, WL=None) == -1                      # K_L without W_L
    assert call(lib, p16, L=None) == -1                       # K_L without a table
    assert call(lib, p16, R=0) == -1 and call(lib, p16, R=4) == -1
    assert call(lib, p16, K=45056, R=3) == -1                 # 1408 groups x 3 slots > 4096
    assert call(lib, p16, N=0) == -1
    assert call(lib, p16, N=2**31 - 16, K=256) == -1
    assert call(lib, p16, **{m: -1}) == -1
    assert call(lib, p16, **{m: 0, "X": None, "QW": None, "SW": None, "WL": None, "L": None, "Y": None}) == 0
    assert call(lib, p16, **{m: 0, "G": 24}) == -3


def test_row_limits(lib, p16):
    assert _gemv(lib, p16, M=65535 * 16 + 1) == -1
    assert _grouped(lib, p16, rows=4097) == -1
    for k in (dict(E=0), dict(E=4097), dict(fan=0), dict(expert=None)):
        assert _grouped(lib, p16, **k) == -1, k
    assert _grouped(lib, p16, expert=_off(p16)) == -2
    assert _gemv(lib, p16, K=262144 + 256, L=None, K_L=0) == -1
    assert _grouped(lib, p16, K=32768 + 256, G=64) == -1
    assert _grouped(lib, p16, E=4096, N=2**19) == -1           # E x N past 31 bits
    small = dict(K=256, L=None, K_L=0)
    assert _gemv(lib, p16, M=8192, N=2**23, **small) == -1     # M x N past 36 bits
    assert _grouped(lib, p16, rows=4096, N=2**24, E=1, **small) == -1


def _cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_before_the_library():
    """Shapes, element sizes, strides and devices that do not fit raise ValueError (CPU tensors are
    refused last, so the messages name the first fault)."""
    from w4a4_outlier_separated_b200 import osc
    X, Y = _cpu(2, 256), _cpu(2, 128)
    QW, SW = _cpu(128, 128, dtype=torch.uint8), _cpu(1024, dtype=torch.uint8)
    ok = dict(X=X, G=32, L=None, K_L=0, QW=QW, SW=SW, WL=None, N=128, Y=Y)
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        osc.osc_gemv(**ok)
    for k, v in (("X", X.float()), ("X", _cpu(2, 512)[:, ::2]), ("QW", QW[:64]), ("SW", SW[:512]), ("Y", Y[:1]),
                 ("Y", Y.float()), ("Yf32", Y)):
        with pytest.raises(ValueError, match=f"^{k}: "):
            osc.osc_gemv(**{**ok, k: v})
    with pytest.raises(osc.OSCError, match="OSC_ERR_G"):
        osc.osc_gemv(**{**ok, "G": 8})
    ids = torch.zeros(2, dtype=torch.int32)
    ok = dict(X=X, fan=1, expert=ids, E=1, G=32, L=None, K_L=0, QW=QW, SW=SW, WL=None, N=128, Y=Y)
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        osc.osc_gemv_grouped(**ok)
    with pytest.raises(ValueError, match="int32"):
        osc.osc_gemv_grouped(**{**ok, "expert": ids.long()})
    for k in (dict(fan=2), dict(fan=0), dict(E=2), dict(X=X[:1])):
        with pytest.raises(ValueError):
            osc.osc_gemv_grouped(**{**ok, **k})
    with pytest.raises(osc.OSCError, match="OSC_ERR_G"):
        osc.osc_gemv_grouped(**{**ok, "G": 8})
    Q, S, gamma = _cpu(2, 256, dtype=torch.uint8), _cpu(1024, dtype=torch.uint8), _cpu(256)
    ok = dict(X=X, res=X, gamma=gamma, eps=1e-6, H=X, Y=None, QX8=Q, SX=S)
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        osc.osc_add_rmsnorm_quantize_fp8(**ok)
    for k, v in (("res", X[:1]), ("gamma", gamma.float()), ("H", X.t()), ("Y", Q), ("QX8", X), ("SX", S[:512])):
        with pytest.raises(ValueError, match=f"^{k}: "):
            osc.osc_add_rmsnorm_quantize_fp8(**{**ok, k: v})
