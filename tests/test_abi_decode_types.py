"""Types of the tensors that the binding of the decoding-step calls takes: those whose bits mean what the library reads
(bf16 or its bits as 16-bit integers, bytes for codes, scales and tables), and no other of the same size."""
import pytest
import torch

BF = torch.bfloat16


def _t(*shape, dtype=BF):
    return torch.zeros(shape, dtype=torch.uint8).repeat_interleave(torch.empty(0, dtype=dtype).element_size(), -1).view(dtype)


def _gemv():
    return dict(X=_t(2, 256), G=32, L=_t(8, dtype=torch.int8), K_L=16, QW=_t(128, 128, dtype=torch.uint8),
                SW=_t(1024, dtype=torch.uint8), WL=_t(128, 16), N=128, Y=_t(2, 128), Yf32=_t(2, 128, dtype=torch.float32))


def _grouped():
    return dict(_gemv(), fan=1, expert=torch.zeros(2, dtype=torch.int32), E=1)


def _norm():
    return dict(X=_t(2, 256), res=_t(2, 256), gamma=_t(256), eps=1e-6, H=_t(2, 256), Y=_t(2, 256),
                QX8=_t(2, 256, dtype=torch.uint8), SX=_t(1024, dtype=torch.uint8))


CALLS = [("osc_gemv", _gemv), ("osc_gemv_grouped", _grouped), ("osc_add_rmsnorm_quantize_fp8", _norm)]
WRONG = {1: (torch.bool, torch.float8_e5m2), 2: (torch.float16,), 4: (torch.int32,)}
ALSO = {1: (torch.int8, torch.uint8), 2: (torch.int16, torch.uint16), 4: ()}


def _as(t, dtype):
    return t if t.dtype == dtype else t.view(dtype)


@pytest.mark.parametrize("name,make", CALLS)
def test_types_of_the_same_size(name, make):
    from w4a4_outlier_separated_b200 import osc
    call = getattr(osc, name)
    with pytest.raises(ValueError, match="expected a CUDA tensor"):      # all types fit
        call(**make())
    for key, t in make().items():
        if not isinstance(t, torch.Tensor) or key == "expert":
            continue
        for dtype in WRONG[t.element_size()]:
            with pytest.raises(ValueError, match=f"^{key}: "):
                call(**{**make(), key: _as(t, dtype)})
        for dtype in ALSO[t.element_size()]:
            with pytest.raises(ValueError, match="expected a CUDA tensor"):
                call(**{**make(), key: _as(t, dtype)})


def test_types_that_name_what_the_bytes_are():
    from w4a4_outlier_separated_b200 import osc
    a, n = _gemv(), _norm()
    for call, ok, key, dtype in ((osc.osc_add_rmsnorm_quantize_fp8, n, "QX8", torch.float8_e4m3fn),
                                 (osc.osc_add_rmsnorm_quantize_fp8, n, "SX", torch.float8_e8m0fnu),
                                 (osc.osc_gemv, a, "SW", torch.float8_e8m0fnu),
                                 (osc.osc_gemv, a, "QW", torch.float4_e2m1fn_x2)):
        with pytest.raises(ValueError, match="expected a CUDA tensor"):
            call(**{**ok, key: ok[key].view(dtype)})
    for call, ok, key, dtype in ((osc.osc_add_rmsnorm_quantize_fp8, n, "SX", torch.float8_e4m3fn),
                                 (osc.osc_gemv, a, "QW", torch.float8_e4m3fn)):
        with pytest.raises(ValueError, match=f"^{key}: "):
            call(**{**ok, key: ok[key].view(dtype)})
