"""Host checks of the int8 rows and product: every refusal comes before any CUDA call."""
import ctypes

import pytest
import torch

import post_weight_quantization_rowwise_b200 as m

V = ctypes.c_void_p


def test_rows_refusals():
    Q = m._lib.iqq_quantize_i8_rows
    ok = [0, V(16), 64, V(16), 64, V(16), 4, 64, None, None]

    def call(**at):
        args = list(ok)
        for i, v in at.items():
            args[int(i[1:])] = v
        return Q(*args)

    assert call(_0=3) == 5 and call(_0=-1) == 5
    assert call(_6=-1) == 2 and call(_7=-1) == 2
    assert call(_2=63) == 2 and call(_4=48) == 2                     # rows that overlap
    assert call(_6=1 << 40, _7=1 << 30) == 2
    assert call(_4=72) == 3 and call(_3=V(8)) == 3 and call(_1=V(2)) == 3 and call(_5=V(2)) == 3
    assert call(_8=V(2)) == 3
    assert call(_1=None) == 1 and call(_3=None) == 1 and call(_5=None) == 1
    assert Q(0, None, 0, None, 0, None, 0, 64, None, None) == 0
    assert Q(0, None, 0, None, 0, None, 4, 0, None, None) == 0


def test_gemm_refusals():
    G = m._lib.iqq_gemm_i8
    ok = [V(16), 64, V(16), V(16), 64, V(16), None, 0, V(16), 8, 4, 8, 64, None, None]

    def call(**at):
        args = list(ok)
        for i, v in at.items():
            args[int(i[1:])] = v
        return G(*args)

    assert call(_7=3) == 5
    assert call(_10=-1) == 2 and call(_11=-1) == 2 and call(_12=-1) == 2 and call(_12=131072, _1=131072, _4=131072) == 2
    assert call(_1=48) == 2 and call(_4=48) == 2 and call(_9=7) == 2
    assert call(_1=72) == 3 and call(_4=72) == 3 and call(_0=V(8)) == 3 and call(_3=V(8)) == 3
    assert call(_2=V(2)) == 3 and call(_5=V(2)) == 3 and call(_6=V(2)) == 3 and call(_8=V(2)) == 3 and call(_13=V(2)) == 3
    assert call(_7=1, _8=V(1)) == 3
    for i in (0, 2, 3, 5, 8):
        assert call(**{"_%d" % i: None}) == 1
    assert G(*[None, 0, None, None, 0, None, None, 0, None, 0, 0, 8, 64, None, None]) == 0
    assert G(*[None, 0, None, None, 0, None, None, 0, None, 0, 4, 0, 64, None, None]) == 0


def test_binding_refusals():
    with pytest.raises(ValueError):
        m.quantize_i8_rows(torch.zeros(2, 64))
    with pytest.raises(ValueError):
        m.quantize_i8_rows(torch.zeros(64))
    with pytest.raises(ValueError):
        m.gemm_i8(torch.zeros(2, 64, dtype=torch.int8), torch.ones(2), torch.zeros(3, 64, dtype=torch.int8), torch.ones(3))
    assert "gemm_i8" in m.__all__ and "quantize_i8_rows" in m.__all__


@pytest.mark.skipif(torch.cuda.is_available(), reason="what calls say without a device")
def test_without_a_device_every_call_says_why():
    """The CUDA error of the call itself (no device, or no driver for it), each time."""
    G, W = m._lib.iqq_gemm_i8, m._lib.iqq_last_cuda_error
    for n_tok, n_out, k in ((1, 8, 64), (4, 8, 64), (4000, 4000, 640), (4, 8, 64)):
        assert G(V(16), 640, V(16), V(16), 640, V(16), None, 0, V(16), n_out, n_tok, n_out, k, None, None) == 4
        assert W() in (35, 100), W()
