"""Host-side checks of the expert operators' edges (no GPU needed)."""
import ctypes

import pytest

from differentiable_soft_top_amd import _lib

FAKE = ctypes.c_void_p(0x100000)
ODD = ctypes.c_void_p(0x100001)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_residual_refusals(lib):
    def call(dy=FAKE, dtype=1, off=FAKE, R=20, E=4, N=8, dr=FAKE):
        return lib.soft_topk_experts_residual_backward(dy, dtype, off, R, E, N, dr, None)

    for bad in (dict(dy=None), dict(off=None), dict(dr=None), dict(dtype=0), dict(dtype=3), dict(R=0), dict(R=-1),
                dict(R=1 << 31), dict(E=0), dict(E=1025), dict(N=0), dict(dy=ODD), dict(dr=ODD)):
        assert call(**bad) == _lib.EINVAL, bad


def test_combine_refuses_unknown_flags(lib):
    def call(y=FAKE, T=4, k=2, P=8, N=16, flags=0):
        return lib.soft_topk_combine_forward_ex(y, FAKE, FAKE, None, 1, T, k, P, N, flags, FAKE, None)

    for bad in (dict(flags=2), dict(flags=-1), dict(y=None), dict(T=0), dict(k=0), dict(P=0), dict(N=0)):
        assert call(**bad) == _lib.EINVAL, bad


def test_products_refuse_what_no_launch_holds(lib):
    # 2^32 work-items: 256 to a tile of 128 rows, or of 64 rows of the activation's gradient
    def fwd(R, K=1, N=1, act=0):
        return lib.soft_topk_experts_forward(FAKE, FAKE, None, None, 1, FAKE, None, R, R, 1, K, N, act, FAKE, None, None)

    def bwd(R, K=1, N=1, act=0, dx=FAKE, dw=FAKE, db=None):
        return lib.soft_topk_experts_backward(FAKE, FAKE, FAKE, FAKE, 1, FAKE, None, None, R, R, 1, 1, K, N, act, dx, dw,
                                              db, ctypes.c_void_p(0x200000), 1 << 50, None)

    most = (1 << 31) - 600
    assert fwd(most, N=130) == _lib.EINVAL  # ((2^31 - 600) / 128 + 1) 256 is still below, for one column of tiles
    assert fwd(1 << 30, N=130) == _lib.EINVAL
    assert bwd(most, K=130) == _lib.EINVAL
    assert bwd((1 << 30) + 64, act=1, dx=None) == _lib.EINVAL
    assert bwd((1 << 30) + 64, db=FAKE, dx=None) == _lib.EINVAL


def test_residual_refuses_host_tensors():
    import torch

    import differentiable_soft_top_amd as stk

    with pytest.raises(TypeError):
        stk.experts_residual_backward(torch.zeros(4, 2).half(), stk.Dispatch(torch.zeros(2, dtype=torch.int32)))
