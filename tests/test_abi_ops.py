"""CPU checks of the operators' entry points (include/moe.h): arguments that they refuse, on the
host, before any CUDA call; workspace sizes; the bindings' checks of tensors."""
import ctypes

import pytest
import torch

import mixture_experts_layer_forward_b200 as moe
from mixture_experts_layer_forward_b200 import build as native_build

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
FAKE = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced: every call here is refused
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    native_build.build_library()
    return moe.library()


def select(**kw):
    args = dict(T=4, E=64, top_k=8, score=moe.SCORE_SIGMOID, n_group=8, top_group=4,
                group_score=moe.GROUP_SUM2, renorm=True, scale=2.5)
    ld = kw.pop("ld", 0)
    dtype = kw.pop("dtype", 1)
    args.update(kw)
    s = moe.Select.make(**args)
    s.ld, s.dtype = ld, dtype
    return s


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(top_k=0), INVALID), (dict(top_k=65), INVALID),
    (dict(score=2), INVALID), (dict(group_score=2), INVALID), (dict(dtype=2), INVALID),
    (dict(n_group=7), INVALID),                       # does not divide E
    (dict(n_group=0), INVALID), (dict(top_group=0), INVALID), (dict(top_group=9), INVALID),
    (dict(top_k=9, top_group=1), INVALID),            # the group that stays holds 8 experts
    (dict(ld=63), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(E=2048), UNSUPPORTED), (dict(E=256, top_k=33, top_group=8), UNSUPPORTED),
    (dict(E=128, n_group=64, top_group=32), UNSUPPORTED),
])
def test_select_problems_refused(lib, kw, code):
    s = select(**kw)
    assert lib.moe_route_select(s, FAKE, None, FAKE, FAKE, None, None) == code
    assert lib.moe_route_select_backward(s, FAKE, FAKE, FAKE, FAKE, None, None) == code


def test_select_pointers_refused(lib):
    s = select()
    for bad in (None, ODD):
        for i in range(3):
            p = [FAKE, FAKE, FAKE]
            p[i] = bad
            assert lib.moe_route_select(s, p[0], None, p[1], p[2], None, None) == INVALID
    assert lib.moe_route_select(s, FAKE, ODD, FAKE, FAKE, None, None) == INVALID
    assert lib.moe_route_select(s, FAKE, None, FAKE, FAKE, ODD, None) == INVALID
    for i in range(4):
        p = [FAKE] * 4
        p[i] = None
        assert lib.moe_route_select_backward(s, *p, None, None) == INVALID
    assert lib.moe_route_select(None, FAKE, None, FAKE, FAKE, None, None) == INVALID
    # no tokens: nothing to do, whatever the pointers
    assert lib.moe_route_select(select(T=0), None, None, None, None, None, None) == 0
    assert lib.moe_route_select_backward(select(T=0), None, None, None, None, None, None) == 0


def linear(**kw):
    lds = {k: kw.pop(k) for k in list(kw) if k.startswith("ld")}
    raw = {k: kw.pop(k) for k in list(kw) if k in ("out", "layout")}
    args = dict(M=16, N=64, K=64)
    args.update(kw)
    p = moe.Linear.make(**args)
    for k, v in lds.items():
        setattr(p, k, v)
    p.out_dtype = raw.get("out", 0)
    p.w_layout = raw.get("layout", 0)
    return p


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(act=4), INVALID),
    (dict(act=-1), INVALID), (dict(layout=2), INVALID), (dict(out=2), INVALID),
    (dict(ldx=56), INVALID), (dict(ldw=56), INVALID), (dict(ldr=56), INVALID), (dict(ldy=56), INVALID),
    (dict(act=moe.ACT_SWIGLU, ldz=64), INVALID),
    (dict(N=60), UNSUPPORTED), (dict(K=4), UNSUPPORTED), (dict(ldx=68), UNSUPPORTED),
    (dict(ldy=66, out=1), UNSUPPORTED), (dict(ldw=1 << 40), UNSUPPORTED),
    (dict(M=1 << 30, N=1 << 20), UNSUPPORTED),
])
def test_linear_problems_refused(lib, kw, code):
    p = linear(**kw)
    assert moe.moe_linear_workspace_size(p) == 0
    assert moe.moe_linear_backward_workspace_size(p) == 0
    assert lib.moe_linear_forward(p, *[FAKE] * 7, 1 << 30, None) == code
    assert lib.moe_linear_backward(p, *[FAKE] * 8, 1 << 30, None) == code


def test_linear_pointers_and_workspace_refused(lib):
    p = linear(act=moe.ACT_GELU_TANH)
    # x, W, bias, residual, y, z, ws
    for i in (0, 1, 4, 6):
        a = [FAKE] * 7
        a[i] = None
        assert lib.moe_linear_forward(p, *a, 1 << 20, None) == INVALID
    for i in range(7):
        a = [FAKE] * 7
        a[i] = ODD
        assert lib.moe_linear_forward(p, *a, 1 << 20, None) == INVALID
    assert lib.moe_linear_forward(p, *[FAKE] * 7, 255, None) == WORKSPACE
    # x, W, z, dy, dx, dW, dbias, ws
    for i in (0, 1, 2, 3, 7):
        a = [FAKE] * 8
        a[i] = None
        assert lib.moe_linear_backward(p, *a, 1 << 20, None) == INVALID
    a = [FAKE] * 8
    a[4] = a[5] = a[6] = None
    assert lib.moe_linear_backward(p, *a, 1 << 20, None) == INVALID
    n = moe.moe_linear_backward_workspace_size(p)
    assert n >= 256 + 16 * 64 * 2 + 64 * 4
    assert lib.moe_linear_backward(p, *[FAKE] * 8, n - 1, None) == WORKSPACE
    # an identity product of bf16 gradients needs no dz
    assert moe.moe_linear_backward_workspace_size(linear()) < n
    for tile, split, rc in ((64, 0, -1), (256, 2, -1), (96, 1, -1), (64, 3, -1), (64, 16, -1), (0, 0, 0)):
        assert lib.moe_set_linear_plan(tile, split) == rc


def test_dropout_arguments_refused(lib):
    f = lib.moe_dropout_add
    assert f(-1, 0, 32768, FAKE, FAKE, None, FAKE, None) == INVALID
    assert f(8, 2, 32768, FAKE, FAKE, None, FAKE, None) == INVALID
    for p in (-1, 65537):
        assert f(8, 0, p, FAKE, FAKE, None, FAKE, None) == INVALID
        assert lib.moe_dropout_add_backward(8, 0, p, FAKE, FAKE, FAKE, None) == INVALID
    for args in ((None, FAKE, None, FAKE), (FAKE, None, None, FAKE), (FAKE, FAKE, None, None),
                 (ODD, FAKE, None, FAKE), (FAKE, ODD, None, FAKE), (FAKE, FAKE, ODD, FAKE),
                 (FAKE, FAKE, None, ODD)):
        assert f(8, 0, 32768, *args, None) == INVALID
    assert f(0, 0, 32768, FAKE, None, None, None, None) == 0


def test_routed_layer_arguments_refused(lib):
    P = moe.Problem.make(16, 256, 512, 8, 2)
    big = 1 << 40
    # x, topk_idx, topk_w, W1, W2, shared, out, ws
    for i in (0, 1, 2, 3, 4, 6, 7):
        a = [FAKE] * 5 + [None, FAKE, FAKE]
        a[i] = None
        assert lib.moe_forward_routed(P, *a, big, None) == INVALID
    a = [FAKE] * 5 + [None, FAKE, FAKE]
    assert lib.moe_forward_routed(P, *a, 16, None) == WORKSPACE
    a[1] = ODD
    assert lib.moe_forward_routed(P, *a, big, None) == INVALID
    a[1] = FAKE
    a[5] = moe.SharedExpert(96, FAKE, FAKE, None)
    assert lib.moe_forward_routed(P, *a, big, None) == UNSUPPORTED
    # x, topk_idx, topk_w, W1, W2, dout, dx, dtopk_w, dW1, dW2, ws
    for i in range(11):
        a = [FAKE] * 11
        a[i] = None
        assert lib.moe_backward_routed(P, *a, big, None) == INVALID
    assert lib.moe_backward_routed(P, *[FAKE] * 11, 16, None) == WORKSPACE
    assert lib.moe_backward_routed(moe.Problem.make(16, 192, 512, 8, 2), *[FAKE] * 11, big,
                                   None) == UNSUPPORTED


def test_bindings_refuse_tensors():
    t = torch.zeros
    s = moe.Select.make(4, 16, 2)
    idx, w = t(4, 2, dtype=torch.int32), t(4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_route_select(s, t(4, 16), None, idx, w)
    with pytest.raises(TypeError):
        moe.moe_route_select(s, t(4, 16, dtype=torch.float16), None, idx, w)
    with pytest.raises(ValueError, match="shape"):
        moe.moe_route_select(s, t(4, 15), None, idx, w)
    p = moe.Linear.make(4, 16, 8)
    bf = torch.bfloat16
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_linear_forward(p, t(4, 8, dtype=bf), t(8, 16, dtype=bf), None, None, t(4, 16, dtype=bf),
                               t(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="shape"):
        moe.moe_linear_forward(p, t(4, 16, dtype=bf), t(8, 16, dtype=bf), None, None, t(4, 16, dtype=bf),
                               t(256, dtype=torch.uint8))
    with pytest.raises(TypeError):
        moe.Linear.make(4, 16, 8, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        moe.moe_set_linear_plan(96, 1)
    with pytest.raises(TypeError):
        moe.moe_dropout_add(t(8, dtype=torch.float64), None, t(8, dtype=torch.float64), 0.5,
                            t(2, dtype=torch.int64))
    for prob in (-0.1, 1.1, float("nan")):
        with pytest.raises(ValueError, match="prob"):
            moe.moe_dropout_add(t(8), None, t(8), prob, t(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_dropout_add(t(8), None, t(8), 0.5, t(2, dtype=torch.int64))
