"""The dense product with its epilogue, and its gradients, on the GPU against 64-bit references of
the formulas, element by element.

Tolerances. A sum of K products accumulates in fp32 in steps of 16: at most (K / 16 + 32) roundings
or truncations of one step (2^-23) of the absolute sum S = |x| |W| + |bias|. The activation passes
that on with a slope of at most 1.13 (GELU), 1.1 |up| + |silu| (SwiGLU), and adds 2^-20 of its value
(fast exponential and quotient). Then the rounding of the output's type, half a step."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_forward_b200 as moe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SWIGLU, GELU, RELU, IDENT = moe.ACT_SWIGLU, moe.ACT_GELU_TANH, moe.ACT_RELU, moe.ACT_IDENTITY
GC = (2 / np.pi) ** 0.5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


@pytest.fixture(autouse=True)
def _auto_plan():
    yield
    moe.moe_set_linear_plan(0, 0)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def make(M, K, N, act, nk, seed, out=BF):
    g = torch.Generator().manual_seed(seed)
    cols = 2 * N if act == SWIGLU else N
    r = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    return dict(x=r(M, K).to(BF), W=r(*((cols, K) if nk else (K, cols)), std=K ** -0.5).to(BF),
                bias=r(cols, std=0.3), res=r(M, N).to(BF), dy=r(M, N).to(out))


def act64(act, z, N):
    if act == SWIGLU:
        return z[:, :N] / (1 + torch.exp(-z[:, :N])) * z[:, N:]
    if act == GELU:
        return 0.5 * z * (1 + torch.tanh(GC * (z + 0.044715 * z ** 3)))
    return z.clamp(min=0) if act == RELU else z


def grad64(act, z, dy, N):
    if act == SWIGLU:
        g, u = z[:, :N], z[:, N:]
        s = torch.sigmoid(g)
        return torch.cat([dy * u * s * (1 + g * (1 - s)), dy * g * s], 1)
    if act == GELU:
        t = torch.tanh(GC * (z + 0.044715 * z ** 3))
        return dy * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * GC * (1 + 3 * 0.044715 * z * z))
    return dy * (z > 0) if act == RELU else dy


def acc_err(K, S):
    return (K / 16 + 32) * 2.0 ** -23 * S


def check_forward(p, d, bias, res, save, y=None, z=None, dev=None, stream=None):
    dev = dev or {k: v.cuda() for k, v in d.items()}
    out = F32 if p.out_dtype == 1 else BF
    y = torch.full((p.M, p.N), 7.0, dtype=out, device="cuda") if y is None else y
    if save and z is None:
        z = torch.full((p.M, p.cols), 7.0, dtype=BF, device="cuda")
    ws = torch.empty(moe.moe_linear_workspace_size(p), dtype=torch.uint8, device="cuda")
    moe.moe_linear_forward(p, dev["x"], dev["W"], dev["bias"] if bias else None,
                           dev["res"] if res else None, y, ws, z=z if save else None, stream=stream)
    assert moe.moe_get_device_status(ws, stream) == 0
    x64, W64 = d["x"].double().cuda(), d["W"].double().cuda()
    W64 = W64.t() if p.w_layout == moe.W_NK else W64
    z64, S = x64 @ W64, x64.abs() @ W64.abs()
    if bias:
        z64, S = z64 + d["bias"].double().cuda(), S + d["bias"].double().cuda().abs()
    ez = acc_err(p.K, S)
    a64 = act64(p.act, z64, p.N)
    if p.act == SWIGLU:
        g, u = z64[:, :p.N], z64[:, p.N:]
        e = (1.1 * u.abs() + 1e-3) * ez[:, :p.N] + (g.abs() + 0.3) * ez[:, p.N:]
    else:
        e = 1.13 * ez
    e = e + 2.0 ** -20 * a64.abs()
    y64 = a64 + d["res"].double().cuda() if res else a64
    tol = e + (half_step(out) + 2.0 ** -23) * (y64.abs() + e) + 1e-30
    err = (y.double() - y64).abs()
    assert (err <= tol).all(), f"y: {(err - tol).max()} over, {(err > tol).sum()} of {err.numel()}"
    if save:
        tz = ez + half_step(BF) * (z64.abs() + ez) + 1e-30
        err = (z.double() - z64).abs()
        assert (err <= tz).all(), f"z: {(err - tz).max()} over"
    return y, z


SHAPES = [(1, 8, 8), (1, 64, 64), (3, 72, 40), (7, 1160, 264), (64, 512, 520), (127, 200, 136), (128, 256, 512),
          (129, 520, 1032), (300, 2056, 64), (1000, 136, 2568)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("act", [SWIGLU, GELU, RELU, IDENT])
def test_forward(M, K, N, act):
    for i, (nk, out, bias, res, save) in enumerate([(False, BF, True, True, True), (True, BF, False, True, False),
                                                    (False, F32, False, False, False), (True, F32, True, True, True)]):
        d = make(M, K, N, act, nk, 10 * M + i)
        p = moe.Linear.make(M, N, K, act=act, w_layout=moe.W_NK if nk else moe.W_KN, out_dtype=out)
        check_forward(p, d, bias, res, save)


PLANS = [(256, 0), (128, 0), (64, 1), (64, 2), (64, 8), (128, 1), (128, 4), (128, 8)]


@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("M,K,N", [(5, 520, 72), (200, 1096, 328), (140, 8, 640)])
def test_every_plan(M, K, N, plan):
    moe.moe_set_linear_plan(*plan)
    for act, nk in ((IDENT, False), (IDENT, True), (SWIGLU, False), (SWIGLU, True), (GELU, False)):
        d = make(M, K, N, act, nk, M + K)
        p = moe.Linear.make(M, N, K, act=act, w_layout=moe.W_NK if nk else moe.W_KN)
        check_forward(p, d, True, True, True)
        check_backward(p, d)


def check_backward(p, d, want=("dx", "dW", "dbias")):
    g = torch.Generator().manual_seed(5)
    out = F32 if p.out_dtype == 1 else BF
    z = torch.randn(p.M, p.cols, generator=g).to(BF)
    dev = {k: v.cuda() for k, v in d.items()}
    nk = p.w_layout == moe.W_NK
    dx = torch.full((p.M, p.K), 7.0, dtype=BF, device="cuda") if "dx" in want else None
    dW = torch.full(tuple(d["W"].shape), 7.0, dtype=BF, device="cuda") if "dW" in want else None
    db = torch.full((p.cols,), 7.0, device="cuda") if "dbias" in want else None
    ws = torch.empty(moe.moe_linear_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    moe.moe_linear_backward(p, dev["x"], dev["W"], z.cuda() if p.act != IDENT else None, dev["dy"].to(out), dx, dW,
                            db, ws)
    assert moe.moe_get_device_status(ws) == 0
    x64, W64 = d["x"].double().cuda(), d["W"].double().cuda()
    W64 = W64.t() if nk else W64
    dz = grad64(p.act, z.double().cuda(), d["dy"].to(out).double().cuda(), p.N)
    # dz: the derivative's fast forms (2^-19 of dy and the other factor), then rounded to bf16
    fast = 2.0 ** -19 * (d["dy"].double().cuda().abs() * 2)
    if p.act == SWIGLU:
        zd = z.double().cuda()
        fast = torch.cat([fast * zd[:, p.N:].abs(), fast * zd[:, :p.N].abs()], 1)
    fast = fast if p.act in (SWIGLU, GELU) else 0 * fast
    exact = p.act in (RELU, IDENT) and out == BF
    edz = (0.0 if exact else half_step(BF)) * (dz.abs() + fast) + fast
    for name, got, ref, S, E, K in (("dx", dx, dz @ W64.t(), dz.abs() @ W64.abs().t(), edz @ W64.abs().t(), p.cols),
                                    ("dW", dW, x64.t() @ dz, x64.abs().t() @ dz.abs(), x64.abs().t() @ edz, p.M)):
        if got is None:
            continue
        got = got.double().t() if nk and name == "dW" else got.double()
        tol = E + acc_err(K, S + E) + half_step(BF) * (ref.abs() + E) + 1e-30
        err = (got - ref).abs()
        assert (err <= tol).all(), f"{name}: {(err - tol).max()} over, {(err > tol).sum()} of {err.numel()}"
    if db is not None:
        ref, S = dz.sum(0), dz.abs().sum(0)
        # fp32 sums of M terms in three levels, and the derivative's fast forms
        tol = (p.M + 8) * 2.0 ** -24 * S + fast.sum(0) + 2.0 ** -24 * ref.abs() + 1e-30
        assert ((db.double() - ref).abs() <= tol).all(), "dbias"
    return dx, dW, db


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("act", [SWIGLU, GELU, RELU, IDENT])
def test_backward(M, K, N, act):
    for i, (nk, out) in enumerate([(False, BF), (True, BF), (False, F32), (True, F32)]):
        d = make(M, K, N, act, nk, 20 * M + i, out)
        p = moe.Linear.make(M, N, K, act=act, w_layout=moe.W_NK if nk else moe.W_KN, out_dtype=out)
        check_backward(p, d)


@pytest.mark.parametrize("act", [GELU, IDENT])
def test_backward_of_single_gradients(act):
    p = moe.Linear.make(70, 136, 264, act=act)
    d = make(70, 264, 136, act, False, 3)
    full = check_backward(p, d)
    for name, want in zip(("dx", "dW", "dbias"), full):
        got = [g for g in check_backward(p, d, (name,)) if g is not None]
        assert len(got) == 1 and torch.equal(got[0], want)


def test_gradients_against_differences():
    """Directional derivatives of L = sum(dy * y) in 64 bits against the returned gradients."""
    M, K, N = 24, 64, 40
    for act in (SWIGLU, GELU, IDENT):
        d = make(M, K, N, act, False, 8)
        p = moe.Linear.make(M, N, K, act=act)
        dev = {k: v.cuda() for k, v in d.items()}
        y, z = (torch.empty(M, c, dtype=BF, device="cuda") for c in (N, p.cols))
        ws = torch.empty(moe.moe_linear_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
        moe.moe_linear_forward(p, dev["x"], dev["W"], dev["bias"], None, y, ws, z=z)
        dx, dW, db = torch.empty_like(dev["x"]), torch.empty_like(dev["W"]), torch.empty_like(dev["bias"])
        moe.moe_linear_backward(p, dev["x"], dev["W"], z, dev["dy"], dx, dW, db, ws)

        def loss(x, W, b):
            return (act64(act, x @ W + b, N) * d["dy"].double()).sum()

        a = [d["x"].double(), d["W"].double(), d["bias"].double()]
        g = torch.Generator().manual_seed(1)
        for i, got in enumerate((dx, dW, db)):
            v = torch.randn(a[i].shape, generator=g, dtype=torch.float64)
            h = 1e-5
            up, dn = list(a), list(a)
            up[i], dn[i] = a[i] + h * v, a[i] - h * v
            num = float((loss(*up) - loss(*dn)) / (2 * h))
            mine = float((got.double().cpu() * v).sum())
            # z, dz and the gradient are rounded to bf16: three half steps of every term, added up
            # like independent errors, six deviations
            size = float(((got.double().cpu() * v) ** 2).sum() ** 0.5)
            assert abs(num - mine) <= 6 * 3 * 2.0 ** -8 * size + 1e-6, (act, i, num, mine)


@pytest.mark.parametrize("out", [BF, F32])
def test_strided_rows_leave_the_rest_alone(out):
    M, K, N = 70, 136, 200
    for act, nk in ((GELU, False), (SWIGLU, True)):
        d = make(M, K, N, act, nk, 4)
        p = moe.Linear.make(M, N, K, act=act, w_layout=moe.W_NK if nk else moe.W_KN, out_dtype=out)

        def wide(t, pad, dtype=None):
            buf = torch.full((t.shape[0] + 2, t.shape[1] + pad), 5.0, dtype=dtype or t.dtype, device="cuda")
            buf[1:-1, :t.shape[1]] = t.cuda()
            return buf, buf[1:-1, :t.shape[1]]

        dev = {k: v.cuda() for k, v in d.items()}
        for k, pad in (("x", 8), ("W", 24), ("res", 16)):
            _, dev[k] = wide(d[k], pad)
        ybuf, y = wide(torch.zeros(M, N), 40, out)
        zbuf, z = wide(torch.zeros(M, p.cols), 8, BF)
        check_forward(p, d, True, True, True, y=y, z=z, dev=dev)
        for buf, n in ((ybuf, N), (zbuf, p.cols)):
            assert (buf[0] == 5).all() and (buf[-1] == 5).all() and (buf[:, n:] == 5).all()
        # the gradient from strided operands equals the one from dense ones
        ws = torch.empty(moe.moe_linear_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
        _, dy = wide(d["dy"].to(out), 8, out)
        grads = []
        for a in ((dev["x"], dev["W"], z, dy), tuple(t.contiguous() for t in (dev["x"], dev["W"], z, dy))):
            o = [torch.empty(M, K, dtype=BF, device="cuda"), torch.empty(d["W"].shape, dtype=BF, device="cuda"),
                 torch.empty(p.cols, device="cuda")]
            moe.moe_linear_backward(p, *a, *o, ws)
            grads.append(o)
        assert all(torch.equal(a, b) for a, b in zip(*grads))


def test_residual_in_place_and_no_rows():
    p = moe.Linear.make(40, 72, 64)
    d = make(40, 64, 72, IDENT, False, 6)
    want, _ = check_forward(p, d, True, True, False)
    buf = d["res"].cuda()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    moe.moe_linear_forward(p, d["x"].cuda(), d["W"].cuda(), d["bias"].cuda(), buf, buf, ws)
    assert torch.equal(buf, want)
    p0 = moe.Linear.make(0, 72, 64, act=GELU)
    e = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device="cuda")
    moe.moe_linear_forward(p0, e(0, 64), d["W"].cuda(), None, None, e(0, 72), ws, z=e(0, 72))
    dW, db = torch.ones(64, 72, dtype=BF, device="cuda"), torch.ones(72, device="cuda")
    wsb = torch.empty(moe.moe_linear_backward_workspace_size(p0), dtype=torch.uint8, device="cuda")
    moe.moe_linear_backward(p0, e(0, 64), d["W"].cuda(), e(0, 72), e(0, 72), e(0, 64), dW, db, wsb)
    assert (dW == 0).all() and (db == 0).all() and moe.moe_get_device_status(wsb) == 0


def test_infinite_and_nan_inputs_stay_in_their_rows():
    p = moe.Linear.make(150, 72, 64)
    d = make(150, 64, 72, IDENT, False, 9)
    want, _ = check_forward(p, d, True, True, False)
    d["x"][7, 3], d["x"][149, 0] = float("nan"), float("inf")
    y = torch.empty_like(want)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    moe.moe_linear_forward(p, d["x"].cuda(), d["W"].cuda(), d["bias"].cuda(), d["res"].cuda(), y, ws)
    assert torch.isnan(y[7]).all() and not torch.isfinite(y[149]).any()
    keep = [i for i in range(150) if i not in (7, 149)]
    assert torch.equal(y[keep], want[keep])


def test_same_bits_every_time_and_two_streams_at_once():
    M, K, N = 64, 2048, 512
    d = make(M, K, N, GELU, False, 2)
    p = moe.Linear.make(M, N, K, act=GELU)
    dev = {k: v.cuda() for k, v in d.items()}
    y0, _ = check_forward(p, d, True, True, False)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(y0) for _ in range(20)] for _ in streams]
    wss = [torch.empty(256, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        for st, o, ws in zip(streams, outs, wss):
            moe.moe_linear_forward(p, dev["x"], dev["W"], dev["bias"], dev["res"], o[i], ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(t, y0) for o in outs for t in o)


def test_captured_forward_and_backward():
    M, K, N = 96, 264, 136
    d = make(M, K, N, SWIGLU, False, 12)
    p = moe.Linear.make(M, N, K, act=SWIGLU)
    dev = {k: v.cuda() for k, v in d.items()}
    e = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device="cuda")
    ws = torch.empty(moe.moe_linear_backward_workspace_size(p), dtype=torch.uint8, device="cuda")

    def step(o):
        moe.moe_linear_forward(p, dev["x"], dev["W"], dev["bias"], dev["res"], o[0], ws, z=o[1])
        moe.moe_linear_backward(p, dev["x"], dev["W"], o[1], dev["dy"], o[2], o[3], o[4], ws)

    buffers = lambda: [e(M, N), e(M, 2 * N), e(M, K), e(K, 2 * N), e(2 * N, dt=F32)]
    eager, cap = buffers(), buffers()
    step(eager)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(cap)
    for scale in (1.0, -0.5):
        dev["x"].mul_(scale)
        g.replay()
        step(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, cap))
    assert moe.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("M,K,N,act", [(2048, 1024, 4096, SWIGLU), (4096, 2048, 256, IDENT), (1, 7168, 4096, GELU),
                                       (700, 4096, 1032, RELU)])
def test_larger_sizes(M, K, N, act):
    out = F32 if act == IDENT else BF
    d = make(M, K, N, act, False, 1, out)
    p = moe.Linear.make(M, N, K, act=act, out_dtype=out)
    check_forward(p, d, True, act != IDENT, True)
    check_backward(p, d)


@pytest.mark.parametrize("nk", [False, True])
@pytest.mark.parametrize("M,K,N,act", [(1304, 200, 3592, GELU), (1304, 72, 1800, SWIGLU), (1304, 3592, 136, IDENT),
                                       (72, 1304, 3592, IDENT), (1300, 264, 3712, RELU)])
def test_last_wave_of_tiles(M, K, N, act, nk):
    """More 256-column tiles than SMs, and few in the last wave (165 of them on 148 SMs), whose last
    columns end just behind a tile's first half, or just inside it."""
    moe.moe_set_linear_plan(256, 0)
    d = make(M, K, N, act, nk, 31)
    p = moe.Linear.make(M, N, K, act=act, w_layout=moe.W_NK if nk else moe.W_KN)
    check_forward(p, d, True, True, True)
    check_backward(p, d)


def test_offsets_past_32_bits():
    """Outputs, residual, saved z and gradients of more than 2^31 elements: the last rows equal those of
    a small call."""
    M, K, N, m = 70016, 64, 32768, 128
    g = torch.Generator().manual_seed(3)
    W = (torch.randn(K, N, generator=g) / 8).to(BF).cuda()
    x = torch.zeros(M, K, dtype=BF, device="cuda")
    x[-m:] = torch.randn(m, K, generator=g).to(BF).cuda()
    res = torch.ones(M, N, dtype=BF, device="cuda")
    p, q = moe.Linear.make(M, N, K, act=GELU), moe.Linear.make(m, N, K, act=GELU)
    moe.moe_set_linear_plan(256, 0)
    ws = torch.empty(moe.moe_linear_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    y, z = (torch.empty(M, N, dtype=BF, device="cuda") for _ in range(2))
    moe.moe_linear_forward(p, x, W, None, res, y, ws, z=z)
    ys, zs = (torch.empty(m, N, dtype=BF, device="cuda") for _ in range(2))
    moe.moe_linear_forward(q, x[-m:], W, None, res[-m:], ys, ws, z=zs)
    assert moe.moe_get_device_status(ws) == 0
    assert torch.equal(y[-m:], ys) and torch.equal(z[-m:], zs) and (y[:m] == 1).all()
    dx, dxs = torch.empty_like(x), torch.empty(m, K, dtype=BF, device="cuda")
    moe.moe_linear_backward(p, x, W, z, res, dx, None, None, ws)
    moe.moe_linear_backward(q, x[-m:], W, zs, res[-m:], dxs, None, None, ws)
    assert moe.moe_get_device_status(ws) == 0
    assert torch.equal(dx[-m:], dxs)


def test_gelu_gradient_far_out():
    """The derivative is 0 and 1 where the gate is shut and open, whatever the size of z; a NaN stays
    one. One row: dbias is dz itself, unrounded."""
    far = [6.0, 9.0, 12.0, 30.0, 31.0, 1e4, 1e13, 1e14, 1e18, 2e19, 1e20, 1e30, 1e37, 3e38]
    z = torch.tensor([v for f in far for v in (f, -f)] + [float("nan"), 0.0, 0.5, -0.5], dtype=BF)[None].cuda()
    n = z.shape[1]
    p = moe.Linear.make(1, n, 8, act=GELU)
    ws = torch.empty(moe.moe_linear_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    dy, db = torch.ones(1, n, dtype=BF, device="cuda"), torch.empty(n, device="cuda")
    x, W = torch.ones(1, 8, dtype=BF, device="cuda"), torch.ones(8, n, dtype=BF, device="cuda")
    moe.moe_linear_backward(p, x, W, z, dy, None, None, db, ws)
    nan = torch.isnan(z[0])
    assert torch.equal(torch.isnan(db), nan)
    z64 = z[0].double()
    z64 = torch.where(z64.abs() > 100, z64.sign() * 100, z64)        # 0 or 1 to the last bit from 10 on
    ref = grad64(GELU, z64, torch.ones_like(z64), n)
    assert ((db.double() - ref).abs() <= 2.0 ** -19)[~nan].all()


def test_swiglu_gradient_of_large_values():
    """A shut gate's gradients are 0 although dy times the gate's or up's value would overflow."""
    g = torch.tensor([-1e30, -1e30, -3e38, -3e38, -2e20, 5.0, 200.0], dtype=BF)
    u = torch.tensor([2.0, 1e30, 3.0, 1e38, -1e30, 1e20, -1e20], dtype=BF)
    dy = torch.tensor([1e10, 1e10, 1e30, -1e30, 1e25, 1e10, 1e10], dtype=BF)
    pad = lambda t: torch.cat([t, torch.zeros(1, dtype=BF)])
    g, u, dy = pad(g), pad(u), pad(dy)
    p = moe.Linear.make(1, 8, 8, act=SWIGLU)
    z = torch.cat([g, u])[None].cuda()
    ws = torch.empty(moe.moe_linear_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    db = torch.empty(16, device="cuda")
    x, W = torch.ones(1, 8, dtype=BF, device="cuda"), torch.ones(8, 16, dtype=BF, device="cuda")
    moe.moe_linear_backward(p, x, W, z, dy[None].cuda(), None, None, db, ws)
    ref = grad64(SWIGLU, z.double().cpu(), dy.double()[None], 8)[0]
    # the derivative's fast forms: 2^-19 of dy and the other factor, where the gate is not shut
    d64 = dy.double()
    fast = 2.0 ** -19 * torch.cat([d64 * u.double(), d64 * g.double()]).abs() * (torch.cat([g, g]) > -100)
    assert ((db.double().cpu() - ref).abs() <= fast + 1e-30).all(), db


def test_the_shortest_wait_limit_still_finishes():
    """The dense product's waits have a least limit of their own, so that copies and products in flight
    are always waited for: a limit of one nanosecond changes nothing."""
    for M, K, N, act, plan in ((300, 2056, 264, SWIGLU, (256, 0)), (64, 4096, 520, IDENT, (128, 4))):
        moe.moe_set_linear_plan(*plan)
        d = make(M, K, N, act, False, 3)
        p = moe.Linear.make(M, N, K, act=act)
        prev = moe.moe_set_wait_timeout_ns(1)
        try:
            check_forward(p, d, True, True, True)
            check_backward(p, d)
        finally:
            moe.moe_set_wait_timeout_ns(prev)


FP32_PLANS = [(128, 0), (64, 1), (64, 2), (64, 4), (64, 8), (128, 1), (128, 2), (128, 4), (128, 8)]


@pytest.mark.parametrize("plan", FP32_PLANS)
@pytest.mark.parametrize("M,K,N", [(5, 1032, 72), (200, 1544, 328), (140, 4104, 136)])
def test_every_plan_with_fp32_outputs_and_long_k(M, K, N, plan):
    """fp32 outputs of more than 512 values of k, whose runs of 512 are summed in registers; the last
    run short, some parts of the split without a whole one."""
    moe.moe_set_linear_plan(*plan)
    for act, nk in ((IDENT, False), (IDENT, True), (SWIGLU, False), (SWIGLU, True), (GELU, False)):
        d = make(M, K, N, act, nk, M + K, F32)
        p = moe.Linear.make(M, N, K, act=act, w_layout=moe.W_NK if nk else moe.W_KN, out_dtype=F32)
        check_forward(p, d, True, True, True)


@pytest.mark.parametrize("nk", [False, True])
@pytest.mark.parametrize("M,K,N,act", [(1304, 1544, 4360, IDENT), (1304, 1096, 2056, SWIGLU), (2600, 600, 2056, GELU)])
def test_fp32_outputs_of_several_tiles_a_block(M, K, N, act, nk):
    """More than two tiles a block of the persistent form: its runs and barriers carry on from one tile to
    the next."""
    moe.moe_set_linear_plan(128, 0)
    d = make(M, K, N, act, nk, 77, F32)
    p = moe.Linear.make(M, N, K, act=act, w_layout=moe.W_NK if nk else moe.W_KN, out_dtype=F32)
    check_forward(p, d, True, True, True)


@pytest.mark.parametrize("plan", [(128, 0), (128, 2), (64, 1), (64, 8)])
@pytest.mark.parametrize("M,K,N", [(200, 7168, 264), (130, 16384, 72)])
def test_fp32_sums_of_one_sign(M, K, N, plan):
    """Products of one sign, where truncation adds up. A run of 512 takes 32 steps of 16 products; a step
    loses at most 2^-23 of the accumulator, which grows evenly over the run: at most 16.5 * 2^-23 of the
    run's sum (with the spread of the runs' growth 18), 2.2e-6. The runs are added in registers (and the
    parts of a split): K / 512 + 8 roundings, each 2^-24 of a sum that grows evenly, so half of them. One
    accumulator over all of K loses 2.9e-5 at K = 7168, 7.5e-5 at 16384."""
    moe.moe_set_linear_plan(*plan)
    g = torch.Generator().manual_seed(K)
    x, W = torch.rand(M, K, generator=g).to(BF).cuda(), torch.rand(K, N, generator=g).to(BF).cuda()
    p = moe.Linear.make(M, N, K, out_dtype=F32)
    y, ws = torch.empty(M, N, device="cuda"), torch.empty(256, dtype=torch.uint8, device="cuda")
    moe.moe_linear_forward(p, x, W, None, None, y, ws)
    assert moe.moe_get_device_status(ws) == 0
    ref = x.double() @ W.double()
    tol = 18 * 2.0 ** -23 + (K / 512 + 10) * 2.0 ** -25
    err = ((y.double() - ref) / ref).abs().max()
    assert err <= tol, float(err)
