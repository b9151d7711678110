"""The operators together, as a layer with grouped sigmoid routing uses them: router logits by the
dense product, routing by scores, the layer with that routing, dropout and the residual; and the
whole way back. Also the layer with a supplied routing on its own."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_forward_b200 as moe
from mixture_experts_layer_forward_b200 import synth

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


def empty(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def zeros(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("T,H,F,E,k,gate", [
    (600, 256, 256, 8, 2, moe.GATE_SOFTMAX_TOPK),     # the persistent launch
    (300, 128, 128, 64, 4, moe.GATE_SELECT_BIAS),     # separate launches
    (5, 256, 128, 16, 3, moe.GATE_SOFTMAX_TOPK),      # a decode batch
])
def test_forward_routed_equals_forward(T, H, F, E, k, gate):
    cfg = synth.LayerConfig("routed", T=T, H=H, F=F, E=E, k=k, gate=gate, zipf_s=0.5)
    inp = synth.make_inputs(cfg, seed=3, device="cuda")
    p = moe.Problem.from_config(cfg)
    ws = zeros(moe.moe_workspace_size(p))
    idx, w, a, b = empty(T, k, dtype=I32), empty(T, k, dtype=F32), empty(T, H), empty(T, H)
    moe.moe_forward(p, inp["x"], inp["Wg"], inp["bias"], inp["W1"], inp["W2"], a, ws, idx, w)
    moe.moe_forward_routed(p, inp["x"], idx, w, inp["W1"], inp["W2"], b, ws)
    assert moe.moe_get_device_status(ws) == 0
    assert torch.equal(a, b)
    # with a shared expert
    W1s, W2s, wsg = synth.make_shared_weights(H, 128, device="cuda")
    ws = zeros(moe.moe_workspace_size_shared(p, 128))
    moe.moe_forward_shared(p, inp["x"], inp["Wg"], inp["bias"], inp["W1"], inp["W2"], W1s, W2s, wsg, a, ws)
    moe.moe_forward_routed(p, inp["x"], idx, w, inp["W1"], inp["W2"], b, ws, shared=(W1s, W2s, wsg))
    assert moe.moe_get_device_status(ws) == 0
    assert torch.equal(a, b)


def test_backward_routed_equals_backward():
    """The experts' gradients equal moe_backward's bit for bit, and dtopk_w taken through the
    softmax gives its router gradients."""
    cfg = synth.LayerConfig("routed", T=500, H=256, F=128, E=16, k=4)
    inp = synth.make_inputs(cfg, seed=4, device="cuda")
    p = moe.Problem.from_config(cfg)
    T, H, F, E, k = 500, 256, 128, 16, 4
    dy = torch.randn(T, H, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(BF)
    ws = zeros(moe.moe_backward_workspace_size(p))
    g = [[empty(T, H), empty(E, H, 2 * F), empty(E, F, H)] for _ in range(2)]
    dWg, db = empty(H, E, dtype=F32), empty(E, dtype=F32)
    moe.moe_backward(p, inp["x"], inp["Wg"], None, inp["W1"], inp["W2"], dy, g[0][0], dWg, db, g[0][1], g[0][2], ws)
    idx, w, dw = empty(T, k, dtype=I32), empty(T, k, dtype=F32), empty(T, k, dtype=F32)
    moe.moe_route(p, inp["x"], inp["Wg"], None, idx, w, ws)
    moe.moe_backward_routed(p, inp["x"], idx, w, inp["W1"], inp["W2"], dy, g[1][0], dw, g[1][1], g[1][2], ws)
    assert moe.moe_get_device_status(ws) == 0
    assert torch.equal(g[0][1], g[1][1]) and torch.equal(g[0][2], g[1][2])
    logits = inp["x"].float() @ inp["Wg"].float()
    s = moe.Select.make(T, E, k, score=moe.SCORE_SOFTMAX)
    dl = empty(T, E, dtype=F32)
    moe.moe_route_select_backward(s, logits, idx, dw, dl)
    ref = inp["x"].double().t() @ dl.double()
    assert float((ref - dWg).abs().max()) <= 1e-4 * float(ref.abs().max())   # logits in another order of sums
    dx = g[1][0].double() + dl.double() @ inp["Wg"].double().t()
    # both round once more or less to bf16: two half steps of the larger value
    assert ((dx - g[0][0].double()).abs() <= 2 * 2.0 ** -8 * (g[1][0].double().abs() + dx.abs()) + 1e-6).all()


@pytest.mark.parametrize("T", [300, 5])
def test_routed_layer_reports_bad_ids(T):
    p = moe.Problem.make(T, 128, 128, 16, 2)
    cfg = synth.LayerConfig("bad", T=T, H=128, F=128, E=16, k=2)
    inp = synth.make_inputs(cfg, seed=1, device="cuda")
    idx = torch.stack([torch.randperm(16)[:2] for _ in range(T)]).to(I32).cuda()
    w = torch.rand(T, 2, device="cuda")
    ws = zeros(moe.moe_backward_workspace_size(p))
    ok, out, dx = empty(T, 128), empty(T, 128), empty(T, 128)
    moe.moe_forward_routed(p, inp["x"], idx, w, inp["W1"], inp["W2"], ok, ws)
    assert moe.moe_get_device_status(ws) == 0
    idx[1, 0], idx[T - 1] = -1, torch.tensor([16, 1 << 30], device="cuda")
    moe.moe_forward_routed(p, inp["x"], idx, w, inp["W1"], inp["W2"], out, ws)
    assert moe.moe_get_device_status(ws) == -6
    keep = [t for t in range(T) if t not in (1, T - 1)]
    assert torch.equal(out[keep], ok[keep]) and (out[T - 1] == 0).all()
    dw, dW1, dW2 = empty(T, 2, dtype=F32), torch.empty_like(inp["W1"]), torch.empty_like(inp["W2"])
    moe.moe_backward_routed(p, inp["x"], idx, w, inp["W1"], inp["W2"], ok, dx, dw, dW1, dW2, ws)
    assert moe.moe_get_device_status(ws) == -6
    assert (dw[T - 1] == 0).all() and float(dw[1, 0]) == 0 and (dx[T - 1] == 0).all()
    assert torch.isfinite(dW1.float()).all() and torch.isfinite(dx.float()).all()


@pytest.mark.parametrize("T,E", [(300, 16), (5, 16), (700, 8)])
def test_routed_layer_reports_an_expert_given_twice(T, E):
    """The call reports it and leaves the other tokens' rows as they should be."""
    cfg = synth.LayerConfig("twice", T=T, H=128, F=128, E=E, k=2)
    inp = synth.make_inputs(cfg, seed=2, device="cuda")
    p = moe.Problem.from_config(cfg)
    idx = torch.stack([torch.randperm(E)[:2] for _ in range(T)]).to(I32).cuda()
    w = torch.rand(T, 2, device="cuda")
    ws = zeros(moe.moe_backward_workspace_size(p))
    ok, out, dx = empty(T, 128), empty(T, 128), empty(T, 128)
    dw, dW1, dW2 = empty(T, 2, dtype=F32), torch.empty_like(inp["W1"]), torch.empty_like(inp["W2"])
    moe.moe_forward_routed(p, inp["x"], idx, w, inp["W1"], inp["W2"], ok, ws)
    idx[2, 1] = idx[2, 0]
    moe.moe_forward_routed(p, inp["x"], idx, w, inp["W1"], inp["W2"], out, ws)
    assert moe.moe_get_device_status(ws) == -6
    keep = [t for t in range(T) if t != 2]
    assert torch.equal(out[keep], ok[keep])
    moe.moe_backward_routed(p, inp["x"], idx, w, inp["W1"], inp["W2"], ok, dx, dw, dW1, dW2, ws)
    assert moe.moe_get_device_status(ws) == -6
    assert torch.isfinite(dx[keep].float()).all()


def test_no_tokens():
    p = moe.Problem.make(0, 128, 128, 16, 2)
    W1, W2 = empty(16, 128, 256), empty(16, 128, 128)
    ws = zeros(moe.moe_backward_workspace_size(p))
    e = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device="cuda")
    moe.moe_forward_routed(p, e(0, 128), e(0, 2, dt=I32), e(0, 2, dt=F32), W1, W2, e(0, 128), ws)
    dW1, dW2 = torch.ones_like(W1), torch.ones_like(W2)
    moe.moe_backward_routed(p, e(0, 128), e(0, 2, dt=I32), e(0, 2, dt=F32), W1, W2, e(0, 128), e(0, 128),
                            e(0, 2, dt=F32), dW1, dW2, ws)
    assert moe.moe_get_device_status(ws) == 0
    assert (dW1 == 0).all() and (dW2 == 0).all()


def test_block_forward_and_backward():
    """x -> logits -> routing -> experts -> dropout + residual, and every gradient, against 64-bit
    autograd of the same formulas with the selection and the mask that the operators used. Every
    intermediate is bf16 with fp32 sums, as in the layer's backward: 2% of a tensor's largest
    magnitude plus 3% of the element's own."""
    T, H, F, E, k, prob = 260, 256, 128, 32, 4, 0.2
    cfg = synth.LayerConfig("block", T=T, H=H, F=F, E=E, k=k)
    inp = synth.make_inputs(cfg, seed=9, device="cuda")
    x, Wg, W1, W2 = (inp[n] for n in ("x", "Wg", "W1", "W2"))
    g = torch.Generator("cuda").manual_seed(2)
    dout = torch.randn(T, H, device="cuda", generator=g).to(BF)
    bias = 0.02 * torch.randn(E, device="cuda", generator=g)
    rng = torch.tensor([11, 100], dtype=torch.int64, device="cuda")
    lin = moe.Linear.make(T, E, H, out_dtype=F32)
    sel = moe.Select.make(T, E, k, n_group=4, top_group=2, group_score=moe.GROUP_SUM2, scale=2.0)
    p = moe.Problem.from_config(cfg)
    lws, ws = zeros(moe.moe_linear_backward_workspace_size(lin)), zeros(moe.moe_backward_workspace_size(p))
    logits, idx, w = empty(T, E, dtype=F32), empty(T, k, dtype=I32), empty(T, k, dtype=F32)
    y, out, dy, dx, dxr = (empty(T, H) for _ in range(5))
    dw, dl = empty(T, k, dtype=F32), empty(T, E, dtype=F32)
    dW1, dW2, dWg = torch.empty_like(W1), torch.empty_like(W2), torch.empty_like(Wg)

    def step():
        moe.moe_linear_forward(lin, x, Wg, None, None, logits, lws)
        moe.moe_route_select(sel, logits, bias, idx, w)
        moe.moe_forward_routed(p, x, idx, w, W1, W2, y, ws)
        moe.moe_dropout_add(y, x, out, prob, rng)
        moe.moe_dropout_add_backward(dout, dy, prob, rng)
        moe.moe_backward_routed(p, x, idx, w, W1, W2, dy, dx, dw, dW1, dW2, ws)
        moe.moe_route_select_backward(sel, logits, idx, dw, dl)
        moe.moe_linear_backward(lin, x, Wg, None, dl, dxr, dWg, None, lws)

    step()
    assert moe.moe_get_device_status(ws) == 0 and moe.moe_get_device_status(lws) == 0
    mask = empty(T, H, dtype=F32)
    moe.moe_dropout_add(torch.ones(T, H, device="cuda"), None, mask, prob, rng)   # 0 or the scale
    x64, Wg64, W164, W264 = (t.double().requires_grad_() for t in (x, Wg, W1, W2))
    s = torch.sigmoid(x64 @ Wg64).gather(1, idx.long())
    w64 = 2.0 * s / s.sum(1, keepdim=True)
    o64 = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        z = x64[t] @ W164[e]
        h = torch.nn.functional.silu(z[:, :F]) * z[:, F:]
        o64 = o64.index_add(0, t, w64[t, j, None] * (h @ W264[e]))
    r64 = o64 * mask.double() + x64
    r64.backward(dout.double())

    def close(got, ref, what):
        scale = float(ref.abs().max())
        err = (got.double() - ref).abs()
        assert (err <= 2e-2 * scale + 3e-2 * ref.abs()).all(), (what, float(err.max()), scale)

    assert float((w.double() - w64.detach()).abs().max()) <= 1e-5
    close(out, r64.detach(), "out")
    close(dx.double() + dxr.double() + dout.double(), x64.grad, "dx")
    for got, ref, name in ((dWg, Wg64, "dWg"), (dW1, W164, "dW1"), (dW2, W264, "dW2")):
        close(got, ref.grad, name)
    # the same step captured: equal bits
    first = [t.clone() for t in (out, dx, dxr, dWg, dW1, dW2)]
    cg = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(cg):
        step()
    for t in (out, dx, dxr, dWg, dW1, dW2):
        t.zero_()
    cg.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (out, dx, dxr, dWg, dW1, dW2)))


@pytest.mark.parametrize("T", [300, 40])
@pytest.mark.parametrize("k", [16, 17, 20, 32])
def test_routed_layer_reports_an_expert_given_twice_among_many(T, k):
    """However many experts a token has."""
    cfg = synth.LayerConfig("many", T=T, H=128, F=128, E=40, k=k)
    inp = synth.make_inputs(cfg, seed=5, device="cuda")
    p = moe.Problem.from_config(cfg)
    g = torch.Generator().manual_seed(k)
    idx = torch.stack([torch.randperm(40, generator=g)[:k] for _ in range(T)]).to(I32).cuda()
    w = torch.rand(T, k, device="cuda")
    ws = zeros(moe.moe_backward_workspace_size(p))
    out, dx = empty(T, 128), empty(T, 128)
    dw, dW1, dW2 = empty(T, k, dtype=F32), torch.empty_like(inp["W1"]), torch.empty_like(inp["W2"])
    for want in (0, -6):
        moe.moe_forward_routed(p, inp["x"], idx, w, inp["W1"], inp["W2"], out, ws)
        assert moe.moe_get_device_status(ws) == want
        moe.moe_backward_routed(p, inp["x"], idx, w, inp["W1"], inp["W2"], out, dx, dw, dW1, dW2, ws)
        assert moe.moe_get_device_status(ws) == want
        idx[T - 3, k - 1] = idx[T - 3, 2]


def test_router_of_a_number_of_experts_that_the_product_refuses():
    """60 experts: the product makes 64 columns of logits, routing reads the first 60 of each row, and the
    gradient's last 4 columns are zeros."""
    T, H, E, k = 70, 128, 60, 4
    g = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(T, H, device="cuda", generator=g).to(BF)
    Wg = torch.zeros(H, 64, dtype=BF, device="cuda")
    Wg[:, :E] = torch.randn(H, E, device="cuda", generator=g).to(BF) * H ** -0.5
    with pytest.raises(moe.MoeError):
        moe.moe_linear_forward(moe.Linear.make(T, E, H, out_dtype=F32), x, Wg[:, :E].contiguous(), None, None,
                               empty(T, E, dtype=F32), zeros(256))
    lin, sel = moe.Linear.make(T, 64, H, out_dtype=F32), moe.Select.make(T, E, k)
    ws = zeros(moe.moe_linear_backward_workspace_size(lin))
    logits, idx, w = empty(T, 64, dtype=F32), empty(T, k, dtype=I32), empty(T, k, dtype=F32)
    moe.moe_linear_forward(lin, x, Wg, None, None, logits, ws)
    moe.moe_route_select(sel, logits[:, :E], None, idx, w)
    own_i, own_w = empty(T, k, dtype=I32), empty(T, k, dtype=F32)
    moe.moe_route_select(sel, logits[:, :E].contiguous(), None, own_i, own_w)
    assert torch.equal(idx, own_i) and torch.equal(w, own_w) and int(idx.max()) < E
    dl, dW, dx = empty(T, E, dtype=F32), empty(H, 64), empty(T, H)
    moe.moe_route_select_backward(sel, logits[:, :E], idx, torch.ones_like(w).cumsum(1), dl)
    dy = torch.nn.functional.pad(dl, (0, 64 - E))
    moe.moe_linear_backward(lin, x, Wg, None, dy, dx, dW, None, ws)
    assert moe.moe_get_device_status(ws) == 0
    assert (dW[:, E:] == 0).all() and not (dW[:, :E] == 0).all()
