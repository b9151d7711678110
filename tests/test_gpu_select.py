"""Routing by scores on the GPU against a 64-bit reference of its definition: the selection
exactly, the weights and their gradient within the roundings of 32-bit arithmetic."""
import math

import numpy as np
import pytest
import torch

import mixture_experts_layer_forward_b200 as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24                        # half a step of fp32, relative


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


def clean(l):
    l = l.astype(np.float64).copy()
    l[np.isnan(l)] = -np.inf
    return np.minimum(l, float(np.finfo(np.float32).max))


def scores(s, l):
    live = l > -np.inf
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if s.score == moe.SCORE_SIGMOID:
            v = 1.0 / (1.0 + np.exp(-l))
        else:
            m = l.max(1, keepdims=True)
            e = np.where(live, np.exp(l - m), 0.0)
            v = e / e.sum(1, keepdims=True)
    return np.where(live, v, 0.0), live


def ref_select(s, logits, bias):
    """(idx, w) by the definition, token by token."""
    l = clean(logits)
    sc, live = scores(s, l)
    T, E, G = s.T, s.E, s.n_group
    idx = np.zeros((T, s.top_k), np.int32)
    for t in range(T):
        with np.errstate(invalid="ignore"):
            val = sc[t] + (0.0 if bias is None else bias.astype(np.float64))
        val = np.where(np.isnan(val), -np.inf, val)
        key = l[t] if bias is None else val
        groups = list(range(G))
        if G > 1:
            gv = []
            for g in range(G):
                m = np.arange(g * E // G, (g + 1) * E // G)
                m = m[live[t, m]]
                if s.group_score == moe.GROUP_SUM2:
                    v = np.sort(val[m])[::-1][:2]
                    v = v[:1] if len(v) == 2 and v[1] == -np.inf else v
                    gv.append(v.sum() if len(v) else -np.inf)
                else:
                    gv.append(key[m].max() if len(m) else -np.inf)
            groups = sorted(range(G), key=lambda g: (-gv[g], g))[:s.top_group]
        cand = [e for e in range(E) if e // (E // G) in groups]
        cand.sort(key=lambda e: (0 if live[t, e] else 1, -key[e] if live[t, e] else 0.0, e))
        idx[t] = cand[:s.top_k]
    sel = np.take_along_axis(sc, idx, 1)
    ll = np.take_along_axis(l, idx, 1)
    if s.renorm:      # ratios of the scores, also where they underflow
        on = ll > -np.inf
        if s.score == moe.SCORE_SIGMOID:
            lg = np.where(on, np.minimum(ll, 0) - np.log1p(np.exp(-np.abs(np.where(on, ll, 0)))), -np.inf)
        else:
            lg = ll
        m = lg.max(1, keepdims=True)
        m = np.where(m == -np.inf, 0.0, m)
        sel = np.where(on, np.exp(lg - m), 0.0)
        tot = sel.sum(1, keepdims=True)
        sel = np.divide(sel, tot, out=np.zeros_like(sel), where=tot > 0)
    return idx, sel * s.scale


def weight_tol(s, logits, w):
    """Roundings of a weight: exp of a difference d rounds by (|d| + 4) half steps, numerator and
    denominator, five additions, a quotient and the scale; the sum over all experts (softmax
    without renormalising) uses the fast exponential, (2 + 1.17 |d|) steps each, and 37 additions."""
    l = clean(logits)
    f = np.where(np.abs(l) < 1e30, l, np.nan)
    span = np.nan_to_num(np.nanmax(np.abs(f), 1, keepdims=True)) * 2
    n = 2 * span + 24 if s.renorm or s.score == moe.SCORE_SIGMOID else 4 * span + 100
    return n * U * np.abs(w) + 1e-37 * s.scale


def check(s, logits, bias, dev_logits=None, **kw):
    x = dev_logits if dev_logits is not None else logits.cuda()
    idx = torch.full((s.T, s.top_k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((s.T, s.top_k), -7.0, device="cuda")
    moe.moe_route_select(s, x, None if bias is None else bias.cuda(), idx, w, **kw)
    torch.cuda.synchronize()
    l = logits.float().numpy()
    ri, rw = ref_select(s, l, None if bias is None else bias.numpy())
    gi, gw = idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    assert np.array_equal(gi, ri), np.argwhere(gi != ri)[:4]
    assert np.all(np.abs(gw - rw) <= weight_tol(s, l, rw)), np.abs(gw - rw).max()
    return idx, w


def draw(T, E, seed, dtype=torch.float32, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * std).to(dtype), torch.randn(E, generator=g) * 0.05


CASES = [  # T, E, k, groups, keep
    (1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (3, 8, 2, 1, 1), (33, 10, 3, 5, 2), (65, 64, 8, 1, 1),
    (17, 40, 4, 5, 3), (9, 60, 6, 4, 1), (40, 160, 6, 8, 3), (64, 256, 8, 8, 4), (20, 384, 32, 32, 8),
    (12, 512, 16, 16, 4), (7, 1000, 5, 1, 1), (5, 1024, 32, 32, 1), (130, 32, 32, 1, 1), (11, 33, 1, 3, 3),
]


@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
@pytest.mark.parametrize("T,E,k,G,keep", CASES)
def test_selection_and_weights(T, E, k, G, keep, score):
    n = 0
    for sum2 in (moe.GROUP_MAX, moe.GROUP_SUM2):
        for biased in (False, True):
            for dtype in (torch.float32, torch.bfloat16):
                n += 1
                l, b = draw(T, E, 100 * T + E + n, dtype)
                s = moe.Select.make(T, E, k, score=score, n_group=G, top_group=keep, group_score=sum2,
                                    renorm=n % 3 != 0, scale=2.5 if n % 2 else 1.0)
                check(s, l, b if biased else None)


@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
def test_ties_go_to_the_lower_id(score):
    s = moe.Select.make(8, 64, 6, score=score, n_group=4, top_group=2, group_score=moe.GROUP_SUM2)
    l = torch.zeros(8, 64)
    check(s, l, None)
    check(s, l, torch.zeros(64))
    l[:, 1::2] = 1.0
    check(s, l, torch.zeros(64))
    l[3] = 0.0
    l[3, 40:44] = -0.0
    check(s, l, None)
    # saturated scores are equal in 64 bits too: the id decides
    if score == moe.SCORE_SIGMOID:
        check(s, torch.rand(8, 64) * 20 + 50, torch.zeros(64))


@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
@pytest.mark.parametrize("steps", [1, 4, 64])
def test_keys_closer_than_32_bits_can_tell(score, steps):
    """Score plus bias nearly equal for all experts: only 64 bits order them."""
    g = torch.Generator().manual_seed(steps)
    l = torch.randn(16, 48, generator=g)
    # the bias undoes one token's scores up to a few steps of fp32
    sc, _ = scores(moe.Select.make(16, 48, 8, score=score), l.numpy().astype(np.float64))
    b = torch.from_numpy((0.5 - sc[0]).astype(np.float32)) + torch.randint(-steps, steps + 1, (48,), generator=g) * 2.0 ** -25
    l[1:] = l[0] + torch.randint(-2, 3, (15, 48), generator=g) * 1e-7
    for G, keep, sum2 in ((1, 1, 0), (4, 2, 1), (6, 3, 0)):
        s = moe.Select.make(16, 48, 8, score=score, n_group=G, top_group=keep, group_score=sum2)
        check(s, l, b)


@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_masked_infinite_and_nan_logits(score, renorm):
    l, b = draw(12, 32, 5)
    l[0] = -math.inf                       # a row with nothing left
    l[1, 3:] = -math.inf                   # fewer live experts than k
    l[2, ::2] = float("nan")               # NaN masks as -inf does
    l[3, 5] = math.inf
    l[4, 5] = l[4, 9] = math.inf
    l[5] = torch.finfo(torch.float32).min  # live, the lowest value of the type
    l[6, :31] = -math.inf
    l[7] = -200.0                          # scores underflow, their ratios do not
    l[7, 4] = -199.0
    l[8, 8:16] = -math.inf                 # a whole group
    l[9] = 1e30
    for bias in (None, b):
        for G, keep, sum2 in ((1, 1, 0), (4, 2, 0), (4, 2, 1), (8, 8, 1)):
            s = moe.Select.make(12, 32, 6, score=score, n_group=G, top_group=keep, group_score=sum2,
                                renorm=renorm, scale=1.5)
            _, w = check(s, l, bias)
            assert torch.isfinite(w).all()
            assert (w[0] == 0).all()


def test_biases_without_bounds():
    l, _ = draw(6, 16, 8)
    b = torch.zeros(16)
    b[3], b[7], b[9], b[11] = math.inf, -math.inf, float("nan"), math.inf
    l[2, 3] = -math.inf
    for G, keep, sum2 in ((1, 1, 0), (4, 4, 1), (4, 2, 1)):
        check(moe.Select.make(6, 16, 8, n_group=G, top_group=keep, group_score=sum2), l, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,ld,shift", [(64, 72, 0), (60, 64, 0), (64, 65, 0), (64, 64, 1), (256, 264, 8)])
def test_row_strides_and_alignment(E, ld, shift, dtype):
    l, b = draw(20, E, E + ld, dtype)
    buf = torch.full((20 * ld + shift,), 9.0, dtype=dtype, device="cuda")
    view = buf[shift:].view(20, ld)[:, :E]
    view.copy_(l)
    s = moe.Select.make(20, E, 6)
    idx, w = check(s, l, b, dev_logits=view)
    # the gradient reads the same strided rows
    dw = torch.randn(20, 6, device="cuda")
    d1, d2 = (torch.empty(20, E, dtype=dtype, device="cuda") for _ in range(2))
    moe.moe_route_select_backward(s, view, idx, dw, d1)
    moe.moe_route_select_backward(s, l.cuda(), idx, dw, d2)
    assert torch.equal(d1, d2)


def test_rows_behind_the_last_token_are_left_alone():
    l, b = draw(50, 32, 3)
    s = moe.Select.make(50, 32, 4)
    full_idx, full_w = check(s, l, b)
    for n in (0, 1, 37, 50, 60, -3):
        cnt = torch.tensor([n], dtype=torch.int32, device="cuda")
        idx = torch.full((50, 4), -5, dtype=torch.int32, device="cuda")
        w = torch.full((50, 4), -5.0, device="cuda")
        moe.moe_route_select(s, l.cuda(), b.cuda(), idx, w, n_rows=cnt)
        m = min(max(n, 0), 50)
        assert torch.equal(idx[:m], full_idx[:m]) and torch.equal(w[:m], full_w[:m])
        assert (idx[m:] == -5).all() and (w[m:] == -5).all()
        d = torch.full((50, 32), 7.0, device="cuda")
        moe.moe_route_select_backward(s, l.cuda(), full_idx, torch.ones(50, 4, device="cuda"), d, n_rows=cnt)
        assert (d[m:] == 7).all() and not (d[:m] == 7).any()


def ref_backward(s, logits, idx, dw):
    """(gradient, the same sum over absolute values) through the explicit Jacobian, in 64 bits."""
    l = clean(logits)
    sc, live = scores(s, l)
    out, size = np.zeros_like(l), np.zeros_like(l)
    for t in range(s.T):
        ids = [int(e) for e in idx[t]]
        g = dw[t].astype(np.float64) * s.scale
        on = live[t, ids]
        if s.score == moe.SCORE_SIGMOID:
            x = l[t, ids]
            rest = np.where(on, 1.0 / (1.0 + np.exp(np.where(on, x, 0.0))), 0.0)
            lg = np.where(on, np.minimum(x, 0) - np.log1p(np.exp(-np.abs(np.where(on, x, 0)))), -np.inf)
        else:
            rest = np.ones(len(ids))
            lg = l[t, ids]
        if s.renorm:
            q = np.exp(lg - lg.max()) if on.any() else np.zeros(len(ids))
            q = q / q.sum() if q.sum() > 0 else q
            J = np.diag(q) - np.outer(q, q)
            for i, e in enumerate(ids):
                out[t, e] += rest[i] * (g @ J[:, i])
                size[t, e] += rest[i] * q[i] * (np.abs(g[i]) + np.abs(g) @ q)
        elif s.score == moe.SCORE_SIGMOID:
            for i, e in enumerate(ids):
                out[t, e] += g[i] * sc[t, e] * rest[i]
                size[t, e] += abs(g[i]) * sc[t, e] * rest[i]
        else:
            for i, e in enumerate(ids):
                p = sc[t, e]
                row = -p * sc[t]
                row[e] += p
                out[t] += g[i] * row
                size[t] += abs(g[i]) * np.abs(p * sc[t])
                size[t, e] += abs(g[i]) * p
    return out, size


def check_backward(s, logits, idx, dw):
    d = torch.full((s.T, s.E), 7.0, dtype=logits.dtype, device="cuda")
    moe.moe_route_select_backward(s, logits.cuda(), idx, dw.cuda(), d)
    l = logits.float().numpy()
    ref, size = ref_backward(s, l, idx.cpu().numpy(), dw.numpy())
    f = clean(l)
    span = 2 * np.nan_to_num(np.nanmax(np.where(np.abs(f) < 1e30, np.abs(f), np.nan), 1, keepdims=True))
    # exponentials (|d| + 4 half steps each), sums over k <= 32 or E <= 1024 (37 additions), the
    # products; then the rounding of the result
    tol = (4 * span + 120) * U * size + torch.finfo(logits.dtype).eps / 2 * np.abs(ref) + 1e-37
    err = np.abs(d.float().cpu().numpy().astype(np.float64) - ref)
    assert np.all(err <= tol), (err - tol).max()
    return d


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (50, 10, 3), (33, 64, 8), (9, 1024, 32), (7, 100, 1)])
def test_gradient(T, E, k, renorm, score, dtype):
    l, b = draw(T, E, T + E, dtype)
    if T >= 9 and E > 4:
        l[0] = -math.inf
        l[1, 1:] = -math.inf
        l[2, 0] = float("nan")
        l[3] = -120.0
        l[4, 2] = 60.0
    s = moe.Select.make(T, E, k, score=score, renorm=renorm, scale=1.7)
    idx, _ = check(s, l, b)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(3))
    d = check_backward(s, l, idx, dw)
    if T >= 9 and E > 4:
        assert (d[0] == 0).all()


def test_gradient_against_differences():
    """dL/dl of L = sum g w against central differences of the 64-bit weights, selection fixed."""
    l, _ = draw(4, 12, 2)
    for score in (moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID):
        for renorm in (True, False):
            s = moe.Select.make(4, 12, 3, score=score, renorm=renorm, scale=2.0)
            idx, _ = check(s, l, None)
            dw = torch.randn(4, 3, generator=torch.Generator().manual_seed(1))
            d = torch.empty(4, 12, device="cuda")
            moe.moe_route_select_backward(s, l.cuda(), idx, dw.cuda(), d)
            ids = idx.cpu().numpy()

            def loss(x):
                sc, _ = scores(s, x)
                sel = np.take_along_axis(sc, ids, 1)
                if renorm:
                    sel = sel / sel.sum(1, keepdims=True)
                return (s.scale * sel * dw.numpy()).sum(1)

            x = l.numpy().astype(np.float64)
            h = 1e-4
            for e in range(12):
                up, dn = x.copy(), x.copy()
                up[:, e] += h
                dn[:, e] -= h
                num = (loss(up) - loss(dn)) / (2 * h)
                # the differences' own error is of the order h^2 times a third derivative of order 10
                assert np.allclose(d[:, e].cpu().numpy(), num, rtol=0, atol=1e-6 + 10 * h * h)


def test_gradient_with_ids_given_twice_or_out_of_range():
    l, _ = draw(6, 20, 4)
    idx = torch.tensor([[1, 1, 3], [-1, 2, 19], [20, 5, 5], [7, 7, 7], [0, 1, 2], [1 << 30, -5, 4]],
                       dtype=torch.int32)
    dw = torch.randn(6, 3, generator=torch.Generator().manual_seed(9))
    s = moe.Select.make(6, 20, 3, score=moe.SCORE_SIGMOID, renorm=False)
    d = torch.empty(6, 20, device="cuda")
    moe.moe_route_select_backward(s, l.cuda(), idx.cuda(), dw.cuda(), d)
    sc, _ = scores(s, l.numpy().astype(np.float64))
    ref = np.zeros((6, 20))
    for t in range(6):
        for j in range(3):
            e = int(idx[t, j])
            if 0 <= e < 20:
                ref[t, e] += float(dw[t, j]) * sc[t, e] * (1 - sc[t, e])
    assert np.allclose(d.cpu().numpy(), ref, rtol=40 * U, atol=40 * U)


def test_other_stream_and_captured_call():
    l, b = draw(300, 256, 6)
    s = moe.Select.make(300, 256, 8, n_group=8, top_group=4, group_score=moe.GROUP_SUM2, scale=2.5)
    want_idx, want_w = check(s, l, b)
    x, bias = l.cuda(), b.cuda()
    idx, w = torch.empty_like(want_idx), torch.empty_like(want_w)
    d = torch.empty(300, 256, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        moe.moe_route_select(s, x, bias, idx, w)
        moe.moe_route_select_backward(s, x, idx, w, d)
    for seed in (6, 7):
        l2, _ = draw(300, 256, seed)
        x.copy_(l2)
        g.replay()
        torch.cuda.synchronize()
        ref_i, _ = ref_select(s, l2.numpy(), b.numpy())
        assert np.array_equal(idx.cpu().numpy(), ref_i)
        check_backward(s, l2, idx, w.cpu())
    idx.zero_()
    moe.moe_route_select(s, l.cuda(), bias, idx, w, stream=st)
    st.synchronize()
    assert torch.equal(idx, want_idx) and torch.equal(w, want_w)


def test_many_rows():
    """More rows than one wave of blocks, both load widths, against the reference on a sample."""
    for dtype, E in ((torch.float32, 256), (torch.bfloat16, 62)):
        l, b = draw(20001, E, 11, dtype)
        s = moe.Select.make(20001, E, 8)
        idx = torch.empty(20001, 8, dtype=torch.int32, device="cuda")
        w = torch.empty(20001, 8, device="cuda")
        moe.moe_route_select(s, l.cuda(), b.cuda(), idx, w)
        rows = torch.arange(0, 20001, 97)
        sub = moe.Select.make(len(rows), E, 8)
        ri, rw = ref_select(sub, l[rows].float().numpy(), b.numpy())
        assert np.array_equal(idx[rows].cpu().numpy(), ri)
        assert np.all(np.abs(w[rows].cpu().numpy() - rw) <= weight_tol(sub, l[rows].float().numpy(), rw))


@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
@pytest.mark.parametrize("E,k,G,keep", [(256, 8, 8, 4), (256, 8, 4, 2), (128, 5, 8, 3), (100, 8, 1, 1), (64, 1, 8, 1),
                                        (64, 8, 2, 1), (31, 7, 1, 1), (10, 3, 5, 2), (8, 8, 1, 1), (5, 2, 1, 1)])
def test_large_batches(E, k, G, keep, score):
    """Batches that put several tokens on a warp: the rows of a small batch (random, tied, nearly
    tied, masked, infinite) many times over, in another order, against the small batch's reference."""
    U0, T = 59, 8203
    for i, (dtype, biased, sum2, renorm) in enumerate([(torch.float32, True, 1, True), (torch.float32, False, 1, False),
                                                       (torch.bfloat16, False, 0, True), (torch.bfloat16, True, 0, False),
                                                       (torch.float32, False, 0, True)]):
        l, b = draw(U0, E, 7 * E + i, dtype)
        l[0] = -math.inf
        l[1, 1:] = -math.inf
        l[2, ::2] = float("nan")
        l[3] = 0.25
        l[4, E // 2:] = l[4, 0]
        l[5, 1] = math.inf
        l[6] = torch.finfo(dtype).min
        l[7, E // 2] = 30000.0
        l[8:12] = (l[8:12].float() * 1e-3).to(dtype)      # nearly tied
        small = moe.Select.make(U0, E, k, score=score, n_group=G, top_group=keep, group_score=sum2, renorm=renorm)
        big = moe.Select.make(T, E, k, score=score, n_group=G, top_group=keep, group_score=sum2, renorm=renorm)
        bias = b if biased else None
        ri, rw = ref_select(small, l.float().numpy(), b.numpy() if biased else None)
        tol = weight_tol(small, l.float().numpy(), rw)
        at = torch.randperm(T, generator=torch.Generator().manual_seed(i)) % U0
        idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
        w = torch.full((T, k), -7.0, device="cuda")
        moe.moe_route_select(big, l[at].cuda(), None if bias is None else bias.cuda(), idx, w)
        gi, gw = idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)
        a = at.numpy()
        assert np.array_equal(gi, ri[a]), (i, np.argwhere(gi != ri[a])[:4])
        assert np.all(np.abs(gw - rw[a]) <= tol[a])


def test_offsets_past_32_bits():
    """More than 2^32 logits: the last rows are the ones that a small call gives."""
    T, E, k = (1 << 22) + 3, 1024, 4
    g = torch.Generator().manual_seed(2)
    tail = torch.randn(64, E, generator=g).to(torch.bfloat16).cuda()
    logits = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    logits[:, 5] = 1.0
    logits[-64:] = tail
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_route_select(moe.Select.make(T, E, k, score=moe.SCORE_SOFTMAX), logits, None, idx, w)
    si, sw = torch.empty(64, k, dtype=torch.int32, device="cuda"), torch.empty(64, k, device="cuda")
    s = moe.Select.make(64, E, k, score=moe.SCORE_SOFTMAX)
    moe.moe_route_select(s, tail, None, si, sw)
    assert torch.equal(idx[-64:], si) and torch.equal(w[-64:], sw)
    assert (idx[:-64] == torch.tensor([5, 0, 1, 2], device="cuda")).all()
    d, sd = torch.empty_like(logits), torch.empty_like(tail)
    moe.moe_route_select_backward(moe.Select.make(T, E, k, score=moe.SCORE_SOFTMAX), logits, idx, w, d)
    moe.moe_route_select_backward(s, tail, si, sw, sd)
    assert torch.equal(d[-64:], sd)


def test_the_largest_row_count():
    """T = 2^31 - 1 with 5 rows in use: the rows behind them are not read or written, so the buffers
    hold those 5 rows."""
    lib, T, n = moe._native.library(), 2**31 - 1, 5
    l, b = draw(n, 16, 21)
    small, s = moe.Select.make(n, 16, 3), moe.Select.make(T, 16, 3)
    ref_idx, ref_w = check(small, l, b)
    cnt = torch.tensor([n], dtype=torch.int32, device="cuda")
    lc, bc, dw = l.cuda(), b.cuda(), torch.arange(15.0, device="cuda").reshape(n, 3)
    idx, w = torch.empty(n, 3, dtype=torch.int32, device="cuda"), torch.empty(n, 3, device="cuda")
    d, ref_d = torch.full((n, 16), 7.0, device="cuda"), torch.empty(n, 16, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert lib.moe_route_select(s, lc.data_ptr(), bc.data_ptr(), idx.data_ptr(), w.data_ptr(), cnt.data_ptr(), st) == 0
    assert lib.moe_route_select_backward(s, lc.data_ptr(), idx.data_ptr(), dw.data_ptr(), d.data_ptr(),
                                         cnt.data_ptr(), st) == 0
    moe.moe_route_select_backward(small, lc, ref_idx, dw, ref_d)
    assert torch.equal(idx, ref_idx) and torch.equal(w, ref_w) and torch.equal(d, ref_d)


def check_rows(rows, E, k, bias, seed=0, **kw):
    """The rows as a small batch, and many times over, in another order, in a batch that puts several
    tokens on a warp: both against the reference."""
    n, T = len(rows), 8203
    check(moe.Select.make(n, E, k, **kw), rows, bias)
    small, big = moe.Select.make(n, E, k, **kw), moe.Select.make(T, E, k, **kw)
    l = rows.float().numpy()
    ri, rw = ref_select(small, l, None if bias is None else bias.numpy())
    at = torch.randperm(T, generator=torch.Generator().manual_seed(seed)) % n
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    moe.moe_route_select(big, rows[at].cuda(), None if bias is None else bias.cuda(), idx, w)
    gi, gw, a = idx.cpu().numpy(), w.cpu().numpy().astype(np.float64), at.numpy()
    assert np.array_equal(gi, ri[a]), np.argwhere(gi != ri[a])[:4]
    assert np.all(np.abs(gw - rw[a]) <= weight_tol(small, l, rw)[a])


LOW = -3.3e38    # finite in bf16 and fp32, and below any key that 32 bits carry through a sum
EDGE_SHAPES = [(8, 1, 1, 1), (8, 2, 2, 1), (60, 2, 5, 2), (64, 3, 1, 1), (64, 8, 8, 3), (256, 8, 8, 4),
               (400, 6, 8, 2)]


@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k,G,keep", EDGE_SHAPES)
def test_live_logits_of_the_lowest_value_with_a_bias(E, k, G, keep, dtype, score):
    """Only -inf and NaN mask: an expert at the type's lowest finite value has score 0 and is selected
    where its bias wins."""
    g = torch.Generator().manual_seed(E + k)
    l, b = draw(48, E, E, dtype)
    b[torch.rand(E, generator=g) < 0.3] = 1.5        # larger than any other key where the score is small
    for v, share in ((torch.finfo(dtype).min, 0.3), (LOW, 0.1), (-math.inf, 0.1)):
        l[torch.rand(48, E, generator=g) < share] = v
    l[0] = l[0].clamp(min=-4)
    l[0, 0], b[0] = torch.finfo(dtype).min, 1.5
    for sum2 in (moe.GROUP_MAX, moe.GROUP_SUM2):
        check_rows(l, E, k, b, score=score, n_group=G, top_group=keep, group_score=sum2)


@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
@pytest.mark.parametrize("k", [1, 3])
@pytest.mark.parametrize("E,G,keep", [(8, 4, 2), (8, 2, 1), (60, 5, 2), (64, 8, 3), (256, 8, 4), (400, 8, 2)])
def test_finite_biases_of_the_lowest_value_in_group_sums(E, G, keep, k, score):
    """A finite bias of the lowest value takes its expert's group down with it where the expert is one
    of the group's two largest; -inf leaves the expert out of the sum."""
    g = torch.Generator().manual_seed(E + k)
    l, _ = draw(48, E, E)
    size = E // G
    for least in (torch.finfo(torch.float32).min, LOW, -1e38):
        b = torch.randn(E, generator=g) * 0.05
        for grp in range(0, G, 2):                   # all but one expert of every second group
            b[grp * size + 1:(grp + 1) * size] = least
        b[G // 2 * size] = -math.inf
        check_rows(l, E, k, b, score=score, n_group=G, top_group=keep, group_score=moe.GROUP_SUM2)
        b[-1] = -least                               # and a largest one
        check_rows(l, E, k, b, score=score, n_group=G, top_group=keep, group_score=moe.GROUP_SUM2)


@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,G,keep", [(8, 4, 2), (60, 5, 3), (64, 8, 4), (256, 8, 5), (400, 8, 3)])
def test_groups_whose_scores_are_zero(E, G, keep, dtype, score):
    """Without a bias: a live group whose scores are 0 in 64 bits (logits of -1000 or the lowest value)
    equals another one, and comes before a masked one."""
    g = torch.Generator().manual_seed(E)
    l, _ = draw(48, E, E, dtype)
    kinds = torch.tensor([0.0, -1000.0, torch.finfo(dtype).min, LOW, -math.inf])
    for t in range(48):
        pick = torch.randint(0, 5, (G,), generator=g)
        pick[t % G] = 0
        base = kinds[pick].repeat_interleave(E // G)
        l[t] = torch.where(base == 0, l[t].float(), base).to(dtype)
    for k in (1, 4):
        check_rows(l, E, k, None, score=score, n_group=G, top_group=keep, group_score=moe.GROUP_SUM2)


@pytest.mark.parametrize("E,G,keep", [(8, 2, 1), (48, 6, 3), (60, 5, 2), (64, 8, 3), (256, 8, 4), (400, 8, 2)])
def test_group_sums_of_logits_whose_steps_are_large(E, G, keep):
    """Softmax without a bias: logits of 1e9 and 1e30, equal in several groups. What a key loses to its
    place in the lane is then more than an exponential can carry."""
    g = torch.Generator().manual_seed(E)
    l = torch.randn(48, E, generator=g)
    for t in range(48):
        top = (1e30, 1.0000001e30, 1e9, 1.00000006e9, 3e7)[t % 5]
        at = torch.randperm(G, generator=g)[:1 + t % G] * (E // G) + torch.randint(0, E // G, (1 + t % G,), generator=g)
        l[t, at] = top
    for k in (1, 2):
        check_rows(l, E, k, None, score=moe.SCORE_SOFTMAX, n_group=G, top_group=keep, group_score=moe.GROUP_SUM2)


@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
@pytest.mark.parametrize("E,G,keep", [(8, 4, 1), (60, 5, 2), (64, 8, 3), (256, 8, 4), (400, 8, 2)])
def test_group_sums_of_opposite_biases(E, G, keep, score):
    """The two largest keys of a group may cancel: its value is then small and as exact as 64 bits make
    it, not as 32 bits make the keys."""
    g = torch.Generator().manual_seed(E)
    size = E // G
    l = torch.randn(64, E, generator=g)
    live = torch.zeros(E, dtype=torch.bool)
    b = torch.zeros(E)
    for grp in range(G):                             # two live experts a group, biases +v and -v
        v = float(10 ** (2 + 4 * torch.rand(1, generator=g)))
        live[grp * size] = live[grp * size + size - 1] = True
        b[grp * size], b[grp * size + size - 1] = v, -v
    l[:, ~live] = -math.inf
    for k in (1, 2):
        check_rows(l, E, k, b, score=score, n_group=G, top_group=keep, group_score=moe.GROUP_SUM2)


@pytest.mark.parametrize("score", [moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID])
@pytest.mark.parametrize("E,G,keep", [(8, 4, 2), (16, 4, 2), (60, 5, 3), (64, 8, 4), (256, 8, 4), (400, 8, 4)])
def test_group_sums_beyond_32_bits(E, G, keep, score):
    """The sum of two finite keys may be larger than a float, or small again: 64 bits order the groups,
    also against a group with nothing left."""
    g = torch.Generator().manual_seed(E)
    size = E // G
    kinds = torch.tensor([1.2e38, 2e38, 2.8e38, -1.2e38, -2e38, -2.5e38, -2.8e38, -3.2e38, 0.25, 0.0])
    for it in range(12):
        l = torch.full((24, E), -math.inf)
        b = kinds[torch.randint(3 if it % 3 else 0, 10, (E,), generator=g)]
        for t in range(24):                          # one to three live experts a group, or none
            for grp in range(G):
                at = grp * size + torch.randperm(size, generator=g)[:int(torch.randint(0, 4, (1,), generator=g))]
                l[t, at] = torch.randn(len(at), generator=g)
            l[t, t % E] = 0.5
        check_rows(l, E, 1 + it % 2, b, score=score, n_group=G, top_group=keep, group_score=moe.GROUP_SUM2)
