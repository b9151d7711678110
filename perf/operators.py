"""Workloads of the operators around the MoE layer: routing by scores, the dense product with a
fused epilogue, and dropout with the residual, each with its gradient.

``own`` picks the side: False computes the plain form (elementary torch operations in 32 bits,
64 where a selection is near a border), True calls the library."""
import math

import numpy as np
import torch

own = False

SWIGLU, GELU, RELU, IDENTITY = 0, 1, 2, 3        # the library's activation codes
SOFTMAX, SIGMOID = 0, 1
DEV = "cuda"


def listed():
    return [
        # one token of a serving step: grouped sigmoid routing over 256 experts
        dict(name="route token", op="route", T=1, E=256, k=8, score=SIGMOID, groups=8, keep=4, sum2=True,
             bias=True, renorm=True, scale=2.5, dtype="float32", dead=0),
        # prompt or training batch, the same router
        dict(name="route batch", op="route", T=16384, E=256, k=8, score=SIGMOID, groups=8, keep=4, sum2=True,
             bias=True, renorm=True, scale=2.5, dtype="float32", dead=0),
        # softmax scores, 64 experts, logits in bf16, some experts out of service
        dict(name="route softmax", op="route", T=8192, E=64, k=8, score=SOFTMAX, groups=1, keep=1, sum2=False,
             bias=False, renorm=True, scale=1.0, dtype="bfloat16", dead=3),
        # training: the router's gradient at the logits
        dict(name="route gradient", op="route_bwd", T=4096, E=256, k=8, score=SIGMOID, groups=8, keep=4, sum2=True,
             bias=True, renorm=True, scale=2.5, dtype="float32", dead=0),
        # one token through a projection with its residual
        dict(name="linear token", op="linear", M=1, K=4096, N=4096, act=IDENTITY, nk=False, out="bfloat16",
             bias=False, residual=True, save=False),
        # a decode batch through a gated FFN's first product
        dict(name="linear decode", op="linear", M=64, K=7168, N=2048, act=SWIGLU, nk=False, out="bfloat16",
             bias=False, residual=False, save=False),
        # ragged sizes, weights stored [N, K], the pre-activation kept for training
        dict(name="linear ragged", op="linear", M=1003, K=1160, N=2568, act=GELU, nk=True, out="bfloat16",
             bias=True, residual=True, save=True),
        # router logits in fp32
        dict(name="linear logits", op="linear", M=4096, K=7168, N=256, act=IDENTITY, nk=False, out="float32",
             bias=False, residual=False, save=False),
        # a prompt batch through a gated FFN's first product
        dict(name="linear ffn", op="linear", M=8192, K=4096, N=14336, act=SWIGLU, nk=False, out="bfloat16",
             bias=False, residual=False, save=False),
        # the gradients of an FFN product
        dict(name="linear gradients", op="linear_bwd", M=4096, K=4096, N=6400, act=GELU, nk=False, out="bfloat16",
             bias=True),
        # the layer's exit in training: dropout, then the residual
        dict(name="dropout residual", op="dropout", n=8192 * 4096, dtype="bfloat16", prob=0.1, residual=True),
        # its gradient on an odd fp32 length
        dict(name="dropout gradient", op="dropout_bwd", n=1000003, dtype="float32", prob=0.25),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_bwd", "linear", "linear", "linear_bwd", "dropout", "dropout_bwd"])
    if op in ("route", "route_bwd"):
        groups = rng.choice([1, 1, 2, 4, 5, 8])
        size = _log_uniform(rng, 8 if groups == 1 else 4, 384 // groups)
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(16, keep * size))
        return dict(op=op, T=_log_uniform(rng, 1, 16384), E=groups * size, k=k,
                    score=rng.choice([SOFTMAX, SIGMOID]), groups=groups, keep=keep, sum2=rng.random() < 0.5,
                    bias=rng.random() < 0.6, renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                    dtype=rng.choice(["float32", "float32", "bfloat16"]), dead=0)
    if op in ("linear", "linear_bwd"):
        act = rng.choice([SWIGLU, GELU, RELU, IDENTITY])
        while True:
            M, K, N = _log_uniform(rng, 1, 8192), 8 * _log_uniform(rng, 8, 1024), 8 * _log_uniform(rng, 2, 1024)
            if M * K * N * (2 if act == SWIGLU else 1) <= 1.2e11:
                break
        c = dict(op=op, M=M, K=K, N=N, act=act, nk=rng.random() < 0.5,
                 out=rng.choice(["bfloat16", "bfloat16", "float32"]), bias=rng.random() < 0.5)
        if op == "linear":
            c.update(residual=rng.random() < 0.5, save=rng.random() < 0.5)
        return c
    c = dict(op=op, n=_log_uniform(rng, 1000, 8192 * 4096), dtype=rng.choice(["bfloat16", "float32"]),
             prob=rng.choice([0.05, 0.1, 0.3, 0.5]))
    if op == "dropout":
        c.update(residual=rng.random() < 0.7)
    return c


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 1000 + 17)


def _randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def prepare(case, seed):
    """Inputs and output buffers; for the library also its problem and workspace."""
    g = _generator(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        dt = getattr(torch, case["dtype"])
        prior = torch.randn(E, generator=g, device=DEV) * 0.5   # some experts are liked more
        logits = torch.randn(T, E, generator=g, device=DEV) * 1.2 + prior
        if case["dead"]:
            gone = torch.randperm(E, generator=g, device=DEV)[:case["dead"]]
            logits[:, gone] = -math.inf
        s["logits"] = logits.to(dt)
        s["bias"] = -0.1 * prior + 0.01 * torch.randn(E, generator=g, device=DEV) if case["bias"] else None
        s["idx"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        s["w"] = torch.empty(T, k, dtype=torch.float32, device=DEV)
        if op == "route_bwd":
            s["idx"], _ = _route_plain(case, s["logits"], s["bias"])
            s["dw"] = torch.randn(T, k, generator=g, device=DEV)
            s["dlogits"] = torch.empty_like(s["logits"])
        if own:
            import mixture_experts_layer_forward_b200 as moe
            s["problem"] = moe.Select.make(
                T, E, k, score=case["score"], n_group=case["groups"], top_group=case["keep"],
                group_score=moe.GROUP_SUM2 if case["sum2"] else moe.GROUP_MAX, renorm=case["renorm"],
                scale=case["scale"])
    elif op in ("linear", "linear_bwd"):
        M, K, N = case["M"], case["K"], case["N"]
        cols = 2 * N if case["act"] == SWIGLU else N
        out = getattr(torch, case["out"])
        s["x"] = _randn(g, M, K)
        s["W"] = _randn(g, *((cols, K) if case["nk"] else (K, cols)), std=K ** -0.5)
        s["bias"] = _randn(g, cols, std=0.1, dtype=torch.float32) if case["bias"] else None
        if op == "linear":
            s["residual"] = _randn(g, M, N) if case["residual"] else None
            s["y"] = torch.empty(M, N, dtype=out, device=DEV)
            s["z"] = torch.empty(M, cols, dtype=torch.bfloat16, device=DEV) if case["save"] else None
        else:
            s["z"] = _randn(g, M, cols) if case["act"] != IDENTITY else None
            s["dy"] = _randn(g, M, N, dtype=out)
            s["dx"] = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
            s["dW"] = torch.empty_like(s["W"])
            s["dbias"] = torch.empty(cols, dtype=torch.float32, device=DEV) if case["bias"] else None
        if own:
            import mixture_experts_layer_forward_b200 as moe
            s["problem"] = moe.Linear.make(M, N, K, act=case["act"], w_layout=moe.W_NK if case["nk"] else moe.W_KN,
                                           out_dtype=out)
            size = moe.moe_linear_workspace_size if op == "linear" else moe.moe_linear_backward_workspace_size
            s["ws"] = torch.empty(size(s["problem"]), dtype=torch.uint8, device=DEV)
    else:
        dt, n = getattr(torch, case["dtype"]), case["n"]
        s["x"] = _randn(g, n, dtype=dt)
        s["residual"] = _randn(g, n, dtype=dt) if case.get("residual") else None
        s["y"] = torch.empty_like(s["x"])
        # the generator's seed and offset, on the device so that a captured step can advance them
        s["rng"] = torch.tensor([0x9E3779B97F4A7C15 // 3 + int(seed) * 7919, int(seed) * 104729 + 5],
                                dtype=torch.int64, device=DEV)
    return s


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------

def _route_plain(c, logits, bias):
    """(idx, w). The selection in 64 bits, stable sorts for ties to the lower id."""
    T, E, k = c["T"], c["E"], c["k"]
    l64 = logits.double()
    live = l64 > -math.inf
    l64 = torch.where(live, l64, -math.inf)
    if c["score"] == SOFTMAX:
        e = torch.exp(l64 - l64.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-l64))
    value = score + bias.double() if bias is not None else score
    key = value if bias is not None else l64
    key = torch.where(live, key, -math.inf)
    if c["groups"] > 1:
        G = c["groups"]
        if c["sum2"]:
            v = torch.where(live, value, -math.inf).view(T, G, E // G).sort(dim=2, descending=True).values[..., :2]
            gone = v[..., 0] == -math.inf
            gv = torch.where(v == -math.inf, 0.0, v).sum(2)
            gv = torch.where(gone, -math.inf, gv)
        else:
            gv = key.view(T, G, E // G).amax(2)
        best = gv.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        chosen = torch.zeros(T, G, dtype=torch.bool, device=logits.device).scatter_(1, best, True)
        key = torch.where(chosen.repeat_interleave(E // G, 1), key, -math.inf)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    l32 = logits.float()
    if c["score"] == SOFTMAX:
        m = l32.amax(1, keepdim=True)
        e = torch.exp(l32 - m)
        w = e.gather(1, idx)
        w = w / (w.sum(1, keepdim=True) if c["renorm"] else e.sum(1, keepdim=True))
    else:
        w = torch.sigmoid(l32).gather(1, idx)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
    return idx.to(torch.int32), w * c["scale"]


def _route_bwd_plain(c, logits, idx, dw):
    l = logits.float()
    idx = idx.long()
    sel = l.gather(1, idx)
    if c["score"] == SIGMOID:
        s = torch.sigmoid(sel)
        if c["renorm"]:
            q = s / s.sum(1, keepdim=True)
            d = q * (1 - s) * (dw - (dw * q).sum(1, keepdim=True))
        else:
            d = dw * s * (1 - s)
        out = torch.zeros_like(l).scatter_(1, idx, d)
    elif c["renorm"]:
        q = torch.softmax(sel, 1)
        out = torch.zeros_like(l).scatter_(1, idx, q * (dw - (dw * q).sum(1, keepdim=True)))
    else:
        p = torch.softmax(l, 1)
        g = torch.zeros_like(l).scatter_(1, idx, dw)
        out = p * (g - (g * p).sum(1, keepdim=True))
    return (out * c["scale"]).to(logits.dtype)


_GC = math.sqrt(2.0 / math.pi)


def _act_plain(act, z):
    if act == SWIGLU:
        gate, up = z.chunk(2, 1)
        return gate * torch.sigmoid(gate) * up
    if act == GELU:
        return 0.5 * z * (1 + torch.tanh(_GC * (z + 0.044715 * z * z * z)))
    return torch.clamp(z, min=0) if act == RELU else z


def _act_grad_plain(act, z, dy):
    if act == SWIGLU:
        gate, up = z.chunk(2, 1)
        s = torch.sigmoid(gate)
        return torch.cat([dy * up * s * (1 + gate * (1 - s)), dy * gate * s], 1)
    if act == GELU:
        t = torch.tanh(_GC * (z + 0.044715 * z * z * z))
        return dy * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _GC * (1 + 3 * 0.044715 * z * z))
    return dy * (z > 0) if act == RELU else dy


def _keep_plain(n, rng, prob):
    """Truth values of the n elements kept, and the scale: ten rounds of the 4 x 32-bit counter
    generator of Salmon, Moraes, Dror and Shaw (2011), 16 bits an element."""
    thr = int(round(prob * 65536))
    low = 0xFFFFFFFF
    ctr = torch.arange((n + 7) // 8, device=rng.device) + rng[1]
    c0, c1 = ctr & low, (ctr >> 32) & low
    c2, c3 = torch.zeros_like(c0), torch.zeros_like(c0)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], 1)
    u = torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:n]
    return u >= thr, 65536.0 / (65536 - thr)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        idx, w = _route_plain(c, s["logits"], s["bias"])
        return {"idx": idx, "w": w}
    if op == "route_bwd":
        return {"dlogits": _route_bwd_plain(c, s["logits"], s["idx"], s["dw"])}
    if op == "linear":
        W = s["W"].float()
        z = s["x"].float() @ (W.t() if c["nk"] else W)
        if s["bias"] is not None:
            z = z + s["bias"]
        y = _act_plain(c["act"], z)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        r = {"y": y.to(s["y"].dtype)}
        if c["save"]:
            r["z"] = z.to(torch.bfloat16)
        return r
    if op == "linear_bwd":
        W = s["W"].float()
        dy = s["dy"].float()
        dz = _act_grad_plain(c["act"], None if s["z"] is None else s["z"].float(), dy)
        x = s["x"].float()
        r = {"dx": (dz @ (W if c["nk"] else W.t())).to(torch.bfloat16),
             "dW": (dz.t() @ x if c["nk"] else x.t() @ dz).to(torch.bfloat16)}
        if c["bias"]:
            r["dbias"] = dz.sum(0)
        return r
    keep, scale = _keep_plain(c["n"], s["rng"], c["prob"])
    y = torch.where(keep, s["x"].float() * scale, 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(s["x"].dtype)}


def _run_own(s):
    import mixture_experts_layer_forward_b200 as moe
    op = s["case"]["op"]
    if op == "route":
        moe.moe_route_select(s["problem"], s["logits"], s["bias"], s["idx"], s["w"])
        return {"idx": s["idx"], "w": s["w"]}
    if op == "route_bwd":
        moe.moe_route_select_backward(s["problem"], s["logits"], s["idx"], s["dw"], s["dlogits"])
        return {"dlogits": s["dlogits"]}
    if op == "linear":
        moe.moe_linear_forward(s["problem"], s["x"], s["W"], s["bias"], s["residual"], s["y"], s["ws"], z=s["z"])
        return {"y": s["y"], "z": s["z"]} if s["z"] is not None else {"y": s["y"]}
    if op == "linear_bwd":
        moe.moe_linear_backward(s["problem"], s["x"], s["W"], s["z"], s["dy"], s["dx"], s["dW"], s["dbias"], s["ws"])
        r = {"dx": s["dx"], "dW": s["dW"]}
        if s["dbias"] is not None:
            r["dbias"] = s["dbias"]
        return r
    if op == "dropout":
        moe.moe_dropout_add(s["x"], s["residual"], s["y"], s["case"]["prob"], s["rng"])
    else:
        moe.moe_dropout_add_backward(s["x"], s["y"], s["case"]["prob"], s["rng"])
    return {"y": s["y"]}


# ---------------------------------------------------------------------------------------
# what a pass cannot do without, and its values in 64 bits
# ---------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "float32" else 2
        if op == "route":
            return {"bytes": T * E * size + T * k * 8 + (4 * E if case["bias"] else 0), "flops": 10 * T * E}
        dense = case["score"] == SOFTMAX and not case["renorm"]
        return {"bytes": T * E * size * (2 if dense else 1) + T * k * (8 if dense else 8 + size), "flops": 10 * T * k}
    if op in ("linear", "linear_bwd"):
        M, K, N = case["M"], case["K"], case["N"]
        cols = 2 * N if case["act"] == SWIGLU else N
        size = 4 if case["out"] == "float32" else 2
        b = 4 * cols if case["bias"] else 0
        if op == "linear":
            moved = 2 * (M * K + K * cols) + b + M * N * (size + (2 if case["residual"] else 0))
            return {"bytes": moved + (2 * M * cols if case["save"] else 0), "flops": 2 * M * K * cols}
        moved = 2 * (M * K + K * cols) * 2 + b + M * N * size
        return {"bytes": moved + (2 * M * cols if case["act"] != IDENTITY else 0), "flops": 4 * M * K * cols}
    size = 4 if case["dtype"] == "float32" else 2
    return {"bytes": case["n"] * size * (3 if case.get("residual") else 2), "flops": 12 * case["n"]}


def _log_sigmoid(l):
    return np.minimum(l, 0.0) - np.log1p(np.exp(-np.abs(l)))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("route", "route_bwd"):
        l = s["logits"].double().cpu().numpy()
        T, E, k = case["T"], case["E"], case["k"]
        top = l.max(1, keepdims=True)
        logp = l - top - np.log(np.exp(l - top).sum(1, keepdims=True))
        logs = _log_sigmoid(l) if case["score"] == SIGMOID else logp
        if op == "route":
            live = np.isfinite(l)
            b = s["bias"].double().cpu().numpy() if case["bias"] else np.zeros(E)
            with np.errstate(invalid="ignore"):
                value = np.where(live, np.exp(logs) + b, -np.inf)
            key = value if case["bias"] else np.where(live, l, -np.inf)
            if case["groups"] > 1:
                G = case["groups"]
                v = -np.sort(-(value if case["sum2"] else key).reshape(T, G, E // G), axis=2)
                total = v[..., 0].copy()
                if case["sum2"] and E // G > 1:
                    total += np.where(np.isfinite(v[..., 1]), v[..., 1], 0.0)
                rank = np.argsort(np.argsort(-total, axis=1, kind="stable"), axis=1, kind="stable")
                key = np.where(np.repeat(rank < case["keep"], E // G, axis=1), key, -np.inf)
            idx = np.argsort(-key, axis=1, kind="stable")[:, :k]
            sel = np.take_along_axis(logs, idx, 1)
            if case["renorm"]:
                w = 1.0 / np.exp(sel[:, None, :] - sel[:, :, None]).sum(2)
            else:
                w = np.exp(sel)
            return {"idx": None, "w": torch.from_numpy(w * case["scale"])}
        idx = s["idx"].long().cpu().numpy()
        g = s["dw"].double().cpu().numpy() * case["scale"]
        sel = np.take_along_axis(logs, idx, 1)
        eye = np.eye(k)
        out = np.zeros_like(l)
        if case["renorm"]:                       # dw_j / dlog s_i, then dlog s_i / dl_i
            q = np.exp(sel - sel.max(1, keepdims=True))
            q /= q.sum(1, keepdims=True)
            jac = q[:, :, None] * (eye[None] - q[:, None, :])
            d = np.einsum("tj,tji->ti", g, jac)
            if case["score"] == SIGMOID:
                d *= np.exp(_log_sigmoid(-np.take_along_axis(l, idx, 1)))
            np.put_along_axis(out, idx, d, 1)
        elif case["score"] == SIGMOID:
            d = g * np.exp(sel + _log_sigmoid(-np.take_along_axis(l, idx, 1)))
            np.put_along_axis(out, idx, d, 1)
        else:
            np.put_along_axis(out, idx, g * np.exp(sel), 1)
            out -= np.exp(logp) * (g * np.exp(sel)).sum(1, keepdims=True)
        return {"dlogits": torch.from_numpy(out)}
    if op in ("linear", "linear_bwd"):
        act, N = case["act"], case["N"]
        x = s["x"].double()
        W = s["W"].double().t() if case["nk"] else s["W"].double()
        c = 2.0 * math.sqrt(2.0 / math.pi)       # gelu(z) = z / (1 + exp(-c (z + 0.044715 z^3)))
        if op == "linear":
            z = torch.mm(x, W)
            if case["bias"]:
                z += s["bias"].double()
            if act == SWIGLU:
                y = z[:, N:] * z[:, :N] / (1 + torch.exp(-z[:, :N]))
            elif act == GELU:
                y = z / (1 + torch.exp(-c * (z + 0.044715 * z ** 3)))
            else:
                y = z * (z > 0) if act == RELU else z
            if case["residual"]:
                y = y + s["residual"].double()
            return {"y": y, "z": z} if case["save"] else {"y": y}
        dy = s["dy"].double()
        if act == IDENTITY:
            dz = dy
        else:
            z = s["z"].double()
            if act == SWIGLU:
                e = 1 / (1 + torch.exp(-z[:, :N]))
                dz = torch.cat([dy * z[:, N:] * (e + z[:, :N] * e * (1 - e)), dy * z[:, :N] * e], 1)
            elif act == GELU:
                e = 1 / (1 + torch.exp(-c * (z + 0.044715 * z ** 3)))
                dz = dy * (e + z * e * (1 - e) * c * (1 + 3 * 0.044715 * z ** 2))
            else:
                dz = dy * (z > 0)
        dW = torch.mm(x.t(), dz)
        r = {"dx": torch.mm(dz, W.t()), "dW": dW.t().contiguous() if case["nk"] else dW}
        if case["bias"]:
            r["dbias"] = torch.ones(1, dz.shape[0], dtype=torch.float64, device=dz.device).mm(dz)[0]
        return r
    n = case["n"]
    seed64, offset = (int(v) for v in s["rng"].cpu())
    # counters and keys as 64-bit words of numpy, products split by hand
    ctr = np.arange(offset, offset + (n + 7) // 8, dtype=np.uint64)
    m32, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    v = [ctr & m32, ctr >> sh, np.zeros_like(ctr), np.zeros_like(ctr)]
    key = [seed64 & 0xFFFFFFFF, (seed64 >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        p0, p1 = v[0] * np.uint64(0xD2511F53), v[2] * np.uint64(0xCD9E8D57)
        v = [(p1 >> sh) ^ v[1] ^ np.uint64(key[0]), p1 & m32, (p0 >> sh) ^ v[3] ^ np.uint64(key[1]), p0 & m32]
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    u = np.stack([w.astype(np.uint32) for w in v], 1).view(np.uint16).reshape(-1)[:n]
    t = int(round(case["prob"] * 65536))
    y = np.where(u >= t, s["x"].double().cpu().numpy() * (65536 / (65536 - t)), 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].double().cpu().numpy()
    return {"y": torch.from_numpy(y)}
