"""Cases for measuring the routing, mixture-of-experts and low-rank-adapter operators.

Every case is one call (or one forward and backward pair) of an operator as a
program makes it.  ``run`` computes it in plain torch operations in fp32,
rounded once at the end, or, with ``own`` true, through the package's entry
points.  ``exact`` restates each operator in fp64.

  route     top-k routing of tokens to experts from router logits
  route_grad  the same in training: routing, then the logits' gradient
  moe       the whole mixture-of-experts layer for a few tokens
  lowrank   a shared projection with one low-rank adapter per row
  lowrank_grad  its gradients: dX, dA, dB (the shared projection is frozen)
"""

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # Routing one decode step of 16 sequences: latency of one small launch.
        {"name": "route_decode", "op": "route", "T": 16, "G": 64, "k": 2, "dtype": "f32", "normalize": 1, "masked": 0},
        # Routing a long prefill over many fine-grained experts; bf16 logits tie often,
        # some experts are masked out, and a few rows have none left.
        {"name": "route_prefill", "op": "route", "T": 65536, "G": 256, "k": 8, "dtype": "bf16", "normalize": 1,
         "masked": 1},
        # A training step's routing with softmax weights over all experts, and the logits' gradient.
        {"name": "route_train", "op": "route_grad", "T": 16384, "G": 64, "k": 2, "dtype": "f32", "normalize": 0,
         "masked": 0},
        # A small layer with odd sizes, three tokens: latency.
        {"name": "moe_small", "op": "moe", "T": 3, "G": 32, "S": 4, "K": 1000, "F": 712, "dtype": "f16", "dropped": 0},
        # One token of a large layer: the weights of its two experts streamed once.
        {"name": "moe_one_token", "op": "moe", "T": 1, "G": 64, "S": 2, "K": 4096, "F": 14336, "dtype": "bf16",
         "dropped": 0},
        # A ragged decode batch over many small experts, some picks dropped (-1).
        {"name": "moe_fine", "op": "moe", "T": 29, "G": 128, "S": 8, "K": 2048, "F": 1024, "dtype": "bf16",
         "dropped": 1},
        # A decode batch of 64 that reads most experts of the large layer.
        {"name": "moe_batch", "op": "moe", "T": 64, "G": 64, "S": 2, "K": 4096, "F": 14336, "dtype": "bf16",
         "dropped": 0},
        # One token of one request through an adapted projection: latency.
        {"name": "lowrank_one_token", "op": "lowrank", "M": 1, "K": 4096, "N": 4096, "R": 16, "G": 8,
         "dtype": "bf16", "runs": 0},
        # A decode batch whose rows belong to different requests and adapters.
        {"name": "lowrank_batch", "op": "lowrank", "M": 61, "K": 4096, "N": 14336, "R": 32, "G": 48,
         "dtype": "f16", "runs": 0},
        # Prefill of many requests, each a run of rows with its own adapter or none.
        {"name": "lowrank_prefill", "op": "lowrank", "M": 8192, "K": 4096, "N": 14336, "R": 16, "G": 12,
         "dtype": "bf16", "runs": 1},
        # Gradients of a small ragged batch with an odd rank.
        {"name": "lowrank_grad_ragged", "op": "lowrank_grad", "M": 1027, "K": 2048, "N": 1000, "R": 12, "G": 5,
         "dtype": "f16", "runs": 1},
        # Gradients of a training step of several adapters at once.
        {"name": "lowrank_grad_train", "op": "lowrank_grad", "M": 8192, "K": 4096, "N": 4096, "R": 16, "G": 8,
         "dtype": "bf16", "runs": 1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dim(rng, lo, hi):
    """A matrix dimension: a multiple of 8 (rows of 16 bytes), most of them no multiple of 64."""
    v = max(lo, min(hi, 8 * int(round(_log(rng, lo, hi) / 8))))
    return v + 8 if v == 3072 else v


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "moe", "moe", "moe", "lowrank", "lowrank", "lowrank",
                     "lowrank_grad", "lowrank_grad"])
    if op in ("route", "route_grad"):
        G = _log(rng, 8, 256)
        return {"op": op, "T": _log(rng, 1, 65536), "G": G, "k": rng.randint(1, min(8, G)),
                "dtype": rng.choice(["f32", "bf16", "f16"]), "normalize": rng.randint(0, 1),
                "masked": rng.randint(0, 1)}
    if op == "moe":
        G = _log(rng, 4, 128)
        K, F = _dim(rng, 256, 4096), _dim(rng, 256, 14336)
        while 3 * G * K * F > 64 * 3 * 4096 * 14336:
            G = max(4, G // 2)
        return {"op": op, "T": _log(rng, 1, 64), "G": G, "S": rng.randint(1, min(8, G)), "K": K, "F": F,
                "dtype": rng.choice(["bf16", "f16"]), "dropped": rng.randint(0, 1)}
    runs = 1 if op == "lowrank_grad" else rng.randint(0, 1)
    K, N = _dim(rng, 512, 4096), _dim(rng, 512, 14336 if op == "lowrank" else 4096)
    return {"op": op, "M": _log(rng, 64, 8192) if runs else _log(rng, 1, 256), "K": K, "N": N,
            "R": rng.choice([4, 8, 12, 16, 16, 24, 32, 64]), "G": _log(rng, 1, 64),
            "dtype": rng.choice(["bf16", "f16"]), "runs": runs}


# ------------------------------------------------------------------ inputs


def _normal(shape, gen, dtype, scale=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=gen, device="cuda").mul_(scale)
    return out


def _picks(case, seed):
    """Distinct experts per token without replacement, popular ones first (p proportional to (g + 1)^-1.1)."""
    rng = np.random.default_rng(seed)
    T, G, S = case["T"], case["G"], case["S"]
    score = -1.1 * np.log(np.arange(1, G + 1)) + rng.gumbel(size=(T, G))
    idx = np.argsort(-score, axis=1, kind="stable")[:, :S].astype(np.int32)
    w = np.exp(rng.normal(size=(T, S)))
    w = (w / w.sum(axis=1, keepdims=True)).astype(np.float32)
    if case["dropped"]:
        gone = rng.random((T, S)) < 0.1
        if T > 2:
            gone[T // 2] = True          # one token with no expert at all
        idx[gone] = -1
        w[gone] = 0.0
    return idx, w


def _adapters(case, seed):
    """Adapter of every row: one per row (a decode batch), or runs of rows (requests); -1 is no adapter."""
    rng = np.random.default_rng(seed)
    M, G = case["M"], case["G"]
    if not case["runs"]:
        a = rng.integers(0, G, size=M)
        if M > 4:
            a[rng.random(M) < 0.1] = -1
        return a.astype(np.int32)
    a = np.empty(M, dtype=np.int32)
    at = 0
    while at < M:
        n = int(np.exp(rng.uniform(np.log(32), np.log(2048))))
        a[at:at + n] = -1 if rng.random() < 0.1 else rng.integers(0, G)
        at += n
    return a


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], _DT[case["dtype"]]
    st = {"case": case}
    if op in ("route", "route_grad"):
        T, G, k = case["T"], case["G"], case["k"]
        logits = torch.randn((T, G), generator=gen, device="cuda").mul_(1.5)
        if case["masked"]:
            off = torch.rand((T, G), generator=gen, device="cuda") < 0.25
            off[torch.rand(T, generator=gen, device="cuda") < 0.01] = True
            logits = logits.masked_fill(off, float("-inf"))
        st["logits"] = logits.to(dt)
        st["dw"] = torch.randn((T, k), generator=gen, device="cuda")
    elif op == "moe":
        G, K, F, T = case["G"], case["K"], case["F"], case["T"]
        st["x"] = _normal((T, K), gen, dt)
        st["w_gate"] = _normal((G, K, F), gen, dt, K ** -0.5)
        st["w_up"] = _normal((G, K, F), gen, dt, K ** -0.5)
        st["w_down"] = _normal((G, F, K), gen, dt, F ** -0.5)
        idx, w = _picks(case, seed)
        st["idx"], st["w"] = torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda()
    else:
        M, K, N, R, G = (case[n] for n in "MKNRG")
        st["X"] = _normal((M, K), gen, dt)
        st["W"] = _normal((K, N), gen, dt, K ** -0.5)
        st["A"] = _normal((G, K, R), gen, dt, K ** -0.5)
        st["B"] = _normal((G, R, N), gen, dt, 0.5 * R ** -0.5)
        st["scales"] = torch.rand(G, generator=gen, device="cuda") + 0.5
        st["idx"] = torch.from_numpy(_adapters(case, seed)).cuda()
        if op == "lowrank_grad":
            st["dY"] = _normal((M, N), gen, dt)
    if own:
        import quantized_gemm_gb300 as qg
        nbytes = 0
        if op == "moe":
            nbytes = qg.mm_moe_layer_workspace_size(st["x"], st["w_gate"], st["w_up"], st["w_down"], st["idx"])
        elif op == "lowrank":
            nbytes = qg.mm_lowrank_matmul_workspace_size(st["X"], st["W"], st["A"], st["B"])
        elif op == "lowrank_grad":
            nbytes = qg.mm_lowrank_matmul_grad_workspace_size(st["X"], st["W"], st["A"], st["B"])
        st["ws"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None
    return st


# ------------------------------------------------------------------ one pass


def _plain_route(logits, k, normalize):
    l = logits.float()
    G = l.shape[1]
    l = torch.where(torch.isnan(l), -math.inf, l)
    top = l.amax(dim=1, keepdim=True)
    # a row with nothing left keeps probability zero everywhere
    e = torch.where(l == top, 1.0, torch.exp(l - top))
    e = torch.where(l == -math.inf, 0.0, e)
    total = e.sum(dim=1, keepdim=True)
    p = e / torch.where(total == 0, 1.0, total)
    at = torch.arange(G, device=l.device)
    left, idx, val = l, [], []
    for _ in range(k):
        best = left.amax(dim=1, keepdim=True)
        i = torch.where(left == best, at, G).amin(dim=1, keepdim=True)
        there = best > -math.inf
        idx.append(torch.where(there, i, -1))
        val.append(torch.where(there, p.gather(1, i), 0.0))
        left = torch.where(at == i, -math.inf, left)
    idx, val = torch.cat(idx, dim=1).to(torch.int32), torch.cat(val, dim=1)
    if normalize:
        s = val.sum(dim=1, keepdim=True)
        val = val / torch.where(s == 0, 1.0, s)
    return idx, val, p


def _plain_route_grad(logits, idx, w, p, dw, normalize):
    G = logits.shape[1]
    hot = (idx.unsqueeze(2) == torch.arange(G, device=idx.device)).float()   # [T, k, G]
    d = (dw.unsqueeze(2) * hot).sum(dim=1)
    if normalize:
        q = (w.unsqueeze(2) * hot).sum(dim=1)
    else:
        q = p
    picked = hot.sum(dim=1)
    dot = (q * d).sum(dim=1, keepdim=True)
    if normalize:
        return q * (d - dot) * picked
    return q * (d - dot)


def _plain_moe(x, wg, wu, wd, idx, w):
    T, S = idx.shape
    G = wg.shape[0]
    xf = x.float()
    out = torch.zeros((T, wd.shape[2]), device=x.device)

    def act(a, b):
        return a / (1.0 + torch.exp(-a)) * b

    if T * S <= G:                       # fewer picks than experts: the picked experts' weights
        for t in range(T):
            for s in range(S):
                e = idx[t, s].clamp(min=0).view(1)
                row = xf[t:t + 1]
                h = act(row @ wg[e][0].float(), row @ wu[e][0].float())
                y = h @ wd[e][0].float()
                out[t:t + 1] += torch.where(idx[t, s] >= 0, w[t, s] * y, 0.0)
    else:                                # every expert on every token, masked
        for e in range(G):
            we = torch.where(idx == e, w, 0.0).sum(dim=1, keepdim=True)
            has = (idx == e).any(dim=1, keepdim=True)
            h = act(xf @ wg[e].float(), xf @ wu[e].float())
            out += torch.where(has, we * (h @ wd[e].float()), 0.0)
    return out.to(x.dtype)


def _row_mask(idx, G, R):
    """[M, G * R]: whether column g * R + r belongs to the row's adapter."""
    return (idx.unsqueeze(1) == torch.arange(G, device=idx.device)).repeat_interleave(R, dim=1)


def _flat_adapters(A, B):
    """A as [K, G * R] and B as [G * R, N], in fp32."""
    return A.float().permute(1, 0, 2).reshape(A.shape[1], -1), B.float().reshape(-1, B.shape[2])


def _plain_lowrank(X, W, A, B, idx, scales):
    G, R = B.shape[0], B.shape[1]
    a, b = _flat_adapters(A, B)
    xf = X.float()
    z = torch.where(_row_mask(idx, G, R), (xf @ a) * scales.repeat_interleave(R), 0.0)
    return (xf @ W.float() + z @ b).to(X.dtype)


def _plain_lowrank_grad(dY, X, W, A, B, idx, scales):
    G, R = B.shape[0], B.shape[1]
    a, b = _flat_adapters(A, B)
    xf, df = X.float(), dY.float()
    mask, s = _row_mask(idx, G, R), scales.repeat_interleave(R)
    v = torch.where(mask, (df @ b.t()) * s, 0.0)
    u = torch.where(mask, (xf @ a) * s, 0.0)
    dX = df @ W.float().t() + v @ a.t()
    dA = (xf.t() @ v).reshape(A.shape[1], G, R).permute(1, 0, 2)
    dB = (u.t() @ df).reshape(G, R, -1)
    return dX.to(X.dtype), dA.to(X.dtype).contiguous(), dB.to(X.dtype)


def run(state):
    case, s = state["case"], state
    op = case["op"]
    if own:
        import quantized_gemm_gb300 as qg
        if op == "route":
            return qg.mm_route_topk(s["logits"], case["k"], case["normalize"])
        if op == "route_grad":
            idx, w = qg.mm_route_topk(s["logits"], case["k"], case["normalize"])
            return idx, w, qg.mm_route_topk_grad(s["logits"], idx, s["dw"], case["normalize"])
        if op == "moe":
            return qg.mm_moe_layer(s["x"], s["w_gate"], s["w_up"], s["w_down"], s["idx"], s["w"], activation="silu",
                                   workspace=s["ws"])
        if op == "lowrank":
            return qg.mm_lowrank_matmul(s["X"], s["W"], s["A"], s["B"], s["idx"], s["scales"], workspace=s["ws"])
        return qg.mm_lowrank_matmul_grad(s["dY"], s["X"], s["W"], s["A"], s["B"], s["idx"], s["scales"],
                                         workspace=s["ws"])
    if op == "route":
        return _plain_route(s["logits"], case["k"], case["normalize"])[:2]
    if op == "route_grad":
        idx, w, p = _plain_route(s["logits"], case["k"], case["normalize"])
        return idx, w, _plain_route_grad(s["logits"], idx, w, p, s["dw"], case["normalize"]).to(s["logits"].dtype)
    if op == "moe":
        return _plain_moe(s["x"], s["w_gate"], s["w_up"], s["w_down"], s["idx"], s["w"])
    if op == "lowrank":
        return _plain_lowrank(s["X"], s["W"], s["A"], s["B"], s["idx"], s["scales"])
    return _plain_lowrank_grad(s["dY"], s["X"], s["W"], s["A"], s["B"], s["idx"], s["scales"])


# ------------------------------------------------------------------ work of one pass


def work(case):
    op, e = case["op"], _SIZE[case["dtype"]]
    if op in ("route", "route_grad"):
        T, G, k = case["T"], case["G"], case["k"]
        fwd = {"bytes": T * G * e + T * k * 8, "flops": 3 * T * G}
        if op == "route":
            return fwd
        return {"bytes": fwd["bytes"] + T * G * e * 2 + T * k * 8, "flops": fwd["flops"] + 6 * T * G}
    if op == "moe":
        T, K, F = case["T"], case["K"], case["F"]
        used = picks = 0
        for seed in range(4):            # the experts that a batch picks, on average
            idx = _picks(case, seed)[0]
            used += len(set(idx[idx >= 0].tolist())) / 4
            picks += int((idx >= 0).sum()) / 4
        return {"bytes": int(used * 3 * K * F * e + 2 * T * K * e + T * case["S"] * 8),
                "flops": int(picks * 6 * K * F)}
    M, K, N, R, G = (case[n] for n in "MKNRG")
    used = with_one = 0
    for seed in range(4):
        a = _adapters(case, seed)
        used += len(set(a[a >= 0].tolist())) / 4
        with_one += int((a >= 0).sum()) / 4
    low = 2 * with_one * R * (K + N)
    if op == "lowrank":
        return {"bytes": int(e * (M * K + K * N + M * N + used * R * (K + N)) + 4 * M + 4 * G),
                "flops": int(2 * M * N * K + low)}
    return {"bytes": int(e * (2 * M * K + K * N + M * N + used * R * (K + N) + G * R * (K + N)) + 4 * M + 4 * G),
            "flops": int(2 * M * N * K + 3 * low)}


# ------------------------------------------------------------------ fp64


def _exact_route(logits, k, normalize):
    l = logits.double().cpu().numpy()
    l = np.where(np.isnan(l), -np.inf, l)
    T = l.shape[0]
    order = np.argsort(-l, axis=1, kind="stable")[:, :k]
    top = l.max(axis=1, keepdims=True)
    none = ~(top > -np.inf)
    with np.errstate(invalid="ignore"):
        e = np.where(l == top, 1.0, np.exp(l - np.where(none, 0.0, top)))
    e[l == -np.inf] = 0.0
    p = e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300)
    rows = np.arange(T)[:, None]
    ok = l[rows, order] > -np.inf
    idx = np.where(ok, order, -1)
    w = np.where(ok, p[rows, order], 0.0)
    if normalize:
        w = w / np.maximum(w.sum(axis=1, keepdims=True), 1e-300)
    return idx.astype(np.int32), w, p


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op in ("route", "route_grad"):
        idx, w, p = _exact_route(st["logits"], case["k"], case["normalize"])
        if op == "route":
            return idx, w
        dw = st["dw"].double().cpu().numpy()
        rows, col = np.nonzero(idx >= 0)
        d = np.zeros_like(p)
        d[rows, idx[rows, col]] = dw[rows, col]
        if case["normalize"]:
            q = np.zeros_like(p)
            q[rows, idx[rows, col]] = w[rows, col]
        else:
            q = p
        return idx, w, q * (d - (q * d).sum(axis=1, keepdims=True))
    if op == "moe":
        x, idx, w = st["x"].double(), st["idx"].cpu().numpy(), st["w"].double()
        out = torch.zeros((x.shape[0], st["w_down"].shape[2]), dtype=torch.float64, device="cuda")
        for e in sorted(set(idx[idx >= 0].tolist())):
            t, s = np.nonzero(idx == e)
            t, s = torch.from_numpy(t).cuda(), torch.from_numpy(s).cuda()
            a, b = x[t] @ st["w_gate"][e].double(), x[t] @ st["w_up"][e].double()
            out.index_add_(0, t, w[t, s].unsqueeze(1) * ((a * torch.sigmoid(a) * b) @ st["w_down"][e].double()))
        return out
    X, W, idx = st["X"].double(), st["W"].double(), st["idx"].cpu().numpy()
    groups = {g: torch.from_numpy(np.nonzero(idx == g)[0]).cuda() for g in sorted(set(idx[idx >= 0].tolist()))}
    scales = st["scales"].double()
    if op == "lowrank":
        Y = X @ W
        for g, m in groups.items():
            Y[m] += scales[g] * ((X[m] @ st["A"][g].double()) @ st["B"][g].double())
        return Y
    dY = st["dY"].double()
    dX = dY @ W.t()
    dA = torch.zeros(st["A"].shape, dtype=torch.float64, device="cuda")
    dB = torch.zeros(st["B"].shape, dtype=torch.float64, device="cuda")
    for g, m in groups.items():
        a, b = st["A"][g].double(), st["B"][g].double()
        v = scales[g] * (dY[m] @ b.t())
        dX[m] += v @ a.t()
        dA[g] = X[m].t() @ v
        dB[g] = scales[g] * ((X[m] @ a).t() @ dY[m])
    return dX, dA, dB
