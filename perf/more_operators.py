"""Cases for measuring 8-bit products, the router's balance loss and the orthogonalised update.

Every case is what a program calls at once.  ``run`` computes it in plain torch operations in fp32, rounded once at the
end, or, with ``own`` true, through the package's entry points.  ``exact`` restates each operator in fp64.

  quantize  rows to int8 with one scale each: s = amax / 127, q = round(x / s), ties to even
  int8      Y = (A B) * a_scale[m] * b_scale[n] + bias[n], A and B int8, the scales per token and per channel
  balance   a training step's balance loss: G * sum_g (picks of g / all picks) * (mean probability of g), with the
            picks per expert, and its gradient added to another gradient of the logits
  orth      an optimiser's update: X = G / |G|, then X = a X + (b X X^T + c (X X^T)^2) X for some steps
"""

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_COEFFICIENTS = (3.4445, -4.7750, 2.0315)
_EPS = 1e-7


def listed():
    return [
        # One token's activations before an 8-bit projection: latency of one small launch.
        {"name": "quant_one_token", "op": "quantize", "M": 1, "K": 4096, "dtype": "bf16"},
        # A prefill's activations.
        {"name": "quant_prefill", "op": "quantize", "M": 16384, "K": 4096, "dtype": "bf16"},
        # One token through a wide projection: the 8-bit weights are read once.
        {"name": "int8_one_token", "op": "int8", "M": 1, "K": 4096, "N": 14336, "dtype": "bf16", "bias": 0, "nk": 1},
        # A decode batch of odd size, with a bias.
        {"name": "int8_batch", "op": "int8", "M": 61, "K": 4096, "N": 14336, "dtype": "f16", "bias": 1, "nk": 1},
        # Ragged sizes, none a multiple of a tile, weights stored [K, N], fp32 out.
        {"name": "int8_ragged", "op": "int8", "M": 1027, "K": 2051, "N": 1001, "dtype": "f32", "bias": 1, "nk": 0},
        # A prefill's tokens through a square projection.
        {"name": "int8_prefill", "op": "int8", "M": 16384, "K": 4096, "N": 4096, "dtype": "bf16", "bias": 0, "nk": 1},
        # The balance of a few tokens: latency of the loss and of its gradient.
        {"name": "balance_small", "op": "balance", "T": 16, "G": 64, "k": 2, "dtype": "f32", "masked": 0},
        # A long batch over many fine-grained experts, some masked out and some rows padding.
        {"name": "balance_train", "op": "balance", "T": 65536, "G": 256, "k": 8, "dtype": "bf16", "masked": 1},
        # A router's small weight matrix kept in fp32, odd sizes: latency of the chain of products.
        {"name": "orth_router", "op": "orth", "B": 1, "M": 61, "N": 1000, "dtype": "f32"},
        # A square projection's update in fp32.
        {"name": "orth_f32", "op": "orth", "B": 1, "M": 2048, "N": 2048, "dtype": "f32"},
        # The stacked updates of 32 experts, taller than wide.
        {"name": "orth_experts", "op": "orth", "B": 32, "M": 2048, "N": 1024, "dtype": "bf16"},
        # One wide projection.
        {"name": "orth_wide", "op": "orth", "B": 1, "M": 4096, "N": 14336, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "int8", "int8", "int8", "balance", "balance", "orth", "orth", "orth"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "quantize":
        K = _log(rng, 64, 14336)
        return {"op": op, "M": _log(rng, 1, max(1, min(16384, 16384 * 4096 // K))), "K": K, "dtype": dtype}
    if op == "int8":
        K, N = _log(rng, 256, 8192), _log(rng, 256, 14336)
        M = _log(rng, 1, max(1, min(16384, 16384 * 4096 * 4096 // (K * N))))
        return {"op": op, "M": M, "K": K, "N": N, "dtype": dtype, "bias": rng.randint(0, 1), "nk": rng.randint(0, 3) > 0}
    if op == "balance":
        G = _log(rng, 8, 256)
        return {"op": op, "T": _log(rng, 1, 65536), "G": G, "k": rng.randint(1, min(8, G)), "dtype": dtype,
                "masked": rng.randint(0, 1)}
    top = 2048 if dtype == "f32" else 4096
    M, N = _log(rng, 32, top), _log(rng, 32, top)
    small = min(M, N)
    B = _log(rng, 1, max(1, min(32, 2048 ** 3 // (small * small * max(M, N)))))
    return {"op": op, "B": B, "M": M, "N": N, "dtype": dtype}


# ------------------------------------------------------------------ inputs


def _quantized(shape, gen):
    """int8 rows as the quantisation of normal values gives them, and their scales."""
    q = torch.empty(shape, dtype=torch.int8, device="cuda")
    s = torch.empty(shape[0], device="cuda")
    for i in range(0, shape[0], 4096):
        x = torch.randn((min(4096, shape[0] - i), shape[1]), generator=gen, device="cuda")
        si = x.abs().amax(dim=1) / 127.0
        q[i:i + 4096] = torch.round(x / si[:, None]).to(torch.int8)
        s[i:i + 4096] = si
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], _DT[case["dtype"]]
    st = {"case": case}
    if op == "quantize":
        M, K = case["M"], case["K"]
        # tokens of different magnitude, and channels that stand out, as activations have them
        x = torch.randn((M, K), generator=gen, device="cuda")
        x *= torch.exp(0.5 * torch.randn((M, 1), generator=gen, device="cuda"))
        x *= 1.0 + 9.0 * (torch.rand(K, generator=gen, device="cuda") < 0.01)
        st["x"] = x.to(dt)
        st["q"] = torch.empty((M, K), dtype=torch.int8, device="cuda")
        st["s"] = torch.empty(M, device="cuda")
    elif op == "int8":
        M, K, N = case["M"], case["K"], case["N"]
        st["A"], st["sa"] = _quantized((M, K), gen)
        w, sb = _quantized((N, K), gen)
        st["B"] = w.t() if case["nk"] else w.t().contiguous()
        st["sb"] = sb / math.sqrt(K)
        st["bias"] = torch.randn(N, generator=gen, device="cuda").to(dt) if case["bias"] else None
        st["Y"] = torch.empty((M, N), dtype=dt, device="cuda")
    elif op == "balance":
        T, G, k = case["T"], case["G"], case["k"]
        logits = torch.randn((T, G), generator=gen, device="cuda").mul_(1.5)
        if case["masked"]:
            off = torch.rand((T, G), generator=gen, device="cuda") < 0.25
            off[torch.rand(T, generator=gen, device="cuda") < 0.05] = True     # padding
            logits = logits.masked_fill(off, -math.inf)
        st["logits"] = logits.to(dt)
        best, idx = st["logits"].float().topk(k, dim=1)
        st["idx"] = torch.where(best > -math.inf, idx, -1).to(torch.int32).contiguous()
        # of a loss summed over the tokens; the other gradient is the one through the picks' weights
        st["dloss"] = torch.full((1,), 0.01 * T, device="cuda")
        st["base"] = torch.randn((T, G), generator=gen, device="cuda").mul_(0.01).to(dt)
        st["loss"] = torch.empty(1, device="cuda")
        st["counts"] = torch.empty(G + 1, dtype=torch.int32, device="cuda")
        st["probs"] = torch.empty(G, device="cuda")
        st["dlogits"] = torch.empty((T, G), dtype=dt, device="cuda")
    else:
        B, M, N = case["B"], case["M"], case["N"]
        # a momentum: a few strong directions over noise
        r = min(8, M, N)
        u = torch.randn((B, M, r), generator=gen, device="cuda")
        v = torch.randn((B, r, N), generator=gen, device="cuda")
        g = torch.randn((B, M, N), generator=gen, device="cuda")
        g += (u * 0.5 ** torch.arange(r, device="cuda")) @ v
        st["G"] = g.mul_(1e-3).to(dt)
        if B == 1:
            st["G"] = st["G"][0]
        st["X"] = torch.empty_like(st["G"])
        st["scale"] = math.sqrt(max(1.0, M / N))
    if own:
        import quantized_gemm_gb300 as qg
        nbytes = 0
        if op == "int8":
            nbytes = qg.mm_int8_matmul_workspace_size(st["A"], st["B"], dt)
        elif op == "balance":
            nbytes = qg.mm_route_balance_workspace_size(st["logits"], st["idx"])
        elif op == "orth":
            nbytes = qg.mm_orthogonalize_workspace_size(st["G"])
        st["ws"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None
    return st


# ------------------------------------------------------------------ one pass


def _plain_quantize(x):
    xf = x.float()
    top = xf.abs().amax(dim=1)
    s = top / torch.full_like(top, 127.0)      # a rounded quotient: by a number, torch multiplies by its reciprocal
    q = torch.round(xf / torch.where(s == 0, 1.0, s)[:, None])
    return torch.clamp(q, -127, 127).to(torch.int8), s


def _plain_int8(A, B, sa, sb, bias, dt):
    y = (A.float() @ B.float()) * sa[:, None] * sb
    if bias is not None:
        y = y + bias.float()
    return y.to(dt)


def _plain_balance(logits, idx, dloss, base):
    T, G = logits.shape
    l = logits.float()
    top = l.amax(dim=1, keepdim=True)
    alive = top > -math.inf
    e = torch.where(alive, torch.exp(l - torch.where(alive, top, 0.0)), 0.0)
    total = e.sum(dim=1, keepdim=True)
    p = e / torch.where(alive, total, 1.0)
    at = torch.arange(G, device=l.device)
    counts = (idx.reshape(-1, 1, idx.shape[1]) == at[None, :, None]).sum(dim=(0, 2))
    rows = alive.sum()
    picks = counts.sum().float().clamp(min=1)
    live = rows.float().clamp(min=1)
    mean = p.sum(dim=0) / live
    share = counts.float() / picks
    loss = G * (share * mean).sum()
    d = dloss * (G / live) * p * (share - (share * p).sum(dim=1, keepdim=True))
    all_counts = torch.cat([counts, rows.view(1)]).to(torch.int32)
    return loss.view(1), all_counts, mean, (base.float() + d).to(logits.dtype)


def _plain_orth(g, steps, scale):
    a, b, c = _COEFFICIENTS
    x = g.float()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.transpose(-2, -1)
    x = x / (x.pow(2).sum(dim=(-2, -1), keepdim=True).sqrt() + _EPS)
    for _ in range(steps):
        A = x @ x.transpose(-2, -1)
        x = a * x + (b * A + c * (A @ A)) @ x
    if tall:
        x = x.transpose(-2, -1)
    return (scale * x).to(g.dtype).contiguous()


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import quantized_gemm_gb300 as qg
        if op == "quantize":
            return qg.mm_quantize_rows(s["x"], out=s["q"], scales=s["s"])
        if op == "int8":
            return qg.mm_int8_matmul(s["A"], s["B"], s["sa"], s["sb"], s["bias"], out=s["Y"], workspace=s["ws"])
        if op == "balance":
            loss, counts, probs = qg.mm_route_balance(s["logits"], s["idx"], loss=s["loss"], counts=s["counts"],
                                                      mean_probs=s["probs"], workspace=s["ws"])
            return loss, counts, probs, qg.mm_route_balance_grad(s["logits"], counts, s["dloss"], base=s["base"],
                                                                 out=s["dlogits"])
        return qg.mm_orthogonalize(s["G"], steps=5, coefficients=_COEFFICIENTS, eps=_EPS, scale=s["scale"],
                                   out=s["X"], workspace=s["ws"])
    if op == "quantize":
        return _plain_quantize(s["x"])
    if op == "int8":
        return _plain_int8(s["A"], s["B"], s["sa"], s["sb"], s["bias"], s["Y"].dtype)
    if op == "balance":
        return _plain_balance(s["logits"], s["idx"], s["dloss"], s["base"])
    return _plain_orth(s["G"], 5, s["scale"])


# ------------------------------------------------------------------ work of one pass


def work(case):
    op, e = case["op"], _SIZE[case["dtype"]]
    if op == "quantize":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * (e + 1) + 4 * M, "flops": 3 * M * K}
    if op == "int8":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": M * K + K * N + M * N * e + 4 * (M + N) + (N * e if case["bias"] else 0),
                "flops": 2 * M * K * N}
    if op == "balance":
        T, G, k = case["T"], case["G"], case["k"]
        # the logits once; the gradient cannot start before the counts are known, but a small batch stays on the chip
        return {"bytes": 3 * T * G * e + 4 * T * k + 8 * G, "flops": 12 * T * G}
    B, M, N = case["B"], case["M"], case["N"]
    m, n = min(M, N), max(M, N)
    # X X^T and its square are symmetric: half of each is enough
    return {"bytes": 2 * B * M * N * e, "flops": B * 5 * (3 * m * m * n + m ** 3)}


# ------------------------------------------------------------------ fp64


def _exact_balance(st):
    l = st["logits"].double().cpu().numpy()
    idx = st["idx"].cpu().numpy()
    T, G = l.shape
    alive = (l > -np.inf).any(axis=1)
    p = np.zeros_like(l)
    z = np.exp(l[alive] - l[alive].max(axis=1, keepdims=True))
    p[alive] = z / z.sum(axis=1, keepdims=True)
    counts = np.bincount(idx[idx >= 0].ravel(), minlength=G)
    rows = int(alive.sum())
    mean = p.sum(axis=0) / max(1, rows)
    share = counts / max(1, counts.sum())
    loss = np.array([G * float(share @ mean)])
    grad = float(st["dloss"].double().item()) * G / max(1, rows) * p * (share - (p @ share)[:, None])
    return loss, np.append(counts, rows).astype(np.int32), mean, st["base"].double().cpu().numpy() + grad


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        # the scale in fp64; the whole numbers follow the scale that is returned, in fp32, so they have no fp64 value
        return None, st["x"].double().abs().amax(dim=1) / 127.0
    if op == "int8":
        y = st["A"].double() @ st["B"].double()
        y *= st["sa"].double()[:, None] * st["sb"].double()[None, :]
        return y if st["bias"] is None else y.add_(st["bias"].double())
    if op == "balance":
        return _exact_balance(st)
    a, b, c = _COEFFICIENTS
    x = st["G"].double()
    x = x / (torch.linalg.matrix_norm(x, keepdim=True) + _EPS)
    wide = case["M"] <= case["N"]
    eye = torch.eye(min(case["M"], case["N"]), dtype=torch.float64, device="cuda")
    for _ in range(5):
        gram = x @ x.mT if wide else x.mT @ x
        poly = a * eye + gram @ (b * eye + c * gram)
        x = poly @ x if wide else x @ poly
    return st["scale"] * x
