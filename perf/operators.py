"""The loss head and the Muon update as measured operators: cases, plain forms, exact values.

Four operators of the training step around a Linear layer:

  xent       loss and log-sum-exp of a language-model head, from X [M,K], W [K,V] and targets,
             without storing the logits (lin_xent)
  xent_bwd   its gradients dX and dW (lin_xent_bwd)
  orth       Newton-Schulz orthogonalisation of a batch of matrices (muon_orth)
  muon       momentum + orthogonalisation + weight update (muon_step)

With ``own`` false, run() computes them in elementary float32 torch operations; with ``own``
true it calls this repository's library.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
IGNORED = -100          # target of a row that takes no part in the loss
LOSS_SCALE = 1024.0     # the loss scale of the repository's mixed-precision workload
NS = (3.4445, -4.7750, 2.0315)   # coefficients of the Newton-Schulz polynomial
STEPS = 5
LR, BETA, DECAY = 3e-4, 0.95, 0.1


def listed():
    return [
        # the loss of one token: scoring during decoding, latency
        dict(name="xent 1 row", op="xent", M=1, K=1024, V=32000, dtype="bf16"),
        # a decode-sized batch against a wide head: the weights are read once
        dict(name="xent 32 rows", op="xent", M=32, K=4096, V=65536, dtype="bf16"),
        # an evaluation batch with a vocabulary that is no multiple of anything
        dict(name="xent odd vocabulary", op="xent", M=777, K=2048, V=50257, dtype="f16"),
        # the head over one training batch (8 sequences of 2048 tokens)
        dict(name="xent batch", op="xent", M=16384, K=4096, V=32000, dtype="bf16"),
        # gradients of a handful of tokens: writing dW is the work
        dict(name="xent_bwd 16 rows", op="xent_bwd", M=16, K=1024, V=32000, dtype="bf16", weights=False),
        # a data-parallel shard with an odd vocabulary and weighted rows
        dict(name="xent_bwd odd vocabulary", op="xent_bwd", M=2048, K=4096, V=50257, dtype="bf16",
             weights=True),
        # fp16 training with a loss scale, a ragged batch
        dict(name="xent_bwd f16", op="xent_bwd", M=1000, K=2048, V=32000, dtype="f16", weights=False),
        # four sequences of 2048 tokens, the largest vocabulary
        dict(name="xent_bwd large", op="xent_bwd", M=8192, K=4096, V=131072, dtype="bf16", weights=False),
        # one small matrix: launches and latency
        dict(name="orth small", op="orth", B=1, K=256, N=256, dtype="f32", out="bf16"),
        # a stack of tall matrices of odd sizes
        dict(name="orth odd stack", op="orth", B=3, K=2050, N=515, dtype="f32", out="f16"),
        # the repository's QKV projection, bf16 gradients under the loss scale
        dict(name="muon projection", op="muon", B=1, K=4096, N=12288, dtype="bf16", copy=True),
        # twelve layers of a small model in one call
        dict(name="muon stack", op="muon", B=12, K=1024, N=1024, dtype="f32", copy=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["xent", "xent_bwd", "orth", "muon"])
    if op in ("xent", "xent_bwd"):
        c = dict(op=op, M=_log(rng, 1, 8192), K=_log(rng, 64, 4096), V=_log(rng, 100, 131072),
                 dtype=rng.choice(["bf16", "f16"]))
        if rng.random() < 0.6:               # widths are multiples of eight more often than not
            c["K"] = max(8, c["K"] // 8 * 8)
            c["V"] = c["V"] // 8 * 8
        if op == "xent_bwd":
            c["weights"] = rng.random() < 0.5
        return c
    c = dict(op=op, K=_log(rng, 32, 4096), N=_log(rng, 32, 8192))
    if rng.random() < 0.6:
        c["K"], c["N"] = c["K"] // 8 * 8, c["N"] // 8 * 8
    c["B"] = min(_log(rng, 1, 12), max(1, (1 << 24) // (c["K"] * c["N"])))
    c["dtype"] = rng.choice(["f32", "bf16", "f16"])
    if op == "orth":
        c["out"] = rng.choice(["bf16", "f16"])
    else:
        c["copy"] = rng.random() < 0.5
    return c


def work(case):
    if case["op"] in ("xent", "xent_bwd"):
        M, K, V, e = case["M"], case["K"], case["V"], SIZE[case["dtype"]]
        read = e * (M * K + K * V) + 8 * M
        if case["op"] == "xent":
            return {"bytes": read + 8 * M + 8, "flops": 2.0 * M * K * V}
        read += 4 * M + 4 + (4 * M if case["weights"] else 0)
        return {"bytes": read + e * (M * K + K * V), "flops": 6.0 * M * K * V}
    B, K, N = case["B"], case["K"], case["N"]
    s, t = min(K, N), max(K, N)
    # each step: a symmetric product s x s over t, the square of a symmetric matrix, a full product
    flops = B * STEPS * (float(s) * s * t + float(s) * s * s + 2.0 * s * s * t)
    n = B * K * N
    if case["op"] == "orth":
        return {"bytes": n * (SIZE[case["dtype"]] + SIZE[case["out"]]), "flops": flops}
    return {"bytes": n * (SIZE[case["dtype"]] + 16 + (2 if case["copy"] else 0)), "flops": flops}


# ---- inputs ----------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(shape, std, g, dtype=torch.float32):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g).to(dtype)


def _gradient(B, K, N, g):
    """A gradient's spectrum: noise, and a few strong directions of about the same energy."""
    r = min(8, K, N)
    noise = _normal((B, K, N), 1e-4, g)
    strong = torch.matmul(_normal((B, K, r), 1.0, g), _normal((B, r, N), 1e-4 / math.sqrt(r), g))
    return noise.add_(strong)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] in ("xent", "xent_bwd"):
        M, K, V, T = case["M"], case["K"], case["V"], TYPES[case["dtype"]]
        s["X"] = _normal((M, K), 1.0, g, T)
        s["W"] = _normal((K, V), 0.02, g, T)
        s["target"] = torch.randint(0, V, (M,), device=DEV, generator=g)
        if M > 1:                             # padding and prompt tokens carry no loss
            s["target"][torch.rand(M, device=DEV, generator=g) < 0.1] = IGNORED
        if case["op"] == "xent_bwd":          # what the forward pass left
            z = torch.matmul(s["X"].float(), s["W"].float())
            s["lse"] = torch.where(s["target"] >= 0, torch.logsumexp(z, 1), 0.0)
            del z
            s["inv_count"] = 1.0 / (s["target"] >= 0).sum().clamp(min=1).float().reshape(1)
            s["row_scale"] = torch.rand(M, device=DEV, generator=g) if case["weights"] else None
            s["dX"] = torch.empty((M, K), dtype=T, device=DEV)
            s["dW"] = torch.empty((K, V), dtype=T, device=DEV)
        return s
    B, K, N, T = case["B"], case["K"], case["N"], TYPES[case["dtype"]]
    if case["op"] == "orth":
        s["G"] = _gradient(B, K, N, g).to(T)
        return s
    s["scale"] = 0.2 * math.sqrt(max(K, N))   # an update of the size of AdamW's
    s["grad"] = (_gradient(B, K, N, g) * LOSS_SCALE).to(T)
    s["W"] = _normal((B, K, N), 0.02, g)
    s["mom"] = _gradient(B, K, N, g) * 3.0
    s["w16"] = torch.empty((B, K, N), dtype=torch.bfloat16, device=DEV) if case["copy"] else None
    return s


# ---- the operators -----------------------------------------------------------------------


def _plain_xent(s):
    z = torch.matmul(s["X"].float(), s["W"].float())
    counted = s["target"] >= 0
    top = z.max(1, keepdim=True).values
    lse = top[:, 0] + torch.exp(z - top).sum(1).log()
    at = z.gather(1, s["target"].clamp(min=0)[:, None])[:, 0]
    loss = torch.where(counted, lse - at, 0.0)
    count = counted.sum().float()
    inv = torch.where(count > 0, 1.0 / count, 0.0)
    out = torch.stack([loss.double().sum().float() * inv, inv])
    return {"loss": loss, "lse": torch.where(counted, lse, 0.0), "out": out}


def _plain_xent_bwd(s):
    W = s["W"].float()
    counted = s["target"] >= 0
    X = torch.where(counted[:, None], s["X"].float(), 0.0)
    scale = LOSS_SCALE * s["inv_count"] * torch.where(counted, 1.0, 0.0)
    if s["row_scale"] is not None:
        scale = scale * s["row_scale"]
    g = torch.exp(torch.matmul(X, W) - s["lse"][:, None])
    g.scatter_add_(1, s["target"].clamp(min=0)[:, None], -torch.ones_like(g[:, :1]))
    g *= scale[:, None]
    s["dX"].copy_(torch.matmul(g, W.t()))
    s["dW"].copy_(torch.matmul(X.t(), g))
    return {"dX": s["dX"], "dW": s["dW"]}


def _plain_orth(u):
    """Newton-Schulz in float32 for u [B, K, N], on the shorter side."""
    a, b, c = NS
    flip = u.shape[1] > u.shape[2]
    x = u.transpose(1, 2).contiguous() if flip else u
    norm = x.double().square().sum((1, 2), keepdim=True).sqrt()
    x = torch.where(norm > 0, x / norm, 0.0).float()
    for _ in range(STEPS):
        gram = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    return x.transpose(1, 2).contiguous() if flip else x


def _plain_muon(s):
    g = s["grad"].float() * (1.0 / LOSS_SCALE)
    s["mom"].mul_(BETA).add_(g)
    o = _plain_orth(g + BETA * s["mom"])
    s["W"].sub_(LR * (s["scale"] * o + DECAY * s["W"]))
    if s["w16"] is not None:
        s["w16"].copy_(s["W"])
    return _muon_outputs(s)


def _muon_outputs(s):
    got = {"W": s["W"], "mom": s["mom"]}
    if s["w16"] is not None:
        got["w16"] = s["w16"]
    return got


def run(s):
    if own:
        import linear_layer_backward_bwd_amd as lb
        if s["op"] == "xent":
            loss, lse, out = lb.lin_xent(s["X"], s["W"], s["target"])
            return {"loss": loss, "lse": lse, "out": out}
        if s["op"] == "xent_bwd":
            lb.lin_xent_bwd(s["X"], s["W"], s["target"], s["lse"], s["dX"], s["dW"], scale=LOSS_SCALE,
                            d_scale=s["inv_count"], row_scale=s["row_scale"])
            return {"dX": s["dX"], "dW": s["dW"]}
        if s["op"] == "orth":
            return lb.muon_orth(s["G"], dtype=TYPES[s["out"]], steps=STEPS)
        lb.muon_step(s["W"], s["grad"], s["mom"], LR, BETA, DECAY, s["scale"], steps=STEPS, nesterov=True,
                     inv_scale=1.0 / LOSS_SCALE, w16=s["w16"])
        return _muon_outputs(s)
    if s["op"] == "xent":
        return _plain_xent(s)
    if s["op"] == "xent_bwd":
        return _plain_xent_bwd(s)
    if s["op"] == "orth":
        return _plain_orth(s["G"].float()).to(TYPES[s["out"]])
    return _plain_muon(s)


# ---- 64-bit values -------------------------------------------------------------------------


def _polar(u):
    """The polynomial iteration on the singular values' side that is shorter, in float64."""
    a, b, c = NS
    y = u / torch.linalg.matrix_norm(u, keepdim=True).clamp(min=1e-300)
    tall = y.shape[-2] > y.shape[-1]
    for _ in range(STEPS):
        yt = y.mT.contiguous()
        if tall:
            s = yt @ y
            y = a * y + b * (y @ s) + c * ((y @ s) @ s)
        else:
            s = y @ yt
            y = a * y + b * (s @ y) + c * (s @ (s @ y))
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("xent", "xent_bwd"):
        kept = s["target"] != IGNORED
        row = torch.nonzero(kept)[:, 0]
        x, w, t = s["X"][row].double(), s["W"].double(), s["target"][row]
        logit = x @ w
        if case["op"] == "xent":
            full = logit.logsumexp(1)
            lse = torch.zeros(case["M"], dtype=torch.float64, device=DEV).index_copy_(0, row, full)
            each = full - logit[torch.arange(len(row), device=DEV), t]
            loss = torch.zeros_like(lse).index_copy_(0, row, each)
            n = len(row)
            out = torch.tensor([float(each.sum()) / n if n else 0.0, 1.0 / n if n else 0.0], dtype=torch.float64)
            return {"loss": loss, "lse": lse, "out": out}
        p = logit.sub_(s["lse"][row].double()[:, None]).exp_()
        p[torch.arange(len(row), device=DEV), t] -= 1.0
        weight = LOSS_SCALE * s["inv_count"].double().expand(len(row))
        if s["row_scale"] is not None:
            weight = weight * s["row_scale"][row].double()
        p.mul_(weight[:, None])
        dX = torch.zeros((case["M"], case["K"]), dtype=torch.float64, device=DEV)
        dX[row] = p @ w.mT
        return {"dX": dX, "dW": x.mT @ p}
    if case["op"] == "orth":
        return _polar(s["G"].double())
    g = s["grad"].double() / LOSS_SCALE
    mom = BETA * s["mom"].double() + g
    W = s["W"].double()
    W = W - LR * (s["scale"] * _polar(g + BETA * mom) + DECAY * W)
    got = {"W": W, "mom": mom}
    if s["w16"] is not None:
        got["w16"] = W
    return got
