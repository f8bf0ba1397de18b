"""What the training operators around the ternary layers are measured on.

Two operators: the softmax cross entropy of an output head over its whole
vocabulary, with its gradient, and the Newton-Schulz orthogonalisation of a
weight update.  `run` computes each in plain torch operations, or through the
framework's entry points when `own` is true.
"""
import math

import torch

own = False

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7


# ------------------------------------------------------------------- cases

def _head(name, op, M, V, K):
    return {"name": name, "op": op, "M": M, "V": V, "K": K}


def _update(name, B, N, K, dtype, kind):
    return {"name": name, "op": "orthogonalize", "B": B, "N": N, "K": K, "dtype": dtype,
            "kind": kind}


def listed():
    return [
        # the log-probability of one sampled token under a 32k-entry head
        _head("score_one_token", "loss", 1, 32000, 4096),
        # rescoring a decode batch at the smallest model's width
        _head("score_batch", "loss", 16, 32000, 3200),
        # perplexity of a ragged document, a vocabulary of no round size
        _head("eval_ragged", "loss", 777, 50021, 2568),
        # perplexity over full-length batches, a large vocabulary
        _head("eval_long", "loss", 8192, 128000, 4096),
        # a fine-tuning step on a handful of tokens
        _head("train_few_tokens", "loss_grad", 64, 32000, 2048),
        # a packed batch of ragged sequences
        _head("train_ragged", "loss_grad", 1999, 50021, 1608),
        # a training step on full-length sequences, a large vocabulary
        _head("train_long", "loss_grad", 8192, 128000, 4096),
        # the update of one small adapter-sized matrix, where launches count
        _update("update_small", 1, 128, 128, "f32", "flat"),
        # a stack of per-head blocks in one call
        _update("update_stack", 16, 256, 512, "bf16", "flat"),
        # a key/value projection, whose gradient is nearly low rank
        _update("update_kv", 1, 1024, 4096, "f32", "lowrank"),
        # a tall matrix of odd sizes
        _update("update_tall_odd", 1, 2731, 1001, "bf16", "flat"),
        # the widest feed-forward matrix
        _update("update_ffn", 1, 8192, 28672, "f32", "lowrank"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "loss_grad", "orthogonalize"])
    if op == "orthogonalize":
        B = rng.choice([1, 1, 1, 2, 3, 7])
        N, K = _spread(rng, 8, 8192), _spread(rng, 8, 8192)
        while B * min(N, K) ** 2 * max(N, K) > 2 ** 39:
            B = 1
            N, K = max(1, N // 2), max(1, K // 2)
        return {"op": op, "B": B, "N": N, "K": K, "dtype": rng.choice(["f32", "bf16"]),
                "kind": rng.choice(["flat", "lowrank"])}
    M, V = _spread(rng, 1, 8192), _spread(rng, 1000, 128000)
    K = 8 * _spread(rng, 32, 512)
    return {"op": op, "M": M, "V": V, "K": K}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if case["op"] == "orthogonalize":
        B, N, K = case["B"], case["N"], case["K"]
        U = rand(B, N, K)
        if case["kind"] == "lowrank":
            # a few strong directions over a floor of noise, as gradients have
            U = 0.05 * U + rand(B, N, 8) @ rand(B, 8, K)
        U = 1e-3 * U
        U = U if case["dtype"] == "f32" else U.bfloat16()
        return {"op": "orthogonalize", "U": U if B > 1 else U[0]}
    M, V, K = case["M"], case["V"], case["K"]
    W = (0.02 * rand(V, K)).bfloat16()
    targets = torch.randint(0, V, (M,), generator=g, device="cuda")
    # normalised hidden states that lean, more or less, towards their target's row
    lean = 8 * torch.rand((M, 1), generator=g, device="cuda")
    rows = W[targets].float()
    x = rand(M, K) + lean * rows / rows.square().sum(1, keepdim=True).sqrt()
    x = (x / x.square().mean(1, keepdim=True).sqrt()).bfloat16()
    state = {"op": case["op"], "x": x, "W": W}
    if M > 1:  # padding and prompt tokens carry no loss
        skip = torch.rand((M,), generator=g, device="cuda") < 0.05
        skip[0] = False
        targets = torch.where(skip, -100, targets)
    state["targets"] = targets
    if case["op"] == "loss_grad":
        valid = (targets >= 0).sum()
        state["dloss"] = torch.full((M,), 1.0, device="cuda") / valid
    return state


# -------------------------------------------------------------- plain forms

def _plain_loss(x, W, targets):
    z = x.float() @ W.float().T
    top = z.amax(1, keepdim=True)
    lse = top[:, 0] + (z - top).exp().sum(1).log()
    valid = (targets >= 0) & (targets < W.shape[0])
    at = torch.where(valid, targets, 0)
    loss = torch.where(valid, lse - z.gather(1, at[:, None])[:, 0], 0.0)
    return z, lse, loss, valid, at


def _plain_grad(x, W, targets, dloss):
    z, lse, loss, valid, at = _plain_loss(x, W, targets)
    p = z.sub_(lse[:, None]).exp_()
    p[torch.arange(x.shape[0], device=x.device), at] -= 1.0
    p *= torch.where(valid, dloss, 0.0)[:, None]
    dx = (p @ W.float()).to(x.dtype)
    dW = (p.T @ x.float()).to(W.dtype)
    return {"loss": loss, "dx": dx, "dW": dW}


def _plain_orthogonalize(U):
    a, b, c = COEFFICIENTS
    X = U.float()
    tall = X.shape[-2] > X.shape[-1]
    X = X.mT if tall else X
    X = X / (X.square().sum((-2, -1), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return (X.mT if tall else X).bfloat16().contiguous()


def run(state):
    if own:
        import ternary_quantized_linear_b200 as tql
        if state["op"] == "orthogonalize":
            return tql.bitnet_orthogonalize(state["U"], steps=STEPS, coefficients=COEFFICIENTS,
                                            eps=EPS)
        x, W, targets = state["x"], state["W"], state["targets"]
        loss, lse = tql.bitnet_cross_entropy_forward(x, W, targets)
        if state["op"] == "loss":
            return {"loss": loss, "lse": lse}
        dx, dW = tql.bitnet_cross_entropy_backward(x, W, targets, lse, state["dloss"])
        return {"loss": loss, "dx": dx, "dW": dW}
    if state["op"] == "orthogonalize":
        return _plain_orthogonalize(state["U"])
    if state["op"] == "loss":
        _, lse, loss, _, _ = _plain_loss(state["x"], state["W"], state["targets"])
        return {"loss": loss, "lse": lse}
    return _plain_grad(state["x"], state["W"], state["targets"], state["dloss"])


# --------------------------------------------------------------------- work

def work(case):
    if case["op"] == "orthogonalize":
        B, n, k = case["B"], min(case["N"], case["K"]), max(case["N"], case["K"])
        size = 4 if case["dtype"] == "f32" else 2
        # A and A A are symmetric: half of each product
        return {"bytes": B * n * k * (size + 2),
                "flops": B * STEPS * (n * n * k + n * n * n + 2 * n * n * k)}
    M, V, K = case["M"], case["V"], case["K"]
    if case["op"] == "loss":
        return {"bytes": 2 * K * (M + V) + 16 * M, "flops": 2 * M * V * K}
    # the gradient is a call of its own: it reads x and W, computes the logits
    # again from them and the saved statistics, and writes both gradients
    return {"bytes": 2 * 2 * K * (M + V) + 2 * K * (M + V) + 36 * M, "flops": 8 * M * V * K}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "orthogonalize":
        a, b, c = COEFFICIENTS
        X = s["U"].double()
        X = X / (torch.linalg.vector_norm(X, dim=(-2, -1), keepdim=True) + EPS)
        tall = X.shape[-2] > X.shape[-1]
        for _ in range(STEPS):
            if tall:
                G = X.mT @ X
                X = X @ (c * G @ G + b * G + a * torch.eye(G.shape[-1], device=G.device,
                                                           dtype=G.dtype))
            else:
                G = X @ X.mT
                X = (c * G @ G + b * G + a * torch.eye(G.shape[-1], device=G.device,
                                                       dtype=G.dtype)) @ X
        return X
    x, W, t = s["x"].double(), s["W"].double(), s["targets"]
    M, V = x.shape[0], W.shape[0]
    loss, lse, dx = [], [], []
    dW = torch.zeros_like(W) if case["op"] == "loss_grad" else None
    for i in range(0, M, 1024):
        xi, ti = x[i:i + 1024], t[i:i + 1024]
        z = xi @ W.T
        l = torch.logsumexp(z, 1)
        ok = (ti >= 0) & (ti < V)
        j = ti.clamp(0, V - 1)
        r = torch.arange(xi.shape[0], device=x.device)
        lse.append(l)
        loss.append(torch.where(ok, l - z[r, j], 0.0))
        if dW is not None:
            g = torch.exp(z - l[:, None])
            g[r, j] -= 1.0
            g *= (s["dloss"][i:i + 1024].double() * ok)[:, None]
            dx.append(g @ W)
            dW += g.T @ xi
    if dW is None:
        return {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    return {"loss": torch.cat(loss), "dx": torch.cat(dx), "dW": dW}
