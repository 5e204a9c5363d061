"""What a quantisation-aware training step needs around the compressed layers, as cases to be timed.

Operators: the token embedding (lookup with scaling) and its gradient, the softmax cross entropy of hidden states
against a vocabulary matrix (loss alone, and loss with the gradients of both), and the Newton-Schulz
orthogonalisation of the latent factors' gradients.  ``own`` chooses between the plain form (elementary torch
operations in float32) and the library's calls.
"""

import math

import torch

own = False

COEFFS = (3.4445, -4.7750, 2.0315)   # the quintic of the orthogonalisation
EPS = 1e-7

_DT = {"float32": torch.float32, "bfloat16": torch.bfloat16}


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a training micro-batch of 8192 tokens into the 7B-shaped model
        {"name": "embed_batch", "op": "embed", "M": 8192, "D": 4096, "V": 32000, "scale": 1.0, "dtype": "bfloat16"},
        # one decoding step of 16 sequences of the 70B-shaped model, scaled embeddings
        {"name": "embed_step", "op": "embed", "M": 16, "D": 8192, "V": 32000, "scale": 90.5, "dtype": "bfloat16"},
        # the gradient of the first, from the layers' float32 dx into a float32 table gradient
        {"name": "embed_grad_batch", "op": "embed_grad", "M": 8192, "D": 4096, "V": 32000, "scale": 1.0,
         "dtype": "float32", "out": "float32"},
        # a short ragged batch of a small model with two added tokens, bfloat16 in and out
        {"name": "embed_grad_ragged", "op": "embed_grad", "M": 1237, "D": 1160, "V": 32002, "scale": 34.06,
         "dtype": "bfloat16", "out": "bfloat16"},
        # scoring the last positions of 16 sequences: the vocabulary matrix is read once, latency and bandwidth
        {"name": "loss_few_rows", "op": "loss", "M": 16, "D": 8192, "V": 32000},
        # evaluation (perplexity) of one 2048-token window of the 13B-shaped model
        {"name": "loss_window", "op": "loss", "M": 2048, "D": 5120, "V": 32000},
        # a training micro-batch of the 7B-shaped model, vocabulary matrix trained
        {"name": "loss_grad_batch", "op": "loss_grad", "M": 4096, "D": 4096, "V": 32000, "head": True},
        # a ragged batch of a small model whose vocabulary matrix is frozen: only the hidden states' gradient
        {"name": "loss_grad_ragged_frozen", "op": "loss_grad", "M": 777, "D": 1160, "V": 32003, "head": False},
        # a vocabulary four times as large
        {"name": "loss_grad_wide", "op": "loss_grad", "M": 4096, "D": 4096, "V": 128256, "head": True},
        # the latent gradients of the smallest layer: U and V of both paths
        {"name": "orth_layer_512", "op": "orth", "shapes": "512x16*4", "dtype": "float32"},
        # odd sizes and a wide one, bfloat16 gradients
        {"name": "orth_odd", "op": "orth", "shapes": "5120x368*2+1001x333+200x1500", "dtype": "bfloat16"},
        # every latent gradient of one block of the 7B-shaped model at 0.55 bits per weight
        {"name": "orth_block", "op": "orth", "shapes": "4096x544*16+11008x800*6+4096x800*6", "dtype": "float32"},
    ]


def _log_int(rng, lo, hi, step=1):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(step, min(hi, n // step * step))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "loss", "loss_grad", "orth"])
    if op in ("embed", "embed_grad"):
        c = {"op": op, "M": _log_int(rng, 1, 8192), "D": _log_int(rng, 64, 8192), "V": _log_int(rng, 500, 130000),
             "scale": rng.choice([1.0, 11.5]), "dtype": rng.choice(["bfloat16", "float32"])}
        if op == "embed_grad":
            c["V"] = min(c["V"], (1 << 29) // c["D"])
            c["out"] = rng.choice(["bfloat16", "float32"])
        return c
    if op in ("loss", "loss_grad"):
        D = _log_int(rng, 128, 8192, 8)
        V = _log_int(rng, 500, 130000)
        M = min(_log_int(rng, 1, 8192), max(1, 4096 * 4096 * 128256 // (D * V)))
        c = {"op": op, "M": M, "D": D, "V": V}
        if op == "loss_grad":
            c["head"] = rng.random() < 0.7
        return c
    parts = []
    for _ in range(rng.randint(1, 3)):
        rows, cols = _log_int(rng, 64, 14000), _log_int(rng, 8, 800)
        if rng.random() < 0.2:
            rows, cols = cols, rows
        parts.append("%dx%d*%d" % (rows, cols, rng.randint(1, 4)))
    return {"op": "orth", "shapes": "+".join(parts), "dtype": rng.choice(["float32", "bfloat16"])}


def _shapes(text):
    out = []
    for part in text.split("+"):
        size, _, n = part.partition("*")
        r, c = size.split("x")
        out += [(int(r), int(c))] * int(n or 1)
    return out


# ------------------------------------------------------------------------------------------------ inputs

def _tokens(g, M, V, ignored):
    """Token numbers as text has them: a few very frequent ones, a long tail, and some positions without one."""
    u = torch.rand(M, generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(V + 1.0)) - 1.0).to(torch.int64).clamp_(0, V - 1)
    ids = (ids * 7919 + 13) % V if V % 7919 else ids
    if M >= 8:
        n = M // 16
        ids[M - n:] = ignored
    return ids


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    st = {"op": op, "case": case}

    def randn(*size):
        return torch.randn(*size, generator=g, device="cuda")

    if op == "embed":
        st["table"] = (randn(case["V"], case["D"]) * 0.02).to(_DT[case["dtype"]])
        st["ids"] = _tokens(g, case["M"], case["V"], -1)
    elif op == "embed_grad":
        st["ids"] = _tokens(g, case["M"], case["V"], -1)
        st["dout"] = (randn(case["M"], case["D"]) * 1e-3).to(_DT[case["dtype"]])
    elif op in ("loss", "loss_grad"):
        M, D, V = case["M"], case["D"], case["V"]
        W = (randn(V, D) * 0.02).to(torch.bfloat16)
        labels = _tokens(g, M, V, -100)
        h = randn(M, D)
        # hidden states of a model that has learnt something: the label's logit stands out, more in some rows
        gain = 8.0 * torch.rand(M, 1, generator=g, device="cuda")
        w = W[labels.clamp(min=0)].float()
        h += gain * w / w.norm(dim=1, keepdim=True)
        st["H"], st["W"], st["labels"] = h.to(torch.bfloat16), W, labels
        if op == "loss_grad":
            valid = (labels >= 0).float()
            st["weight"] = valid / valid.sum().clamp(min=1.0)     # mean over the positions that count
    else:
        mats = []
        for m, n in _shapes(case["shapes"]):
            t = min(64, m, n)
            decay = 1.0 / torch.arange(1, t + 1, device="cuda", dtype=torch.float32)
            G = (randn(m, t) * decay) @ randn(t, n) + 0.05 * randn(m, n)
            u = randn(m, n) * 0.01
            G = 1e-4 * torch.exp(0.5 * randn(m, 1)) * G * (1.0 - torch.tanh(100.0 * u) ** 2)
            mats.append(G.to(_DT[case["dtype"]]))
        st["G"] = mats
    return st


# ------------------------------------------------------------------------------------------------ one pass

def _own(st):
    from sub_bit_weight_b200 import lib
    c, op = st["case"], st["op"]
    if op == "embed":
        return lib.lb_embedding_forward(st["ids"], st["table"], scale=c["scale"])
    if op == "embed_grad":
        return lib.lb_embedding_backward(st["ids"], st["dout"], c["V"], scale=c["scale"], dtype=_DT[c["out"]])
    if op == "loss":
        return lib.lb_cross_entropy_forward(st["H"], st["W"], st["labels"])
    if op == "loss_grad":
        loss, dH, dW = lib.lb_cross_entropy_gradient(st["H"], st["W"], st["labels"], st["weight"], head=c["head"])
        return (loss, dH, dW) if c["head"] else (loss, dH)
    return lib.lb_orthogonalise(st["G"])


def _plain_orth(G):
    a, b, c = COEFFS
    X = G.float()
    wide = X.shape[0] < X.shape[1]
    if wide:
        X = X.T
    X = X / (X.norm() + EPS)
    for _ in range(5):
        A = X.T @ X
        X = a * X + X @ (b * A + c * (A @ A))
    return (X.T if wide else X).to(torch.bfloat16).contiguous()


def run(state):
    if own:
        return _own(state)
    c, op = state["case"], state["op"]
    if op == "embed":
        ids, T = state["ids"], state["table"]
        ok = (ids >= 0) & (ids < c["V"])
        rows = T[torch.where(ok, ids, 0)].float() * c["scale"]
        return torch.where(ok[:, None], rows, 0.0).to(T.dtype)
    if op == "embed_grad":
        ids = state["ids"]
        ok = (ids >= 0) & (ids < c["V"])
        d = torch.zeros(c["V"] + 1, c["D"], device=ids.device)
        d.index_add_(0, torch.where(ok, ids, c["V"]), state["dout"].float())
        return (d[:-1] * c["scale"]).to(_DT[c["out"]])
    if op in ("loss", "loss_grad"):
        H, W, labels = state["H"].float(), state["W"].float(), state["labels"]
        z = H @ W.T
        ok = (labels >= 0) & (labels < c["V"])
        at = torch.where(ok, labels, 0)[:, None]
        top = z.max(dim=1, keepdim=True).values
        e = torch.exp(z - top)
        s = e.sum(dim=1, keepdim=True)
        lse = (top + torch.log(s))[:, 0]
        loss = torch.where(ok, lse - z.gather(1, at)[:, 0], 0.0)
        if op == "loss":
            return loss, lse
        w = torch.where(ok, state["weight"], 0.0)[:, None]
        P = e / s
        P.scatter_add_(1, at, torch.full_like(w, -1.0))
        P *= w
        dH = (P @ W).to(torch.bfloat16)
        return (loss, dH, (P.T @ H).to(torch.bfloat16)) if c["head"] else (loss, dH)
    return [_plain_orth(G) for G in state["G"]]


# ------------------------------------------------------------------------------------------------ least work

def work(case):
    op = case["op"]
    size = {"float32": 4, "bfloat16": 2}
    if op == "embed":
        rows = case["M"] * case["D"]
        return {"bytes": 8 * case["M"] + 2 * rows * size[case["dtype"]], "flops": rows}
    if op == "embed_grad":
        rows = case["M"] * case["D"]
        return {"bytes": 8 * case["M"] + rows * size[case["dtype"]] + case["V"] * case["D"] * size[case["out"]],
                "flops": rows}
    if op in ("loss", "loss_grad"):
        M, D, V = case["M"], case["D"], case["V"]
        read = 2 * D * (M + V) + 8 * M
        if op == "loss":
            return {"bytes": read + 8 * M, "flops": 2 * M * V * D}
        head = case["head"]
        return {"bytes": read + 8 * M + 2 * M * D + (2 * V * D if head else 0), "flops": (6 if head else 4) * M * V * D}
    nbytes = flops = 0
    for r, c in _shapes(case["shapes"]):
        m, n = max(r, c), min(r, c)
        nbytes += m * n * (size[case["dtype"]] + 2)
        # X0^T X0 (symmetric), the polynomial's symmetric n x n products (two a step), and X0 times their result
        flops += m * n * n + 5 * 2 * n ** 3 + 2 * m * n * n
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    op = case["op"]
    if op in ("loss", "loss_grad"):
        if 6 * case["M"] * case["V"] * case["D"] > 2.5e14:
            return None
    elif op == "orth":
        if sum(20 * r * c * min(r, c) for r, c in _shapes(case["shapes"])) > 2.5e14:
            return None
    st = prepare(case, seed)
    d = torch.float64
    if op == "embed":
        out = torch.zeros(case["M"], case["D"], dtype=d, device="cuda")
        seen = torch.nonzero(st["ids"] >= 0)[:, 0]
        out[seen] = st["table"].to(d)[st["ids"][seen]] * case["scale"]
        return out
    if op == "embed_grad":
        # sums by sorted tokens: differences of a running sum in 64 bits lose too much, so one row at a time by matrix
        seen = torch.nonzero(st["ids"] >= 0)[:, 0]
        which, back = torch.unique(st["ids"][seen], return_inverse=True)
        out = torch.zeros(case["V"], case["D"], dtype=d, device="cuda")
        sums = torch.zeros(which.numel(), case["D"], dtype=d, device="cuda")
        sums.index_add_(0, back, st["dout"][seen].to(d))
        out[which] = sums * case["scale"]
        return out
    if op in ("loss", "loss_grad"):
        H, W, labels = st["H"].to(d), st["W"].to(d), st["labels"]
        logits = torch.einsum("md,vd->mv", H, W)
        lse = torch.logsumexp(logits, dim=1)
        counts = labels >= 0
        target = (H * W[labels.clamp(min=0)]).sum(dim=1)
        loss = torch.zeros_like(lse)
        loss[counts] = (lse - target)[counts]
        if op == "loss":
            return loss, lse
        G = torch.exp(logits - lse[:, None])
        del logits
        G[torch.arange(G.shape[0], device="cuda")[counts], labels[counts]] -= 1.0
        G = G * (st["weight"].to(d) * counts)[:, None]
        dH = torch.einsum("mv,vd->md", G, W)
        return (loss, dH, torch.einsum("mv,md->vd", G, H)) if case["head"] else (loss, dH)
    out = []
    a, b, c = COEFFS
    for G in st["G"]:
        X = G.to(d)
        X = X / (torch.sqrt((X * X).sum()) + EPS)
        for _ in range(5):
            if X.shape[0] >= X.shape[1]:
                A = X.T @ X
                X = a * X + b * (X @ A) + c * (X @ A @ A)
            else:
                A = X @ X.T
                X = a * X + b * (A @ X) + c * (A @ A @ X)
        out.append(X)
    return out
