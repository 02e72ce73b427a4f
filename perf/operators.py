"""Timing cases for the vocabulary-sized operators of a language model.

Three operators, each with the forms in which a program calls it:

stats   log-probabilities of given tokens with the entropy and the top
        alternatives of every row of logits (``lse_token_stats``); the
        ``train`` form adds the gradient (``lse_token_stats_backward``);
norm    the global norm of many gradient tensors (``lse_grad_norm``); the
        ``clip`` form writes the clipped gradients too (``lse_grad_clip``);
embed   rows of a table for given tokens, scaled (``lse_embedding``); the
        ``embgrad`` form returns the table's gradient (``lse_embedding_backward``).

``run`` makes one pass in plain torch operations, or, where ``own`` is set,
through this package.  ``exact`` computes the same results in 64 bits.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_EB = {"f32": 4, "bf16": 2, "f16": 2}
_EPS = 1e-6  # added to the norm before the division, as is usual for clipping


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One decoding step of one sequence, with the alternatives a client asks for.
        {"name": "stats-one-token", "op": "stats", "dtype": "bf16", "B": 1, "N": 128256, "K": 20},
        # A decoding step of a batch; an odd vocabulary, so rows start off 16-byte boundaries.
        {"name": "stats-decode-batch", "op": "stats", "dtype": "f16", "B": 48, "N": 50257, "K": 5},
        # Scoring the tokens of a prompt: many rows of the whole vocabulary.
        {"name": "stats-score-prompt", "op": "stats", "dtype": "bf16", "B": 2048, "N": 128256, "K": 20},
        # Many short rows: a byte vocabulary with a few special tokens.
        {"name": "stats-byte-rows", "op": "stats", "dtype": "f32", "B": 65536, "N": 261, "K": 8},
        # A policy-gradient step with an entropy term; prompt positions carry no gradient.
        {"name": "train-policy-step", "op": "train", "dtype": "bf16", "B": 4096, "N": 32000, "K": 0,
         "prompt": 0.25},
        # The same for a few f32 rows of an odd vocabulary, and the top alternatives' gradients.
        {"name": "train-top-alternatives", "op": "train", "dtype": "f32", "B": 96, "N": 100003, "K": 16,
         "prompt": 0.0},
        # Clipping the gradients of a small model: many small tensors, launch-bound.
        {"name": "clip-small-model", "op": "clip", "dtype": "f32", "tensors": 148, "total": 400000},
        # Clipping the gradients of a large model's layers.
        {"name": "clip-large-layers", "op": "clip", "dtype": "bf16", "tensors": 290, "total": 400000000},
        # The norm alone, for monitoring, over tensors of all three types and odd sizes.
        {"name": "norm-mixed-types", "op": "norm", "dtype": "mixed", "tensors": 75, "total": 90000003},
        # The lookup of one decoding step.
        {"name": "embed-decode-batch", "op": "embed", "dtype": "bf16", "V": 128256, "D": 2048, "T": 64},
        # The lookup of a training batch, odd width in f32.
        {"name": "embed-odd-width", "op": "embed", "dtype": "f32", "V": 50257, "D": 1001, "T": 20000},
        # The table's gradient for a training batch: few tokens are very frequent.
        {"name": "embgrad-train-batch", "op": "embgrad", "dtype": "bf16", "V": 128256, "D": 2048,
         "T": 32768},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["stats", "stats", "train", "train", "clip", "norm", "embed", "embgrad"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op in ("stats", "train"):
        most = 120_000_000 if op == "stats" else 60_000_000  # elements
        N = _log_int(rng, 200, 262144)
        B = _log_int(rng, 1, max(1, min(131072, most // N)))
        K = rng.choice([0, 1, 5, 8, 20, 32]) if op == "stats" else rng.choice([0, 0, 4, 16])
        c = {"op": op, "dtype": dtype, "B": B, "N": N, "K": K}
        if op == "train":
            c["prompt"] = rng.choice([0.0, 0.25, 0.5])
        return c
    if op in ("clip", "norm"):
        if op == "norm":
            dtype = rng.choice([dtype, "mixed"])
        tensors = _log_int(rng, 1, 600)
        return {"op": op, "dtype": dtype, "tensors": tensors,
                "total": _log_int(rng, max(20000, 40 * tensors), 200_000_000)}
    V = _log_int(rng, 300, 200000)
    D = _log_int(rng, 64, 8192)
    if rng.random() < 0.7:
        D = D // 64 * 64
    D += 128 * (D == 3 << 10)
    while V * D > 250_000_000:
        V = V // 2 + 1
    T = _log_int(rng, 1, min(65536, max(2, 60_000_000 // D)))
    return {"op": op, "dtype": dtype, "V": V, "D": D, "T": T}


def work(case):
    op = case["op"]
    if op in ("stats", "train"):
        n, eb, B = case["B"] * case["N"], _EB[case["dtype"]], case["B"]
        rows = B * (8 + 12 + 12 * case["K"])
        if op == "stats":
            return {"bytes": n * eb + rows, "flops": 6 * n}
        return {"bytes": 2 * n * eb + rows + B * (8 + 4 * case["K"]), "flops": 14 * n}
    if op in ("clip", "norm"):
        size = sum(k * _EB[d] for k, d in _tensor_list(case))
        total = sum(k for k, _ in _tensor_list(case))
        return {"bytes": size + 4, "flops": 2 * total} if op == "norm" else \
            {"bytes": 2 * size + 4, "flops": 3 * total}
    V, D, T, eb = case["V"], case["D"], case["T"], _EB[case["dtype"]]
    if op == "embed":
        return {"bytes": 2 * T * D * eb + 8 * T, "flops": T * D}
    return {"bytes": (T + V) * D * eb + 8 * T, "flops": T * D + V * D}


def _tensor_list(case):
    """(elements, type) of every tensor: as in a model, a few large ones next to
    many short vectors, with odd sizes among them."""
    n, total = case["tensors"], case["total"]
    types = ["f32", "bf16", "f16"] if case["dtype"] == "mixed" else [case["dtype"]]
    weights = [(1, 300, 90, 1100)[i % 4] for i in range(n)]
    per = total / sum(weights)
    return [(max(1, int(per * w) - (i % 3)), types[(i // 2) % len(types)])
            for i, w in enumerate(weights)]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _logits(case, g, dev):
    """Rows of logits: an offset for each row, a spread of 3, one token in ten
    rows' favour, the vocabulary's padded tail masked with -inf, and a few
    rows' tokens masked with the type's lowest value."""
    B, N, dt = case["B"], case["N"], _DT[case["dtype"]]
    x = torch.randn((B, N), generator=g, device=dev).mul_(3.0)
    x += torch.rand((B, 1), generator=g, device=dev).mul_(40.0).sub_(20.0)
    peak = torch.randint(0, N, (B,), generator=g, device=dev)
    x[torch.arange(B, device=dev), peak] += 9.0
    x = x.to(dt)
    pad = N % 64 // 8
    if pad and N > 400:
        x[:, N - pad:] = -math.inf
    if N > 400:
        x[::7, 100:140] = torch.finfo(dt).min
    return x


def _views(flat, like):
    """Views of a flat buffer in the sizes of the tensors ``like``."""
    views, at = [], 0
    for t in like:
        views.append(flat[at:at + t.numel()])
        at += -(-t.numel() // 64) * 64
    return views


def _tokens(n, V, g, dev):
    """Token ids with the frequencies of text: the r-th token's about 1 / r."""
    u = torch.rand(n, generator=g, device=dev, dtype=torch.float64)
    rank = torch.exp(u * math.log(V + 1.0)).floor().long().sub_(1).clamp_(0, V - 1)
    return rank.mul_(48271).add_(7).remainder_(V)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op in ("stats", "train"):
        B, N, K = case["B"], case["N"], case["K"]
        st["x"] = _logits(case, g, dev)
        t = torch.randint(0, max(1, N - 8), (B,), generator=g, device=dev)
        st["target"] = torch.where((t >= 100) & (t < 140), t - 100, t)  # no masked token
        if op == "train":
            adv = torch.randn(B, generator=g, device=dev)
            used = (torch.rand(B, generator=g, device=dev) >= case["prompt"]).float()
            st["grad_logprob"] = -adv * used
            st["grad_entropy"] = -0.01 * used
            st["grad_top"] = torch.randn((B, K), generator=g, device=dev) * 0.1 * used[:, None] \
                if K else None
    elif op in ("clip", "norm"):
        st["grads"] = [(torch.randn(n, generator=g, device=dev) * (0.02 if i % 4 else 0.5)).to(_DT[d])
                       for i, (n, d) in enumerate(_tensor_list(case))]
        if op == "clip":
            # The clipped gradients go to one flat buffer, each tensor on a boundary of
            # 64 elements, as optimizers keep them.
            st["flat"] = torch.zeros(sum(-(-t.numel() // 64) * 64 for t in st["grads"]),
                                     dtype=_DT[case["dtype"]], device=dev)
            st["out"] = _views(st["flat"], st["grads"])
            st["max_norm"] = 1.0
        if own:  # a program keeps its list of gradients, checked and laid out once
            import log_sum_exp_gb300 as L
            st["list"] = L.GradList(st["grads"], out=st.get("out"))
    else:
        V, D, T, dt = case["V"], case["D"], case["T"], _DT[case["dtype"]]
        st["ids"] = _tokens(T, V, g, dev)
        st["scale"] = math.sqrt(D)
        if op == "embed":
            st["table"] = (torch.randn((V, D), generator=g, device=dev) * 0.02).to(dt)
        else:
            st["grad"] = (torch.randn((T, D), generator=g, device=dev) * 0.1).to(dt)
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import log_sum_exp_gb300 as L

    case = st["case"]
    op = case["op"]
    if op in ("stats", "train"):
        s = L.lse_token_stats(st["x"], st["target"], top_k=case["K"])
        out = {"logprob": s.logprob, "entropy": s.entropy, "lse": s.lse}
        if case["K"]:
            out["top_logprob"], out["top_index"] = s.top_logprob, s.top_index
        if op == "train":
            out["dx"] = L.lse_token_stats_backward(st["x"], s, st["target"],
                                                   grad_logprob=st["grad_logprob"],
                                                   grad_entropy=st["grad_entropy"],
                                                   grad_top=st["grad_top"])
        return out
    if op == "norm":
        return L.lse_grad_norm(st["list"])
    if op == "clip":
        return [L.lse_grad_clip(st["list"], st["max_norm"]), st["flat"]]
    if op == "embed":
        return L.lse_embedding(st["table"], st["ids"], scale=st["scale"])
    return L.lse_embedding_backward(st["grad"], st["ids"], case["V"], scale=st["scale"])


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op in ("stats", "train"):
        K = case["K"]
        x = st["x"].float()
        m = x.amax(1, keepdim=True)
        z = x - m
        e = torch.exp(z)
        s = e.sum(1, keepdim=True)
        logs = torch.log(s)
        lse = m + logs
        ez = torch.where(e > 0, e * z, torch.zeros((), device=x.device))
        entropy = logs - ez.sum(1, keepdim=True) / s
        t = st["target"][:, None]
        out = {"logprob": (x.gather(1, t) - lse)[:, 0], "entropy": entropy[:, 0], "lse": lse[:, 0]}
        if K:
            v, i = torch.sort(x, dim=1, descending=True, stable=True)
            out["top_logprob"] = v[:, :K] - lse
            out["top_index"] = i[:, :K].contiguous()
            del v, i
        if op == "train":
            # With p the row's softmax: d logprob = [n = t] - p, d entropy =
            # -p (log p + H), d top_k = [n = i_k] - p.
            p = e / s
            logp = z - logs
            gl, ge = st["grad_logprob"][:, None], st["grad_entropy"][:, None]
            hot = -gl
            if K:
                hot = hot - st["grad_top"].sum(1, keepdim=True)
            dx = p * hot
            dx -= ge * torch.where(p > 0, p * (logp + entropy), torch.zeros((), device=x.device))
            dx.scatter_add_(1, t, gl)
            if K:
                dx.scatter_add_(1, out["top_index"], st["grad_top"])
            out["dx"] = dx.to(st["x"].dtype)
        return out
    if op in ("norm", "clip"):
        sums = [(t.float() * t.float()).sum() for t in st["grads"]]
        norm = torch.sqrt(torch.stack(sums).sum())
        if op == "norm":
            return norm
        coef = torch.clamp(st["max_norm"] / (norm + _EPS), max=1.0)
        for t, o in zip(st["grads"], st["out"]):
            o.copy_(t.float() * coef)
        return [norm, st["flat"]]
    if op == "embed":
        return (st["table"][st["ids"]].float() * st["scale"]).to(st["table"].dtype)
    grad = st["grad"]
    total = torch.zeros((case["V"], case["D"]), device=grad.device)
    total.index_add_(0, st["ids"], grad.float())
    return (total * st["scale"]).to(grad.dtype)


# ---------------------------------------------------------------------------
# The same in 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("stats", "train"):
        x, B, N, K = st["x"], case["B"], case["N"], case["K"]
        rows = max(1, (1 << 25) // N)
        parts = []
        for b in range(0, B, rows):
            parts.append(_exact_rows(st, x[b:b + rows].double(), slice(b, b + rows), K, op))
        return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if op in ("norm", "clip"):
        norm = math.sqrt(math.fsum(float((c.double() ** 2).sum()) for t in st["grads"]
                                   for c in t.split(1 << 24)))
        n = torch.tensor(norm, dtype=torch.float64, device=st["grads"][0].device)
        if op == "norm":
            return n
        coef = min(1.0, st["max_norm"] / (norm + _EPS))
        flat = torch.zeros(st["flat"].numel(), dtype=torch.float64, device=n.device)
        for v, t in zip(_views(flat, st["grads"]), st["grads"]):
            v.copy_(t.double() * coef)
        return [n, flat]
    if op == "embed":
        return st["table"].index_select(0, st["ids"]).double() * st["scale"]
    order = torch.argsort(st["ids"], stable=True)
    ids, counts = torch.unique_consecutive(st["ids"][order], return_counts=True)
    out = torch.zeros((case["V"], case["D"]), dtype=torch.float64, device=order.device)
    ends = torch.cumsum(counts, 0)
    cols = max(1, (1 << 26) // max(1, case["T"]))
    for c in range(0, case["D"], cols):
        running = torch.cumsum(st["grad"][order, c:c + cols].double(), 0)[ends - 1]
        running[1:] -= running[:-1].clone()
        out[ids, c:c + cols] = running * st["scale"]
    return out


def _exact_rows(st, x, rows, K, op):
    """Rows of ``stats`` (and ``train``) from log p = x - log sum exp x."""
    lse = torch.logsumexp(x, 1, keepdim=True)
    logp = x - lse
    p = torch.exp(logp)
    plogp = torch.where(p > 0, p * logp.clamp(min=-1e300), torch.zeros((), dtype=x.dtype, device=x.device))
    entropy = -plogp.sum(1)
    at = torch.arange(x.shape[0], device=x.device)
    t = st["target"][rows]
    out = {"logprob": logp[at, t], "entropy": entropy, "lse": lse[:, 0]}
    if K:
        # Keys in the order (value descending, index ascending), all different.
        bits = (x.float() + 0.0).view(torch.int32).long()
        bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
        key = bits * (1 << 24) - torch.arange(x.shape[1], device=x.device)
        top = torch.topk(key, K, dim=1).indices
        out["top_logprob"], out["top_index"] = logp.gather(1, top), top
    if op == "train":
        gl = st["grad_logprob"][rows].double()
        ge = st["grad_entropy"][rows].double()
        dx = -gl[:, None] * p - ge[:, None] * (plogp + p * entropy[:, None])
        dx[at, t] += gl
        for k in range(K):
            gt = st["grad_top"][rows, k].double()
            dx -= gt[:, None] * p
            dx[at, out["top_index"][:, k]] += gt
        out["dx"] = dx
    return out
