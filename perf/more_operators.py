"""Timing cases for the operators between a model's last block and its next token.

Four operators, each with the forms in which a program calls it:

sample  a token for every row of logits from a given uniform number, after
        temperature, top-k, top-p and min-p (``lse_sample``);
linear4 logits (or any projection) of a few tokens by a matrix held in 4 bits
        with a scale for each group of columns (``lse_linear4``);
quant   a matrix into that form and read back (``lse_quantize4``,
        ``lse_dequantize4``);
norm    the end of a block: norm of its output, gate, residual scale, sum with
        the residual stream and the norm of the sum (``lse_residual_norm``); the
        ``normgrad`` form adds every gradient (``lse_residual_norm_backward``).

``run`` makes one pass in plain torch operations, or, where ``own`` is set,
through this package.  ``exact`` computes the same results in 64 bits.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_EB = {"f32": 4, "bf16": 2, "f16": 2}
_EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One decoding step of one sequence, with a chat program's usual settings.
        {"name": "sample-one-token", "op": "sample", "dtype": "bf16", "B": 1, "N": 128256, "set": "chat"},
        # A decoding step of a serving batch: every request has settings of its own (greedy
        # ones among them); an odd vocabulary, so rows start off 16-byte boundaries.
        {"name": "sample-serving-batch", "op": "sample", "dtype": "f16", "B": 48, "N": 50257, "set": "mixed"},
        # Rollouts of a policy-gradient step: the model's own distribution, nothing cut off.
        {"name": "sample-rollouts", "op": "sample", "dtype": "bf16", "B": 2048, "N": 128256, "set": "plain"},
        # Many short rows: a byte vocabulary with a few special tokens, the nucleus only.
        {"name": "sample-byte-rows", "op": "sample", "dtype": "f32", "B": 65536, "N": 261, "set": "nucleus"},
        # The output matrix of one decoding step, f32 logits for the sampler.
        {"name": "linear4-one-token", "op": "linear4", "dtype": "bf16", "T": 1, "N": 128256, "K": 2048,
         "G": 128, "out": "f32"},
        # The same for a serving batch and finer groups.
        {"name": "linear4-serving-batch", "op": "linear4", "dtype": "f16", "T": 16, "N": 32000, "K": 4096,
         "G": 64, "out": "f16"},
        # f32 tokens, an odd vocabulary and an odd width.
        {"name": "linear4-odd", "op": "linear4", "dtype": "f32", "T": 3, "N": 50257, "K": 1001, "G": 32,
         "out": "f32"},
        # An output matrix going into 4 bits when a model is loaded.
        {"name": "quant-output-matrix", "op": "quant", "dtype": "bf16", "N": 128256, "K": 2048, "G": 128},
        # The same of odd sizes in f32.
        {"name": "quant-odd", "op": "quant", "dtype": "f32", "N": 50257, "K": 1001, "G": 32},
        # The end of a block in a decoding step.
        {"name": "norm-decode-batch", "op": "norm", "dtype": "bf16", "T": 64, "D": 2048, "post": True,
         "gate": "none"},
        # The same in a training step, with a gate for every channel, and all gradients.
        {"name": "normgrad-train-batch", "op": "normgrad", "dtype": "bf16", "T": 16384, "D": 4096, "post": True,
         "gate": "channel"},
        # An odd width in f32 without a norm after the block, a gate for every element.
        {"name": "normgrad-odd", "op": "normgrad", "dtype": "f32", "T": 5000, "D": 1001, "post": False,
         "gate": "element"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sample", "sample", "sample", "linear4", "linear4", "quant", "norm", "normgrad"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "sample":
        N = _log_int(rng, 200, 262144)
        return {"op": op, "dtype": dtype, "B": _log_int(rng, 1, max(1, min(65536, 50_000_000 // N))), "N": N,
                "set": rng.choice(["chat", "mixed", "plain", "nucleus", "few", "floor"])}
    if op in ("linear4", "quant"):
        K = _log_int(rng, 48, 8192)
        if rng.random() < 0.7:
            K = max(64, K // 64 * 64)
        N = _log_int(rng, 100, min(131072, 130_000_000 // K))
        G = rng.choice([32, 64, 128])
        if op == "quant":
            return {"op": op, "dtype": dtype, "N": N, "K": K, "G": G}
        return {"op": op, "dtype": dtype, "T": _log_int(rng, 1, 32), "N": N, "K": K, "G": G,
                "out": rng.choice([dtype, "f32"])}
    D = _log_int(rng, 32, 16384)
    if rng.random() < 0.7:
        D = max(64, D // 64 * 64)
    T = _log_int(rng, 1, min(65536, 60_000_000 // D))
    return {"op": op, "dtype": dtype, "T": T, "D": D, "post": rng.random() < 0.7,
            "gate": rng.choice(["none", "channel", "element"])}


def work(case):
    op, eb = case["op"], _EB[case["dtype"]]
    if op == "sample":
        n, B = case["B"] * case["N"], case["B"]
        return {"bytes": n * eb + B * 16 + (B * 20 if case["set"] == "mixed" else 0), "flops": 4 * n}
    if op in ("linear4", "quant"):
        N, K = case["N"], case["K"]
        held = N * K // 2 + N * -(-K // case["G"]) * eb
        if op == "quant":
            return {"bytes": 2 * N * K * eb + 2 * held, "flops": 4 * N * K}
        T = case["T"]
        return {"bytes": held + T * K * eb + T * N * _EB[case["out"]], "flops": 2 * T * N * K}
    T, D = case["T"], case["D"]
    full = T * D * eb
    gate = full if case["gate"] == "element" else 0
    vectors = (1 + case["post"] + (case["gate"] == "channel")) * D * eb
    if op == "norm":
        return {"bytes": 4 * full + gate + vectors, "flops": 8 * T * D}
    # Both passes: the forward's results and the sums' gradients are read in the second.
    return {"bytes": 4 * full + gate + vectors + 6 * full + 2 * gate + 2 * vectors, "flops": 30 * T * D}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _logits(case, g, dev):
    """Rows of logits: an offset and a spread for each row, from peaked ones to flat
    ones, one token in every row's favour, the vocabulary's padded tail masked with
    -inf, and a few rows' tokens masked with the type's lowest value."""
    B, N, dt = case["B"], case["N"], _DT[case["dtype"]]
    x = torch.randn((B, N), generator=g, device=dev)
    x *= torch.rand((B, 1), generator=g, device=dev).mul_(3.0).add_(1.0)
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


def _settings(case, g, dev):
    """temperature, top_k, top_p, min_p: a number for all rows, or one for each."""
    if case["set"] != "mixed":
        return {"plain": (1.0, 0, 1.0, 0.0), "chat": (0.7, 50, 0.95, 0.0), "nucleus": (0.9, 0, 0.9, 0.0),
                "few": (1.0, 1000, 1.0, 0.0), "floor": (1.3, 0, 1.0, 0.02)}[case["set"]]

    def pick(values, dtype):
        at = torch.randint(0, len(values), (case["B"],), generator=g, device=dev)
        return torch.tensor(values, dtype=dtype, device=dev)[at]

    return (pick([0.0, 0.5, 0.7, 1.0, 1.3], torch.float32), pick([0, 20, 50, 1000], torch.int64),
            pick([1.0, 0.95, 0.9, 0.5], torch.float32), pick([0.0, 0.0, 0.05, 0.1], torch.float32))


def _weights4(case, g, dev):
    """Whole numbers of -8 .. 7 and scales as a quantiser leaves them."""
    N, K = case["N"], case["K"]
    q = torch.randn((N, K), generator=g, device=dev).mul_(2.4).round_().clamp_(-8, 7).to(torch.int8)
    s = torch.rand((N, -(-K // case["G"])), generator=g, device=dev).add_(0.5).mul_(0.02 / 2.4)
    return q, s.to(_DT[case["dtype"]])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, dt = case["op"], _DT[case["dtype"]]
    st = {"case": dict(case)}
    if op == "sample":
        st["x"] = _logits(case, g, dev)
        st["u"] = torch.rand(case["B"], generator=g, device=dev)
        st["set"] = _settings(case, g, dev)
    elif op == "linear4":
        q, st["scales"] = _weights4(case, g, dev)
        st["x"] = torch.randn((case["T"], case["K"]), generator=g, device=dev).to(dt)
        if own:  # a program lays its weights out once
            import log_sum_exp_gb300 as L
            st["w"] = L.Weights4.from_values(q, st["scales"], case["G"])
        else:
            odd = case["K"] % 2
            c = torch.nn.functional.pad(q + 8, (0, odd)).to(torch.uint8)
            st["codes"] = c[:, 0::2] | (c[:, 1::2] << 4)  # two to a byte
    elif op == "quant":
        st["w"] = (torch.randn((case["N"], case["K"]), generator=g, device=dev) * 0.02).to(dt)
    else:
        T, D = case["T"], case["D"]

        def full(scale):
            return (torch.randn((T, D), generator=g, device=dev) * scale).to(dt)

        def vector(mean, spread):
            return (torch.randn(D, generator=g, device=dev) * spread + mean).to(dt)

        st["x"], st["y"] = full(1.5), full(0.4)
        st["weight"] = vector(1.0, 0.2)
        st["post"] = vector(1.0, 0.2) if case["post"] else None
        st["gate"] = {"none": None, "channel": vector(0.5, 0.3) if case["gate"] == "channel" else None,
                      "element": torch.sigmoid(full(1.0).float()).to(dt) if case["gate"] == "element" else None
                      }[case["gate"]]
        st["scale"] = 0.7
        if op == "normgrad":
            st["dh"], st["dout"] = full(0.1), full(0.1)
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
    if op == "sample":
        t, k, p, low = st["set"]
        s = L.lse_sample(st["x"], st["u"], temperature=t, top_k=k, top_p=p, min_p=low)
        return {"token": s.token, "logprob": s.logprob}
    if op == "linear4":
        return L.lse_linear4(st["x"], st["w"], out_dtype=_DT[case["out"]])
    if op == "quant":
        w = L.lse_quantize4(st["w"], group=case["G"])
        return [w.scales, L.lse_dequantize4(w)]
    s = L.lse_residual_norm(st["x"], st["y"], st["weight"], post_weight=st["post"], gate=st["gate"],
                            scale=st["scale"], eps=_EPS)
    out = {"h": s.h, "out": s.out}
    if op == "normgrad":
        d = L.lse_residual_norm_backward(st["dout"], st["dh"], st["x"], st["y"], s, st["weight"],
                                         post_weight=st["post"], gate=st["gate"], scale=st["scale"])
        out |= {"dx": d.x, "dy": d.y, "dweight": d.weight}
        if st["post"] is not None:
            out["dpost"] = d.post_weight
        if st["gate"] is not None:
            out["dgate"] = d.gate
    return out


def _column(v, like):
    """A setting as a 64-bit column, of one number or of one for each row; settings are
    32-bit numbers."""
    return torch.as_tensor(v, dtype=torch.float32, device=like.device).double().reshape(-1, 1)


def _sample_plain(st):
    # In 64 bits: a token is drawn where running sums pass a border, and in 32 bits
    # tokens next to it change places.
    x = st["x"].double()
    B, N = x.shape
    t, k, p, low = (_column(v, x) for v in st["set"])
    greedy = t == 0
    t = torch.where(greedy, 1.0, t)
    m = x.amax(1, keepdim=True)
    z = (x - m) / t
    w = torch.exp(z)
    if st["case"]["set"] != "plain":
        xs, order = torch.sort(x, dim=1, descending=True, stable=True)
        ws = torch.exp((xs - m) / t)
        ws = torch.where((torch.arange(N, device=x.device) < k) | (k <= 0), ws, 0.0)
        before = torch.cumsum(ws, 1) - ws
        keep = ((before < p * ws.sum(1, keepdim=True)) | (p >= 1)) & (xs - m >= t * torch.log(low))
        w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, 0.0))
        del xs, order, ws, before, keep
    running = torch.cumsum(w, 1)
    total = running[:, -1:]
    token = (running <= st["u"].double()[:, None] * total).sum(1, keepdim=True)
    token = torch.where(greedy, x.argmax(1, keepdim=True), token)
    logprob = z.gather(1, token) - torch.log(total)
    logprob = torch.where(greedy, 0.0, logprob)
    return {"token": token[:, 0], "logprob": logprob[:, 0].float()}


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "sample":
        return _sample_plain(st)
    if op == "linear4":
        N, K, G = case["N"], case["K"], case["G"]
        c = st["codes"]
        q = torch.stack((c & 15, c >> 4), 2).reshape(N, -1)[:, :K].float() - 8.0
        w = q * st["scales"].float().repeat_interleave(G, 1)[:, :K]
        return (st["x"].float() @ w.t()).to(_DT[case["out"]])
    if op == "quant":
        w, G = st["w"], case["G"]
        N, K = w.shape
        g = torch.nn.functional.pad(w.float(), (0, -K % G)).reshape(N, -1, G)
        # Quotients in 64 bits: in 32, one next to a half may round onto it.
        s = (g.abs().amax(2).double() / 7.0).to(w.dtype)
        f = s.float()[:, :, None]
        q = torch.where(f > 0, (g.double() / f.double()).round().clamp(-8.0, 7.0).float(), 0.0)
        return [s, (q * f).reshape(N, -1)[:, :K].to(w.dtype).contiguous()]
    dt = st["x"].dtype
    x, y, weight = st["x"].float(), st["y"].float(), st["weight"].float()
    D = x.shape[1]
    post = None if st["post"] is None else st["post"].float()
    gate = st["scale"] if st["gate"] is None else st["gate"].float() * st["scale"]
    r1 = a = None
    if post is None:
        a = y
    else:
        r1 = torch.rsqrt((y * y).mean(1, keepdim=True) + _EPS)
        a = y * r1 * post
    h = x + gate * a
    r2 = torch.rsqrt((h * h).mean(1, keepdim=True) + _EPS)
    out = {"h": h.to(dt), "out": (h * r2 * weight).to(dt)}
    if op == "normgrad":
        dn, dh = st["dout"].float(), st["dh"].float()
        n = dn * weight
        gr = dh + r2 * n - h * (r2 ** 3 / D) * (n * h).sum(1, keepdim=True)
        da = gr * gate
        if post is None:
            dy = da
        else:
            e = da * post
            dy = r1 * e - y * (r1 ** 3 / D) * (e * y).sum(1, keepdim=True)
        out |= {"dx": gr.to(dt), "dy": dy.to(dt), "dweight": (dn * h * r2).sum(0).to(dt)}
        if post is not None:
            out["dpost"] = (da * y * r1).sum(0).to(dt)
        if case["gate"] == "channel":
            out["dgate"] = (gr * a * st["scale"]).sum(0).to(dt)
        elif case["gate"] == "element":
            out["dgate"] = (gr * a * st["scale"]).to(dt)
    return out


# ---------------------------------------------------------------------------
# The same in 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "sample":
        rows = max(1, (1 << 24) // case["N"])
        parts = [_exact_rows(st, slice(b, min(case["B"], b + rows))) for b in range(0, case["B"], rows)]
        return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if op == "linear4":
        g = torch.Generator(device=st["x"].device)
        g.manual_seed(seed)
        q, s = _weights4(case, g, st["x"].device)  # what prepare() drew first
        rows = max(1, (1 << 25) // case["K"])
        columns = torch.arange(case["K"], device=q.device) // case["G"]
        return torch.cat([st["x"].double() @ (q[n:n + rows].double() * s[n:n + rows].double()[:, columns]).t()
                          for n in range(0, case["N"], rows)], 1)
    if op == "quant":
        return _exact_quant(st["w"], case["G"])
    need = op == "normgrad"
    leaves = {k: st[k].double().requires_grad_(need) for k in ("x", "y", "weight", "post", "gate")
              if st[k] is not None}
    a = leaves["y"]
    if "post" in leaves:
        a = a / torch.sqrt((a ** 2).mean(1, keepdim=True) + _EPS) * leaves["post"]
    if "gate" in leaves:
        a = a * leaves["gate"]
    h = leaves["x"] + st["scale"] * a
    n = h / torch.sqrt((h ** 2).mean(1, keepdim=True) + _EPS) * leaves["weight"]
    out = {"h": h.detach(), "out": n.detach()}
    if need:
        names = [k for k in ("x", "y", "weight", "post", "gate") if k in leaves]
        grads = torch.autograd.grad([h, n], [leaves[k] for k in names], [st["dh"].double(), st["dout"].double()])
        out |= {"d" + k: d for k, d in zip(names, grads)}
    return out


def _exact_rows(st, rows):
    """Rows of ``sample`` by rank: probabilities in the order of the values, cut by
    counting, and the draw over the kept ones put back in column order."""
    x = st["x"][rows].double()
    R, N = x.shape
    dev = x.device
    t, k, p, low = (_column(v, x).expand(st["x"].shape[0], 1)[rows] for v in st["set"])
    # Keys in the order (value descending, column ascending), all different.
    bits = (st["x"][rows].float() + 0.0).view(torch.int32).long()
    bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    order = torch.argsort(bits * (1 << 24) - torch.arange(N, device=dev), dim=1, descending=True)
    warm = torch.where(t > 0, t, 1.0)
    logits = x.gather(1, order) / warm
    at = torch.arange(N, device=dev)
    logits = torch.where((k <= 0) | (at < k), logits, -math.inf)
    prob = torch.softmax(logits, 1)
    count = ((torch.cumsum(prob, 1) - prob < p) | (p >= 1)).sum(1, keepdim=True)  # a prefix: sums only grow
    floor = logits[:, :1] + torch.log(low)
    kept = (at < count) & (logits >= floor)
    kept = torch.where(t > 0, kept, at < 1)  # greedy: the first alone
    prob = torch.where(kept, torch.softmax(torch.where(kept, logits, -math.inf), 1), 0.0)
    back = torch.zeros_like(prob).scatter_(1, order, prob)
    running = torch.cumsum(back, 1)
    border = st["u"][rows].double()[:, None] * running[:, -1:]
    token = torch.searchsorted(running, border, right=True)
    return {"token": token[:, 0], "logprob": torch.log(back.gather(1, token))[:, 0]}


def _exact_quant(w, G):
    scales, values = [], []
    step = max(1, (1 << 25) // w.shape[1])
    for n in range(0, w.shape[0], step):
        part = w[n:n + step].double()
        groups = part.split(G, 1)
        # The scale is defined as a value of the matrix's type, so it is rounded here too.
        s = torch.stack([(v.abs().amax(1) / 7.0).to(w.dtype) for v in groups], 1)
        wide = s.double().repeat_interleave(G, 1)[:, :w.shape[1]]
        units = torch.where(wide > 0, part / wide, 0.0)
        values.append(torch.round(units).clamp(-8.0, 7.0) * wide)
        scales.append(s.double())
    return [torch.cat(scales), torch.cat(values)]
