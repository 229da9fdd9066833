"""Cases that measure the operators of a transformer's training step around the gradient average.

norm          h = x + residual, mean and rstd = 1/sqrt(var + eps) of every row, y = (h - mean) * rstd * gamma + beta
norm_grad     the gradient of norm with respect to x (= residual), gamma and beta
logprob       per token: log p[target] of p = softmax(logits / tau), the entropy of p, its log-sum-exp, and the k most
              probable entries with their log probabilities (the lowest index first among equals); a target outside
              the vocabulary counts as 0
logprob_grad  the gradient of log p[target] and of the entropy with respect to the logits
orthogonalise Newton-Schulz steps X <- a X + (b A + c A A) X with A = X X^T on matrices divided by their norm
muon          the average of the replicas' gradients, momentum, the orthogonalised update, the weights

A case is a dict of plain values; ``own`` chooses between the plain form
(elementary torch operations in 32 bits, rounded once at the end) and the
package's entry points.
"""
import math

import torch

own = False

EPS = 1e-5
NS_EPS = 1e-7
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
# a fine-tuning step: a learning rate of 1e-4, updates scaled to the size that AdamW's have
LR, MOMENTUM, DECAY, RMS = 1e-4, 0.95, 0.1, 0.2


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the last norm of one GPT-2 small token (d = 768): a decoding step, latency only
        {"name": "norm 1x768", "kind": "norm", "T": 1, "D": 768, "dtype": "bf16", "residual": True},
        # a training batch of 16 x 1024 tokens at a width of 4096
        {"name": "norm 16384x4096", "kind": "norm", "T": 16384, "D": 4096, "dtype": "bf16", "residual": True},
        # backward of a GPT-2 small batch: 8 x 1024 tokens
        {"name": "norm grad 8192x768", "kind": "norm_grad", "T": 8192, "D": 768, "dtype": "bf16", "residual": True},
        # the same in fp32 at an odd width: rows that are not whole vectors
        {"name": "norm grad 4099x2051 f32", "kind": "norm_grad", "T": 4099, "D": 2051, "dtype": "f32",
         "residual": True},
        # the next token's log probability and 20 alternatives, as a server answers them (fp32 logits)
        {"name": "logprob 1x50257 f32", "kind": "logprob", "T": 1, "V": 50257, "k": 20, "dtype": "f32", "tau": 1.0,
         "masked": False},
        # a teacher's batch: 8 x 1024 tokens with the 64 entries that a student is distilled from
        {"name": "logprob 8192x50257", "kind": "logprob", "T": 8192, "V": 50257, "k": 64, "dtype": "bf16", "tau": 1.0,
         "masked": False},
        # a policy's ragged batch with part of the vocabulary masked, sampled at a temperature
        {"name": "logprob grad 517x32003 f32", "kind": "logprob_grad", "T": 517, "V": 32003, "dtype": "f32",
         "tau": 0.7, "masked": True},
        # the backward pass of a training step: 8 x 1024 tokens of the GPT-2 small vocabulary
        {"name": "logprob grad 8192x50257", "kind": "logprob_grad", "T": 8192, "V": 50257, "dtype": "bf16",
         "tau": 1.0, "masked": False},
        # the attention projections of GPT-2 small's 12 layers
        {"name": "orthogonalise 12x768x768", "kind": "orthogonalise", "count": 12, "rows": 768, "cols": 768,
         "dtype": "f32"},
        # one large projection
        {"name": "orthogonalise 4096x4096", "kind": "orthogonalise", "count": 1, "rows": 4096, "cols": 4096,
         "dtype": "bf16"},
        # a classifier's weight (ResNet-50's 1000 x 2048) on 8 replicas
        {"name": "muon 1000x2048 f32", "kind": "muon", "count": 1, "rows": 1000, "cols": 2048, "dtype": "f32",
         "replicas": 8},
        # the attention inputs of GPT-2 small's 12 layers ([d, 3 d]) on 8 replicas of bf16 gradients
        {"name": "muon 12x768x2304", "kind": "muon", "count": 12, "rows": 768, "cols": 2304, "dtype": "bf16",
         "replicas": 8},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "norm_grad", "logprob", "logprob", "logprob_grad", "orthogonalise", "muon"])
    if kind in ("norm", "norm_grad"):
        d = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            d = max(64, d // 64 * 64)
        t = _log_int(rng, 1, max(1, min(65536, 16384 * 4096 // d // 2)))
        return {"kind": kind, "T": t, "D": d, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "residual": rng.random() < 0.75}
    if kind in ("logprob", "logprob_grad"):
        v = _log_int(rng, 1000, 160000)
        t = _log_int(rng, 1, max(1, min(16384, 8192 * 50257 // v // 2)))
        case = {"kind": kind, "T": t, "V": v, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "tau": rng.choice([0.7, 1.0, 2.0]), "masked": rng.random() < 0.3}
        if kind == "logprob":
            case["k"] = rng.choice([0, _log_int(rng, 1, 128), _log_int(rng, 1, 128), _log_int(rng, 1, 128)])
        return case
    rows, cols = _log_int(rng, 64, 4096), _log_int(rng, 64, 4096)
    if rng.random() < 0.5:
        rows, cols = max(64, rows // 64 * 64), max(64, cols // 64 * 64)
    short = min(rows, cols)
    count = _log_int(rng, 1, max(1, min(16, 4096 ** 3 // (short * rows * cols) // 2)))
    case = {"kind": kind, "count": count, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "f32"])}
    if kind == "muon":
        case["replicas"] = rng.choice([1, 2, 4, 8])
    return case


# ------------------------------------------------------------------ inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _gradient(gen, *shape):
    """A weight's gradient: a few directions that all examples share, and noise of about their size."""
    *count, rows, cols = shape
    shared = _randn(gen, *count, rows, 8) @ _randn(gen, *count, 8, cols) / math.sqrt(8)
    return (shared + _randn(gen, *shape)) * 1e-3


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["kind"] in ("norm", "norm_grad"):
        T, D, dt = case["T"], case["D"], DTYPES[case["dtype"]]
        # activations: unit variance, one channel in 64 a few times larger and off centre
        large = torch.rand(D, generator=gen, device="cuda") < 1 / 64
        chan, off = torch.where(large, 3.0, 1.0), torch.where(large, 4.0, 0.2)
        s["gamma"], s["beta"] = 1 + 0.1 * _randn(gen, D), 0.1 * _randn(gen, D)
        if case["kind"] == "norm":
            s["x"] = (_randn(gen, T, D) * chan).to(dt)
            s["r"] = (_randn(gen, T, D) * 2 + off).to(dt) if case["residual"] else None
        else:
            h = (_randn(gen, T, D) * chan * 2 + off).to(dt)
            s["h"], s["dy"] = h, (_randn(gen, T, D) * 0.1).to(dt)
            s["dh"] = (_randn(gen, T, D) * 0.1).to(dt) if case["residual"] else None
            s["mean"] = h.float().mean(1)
            s["rstd"] = torch.rsqrt((h.float() - s["mean"][:, None]).square().mean(1) + EPS)
        return s
    if case["kind"] in ("logprob", "logprob_grad"):
        T, V, dt = case["T"], case["V"], DTYPES[case["dtype"]]
        z = _randn(gen, T, V) * 2.5
        if case["masked"]:                       # a vocabulary of which 2 entries in 3 may be answered
            z.masked_fill_(torch.rand(V, generator=gen, device="cuda") < 1 / 3, -math.inf)
        target = torch.randint(0, V, (T, 1), generator=gen, device="cuda")
        some = torch.rand(T, 1, generator=gen, device="cuda") < 0.5       # the model is sure of half of its tokens
        z.scatter_add_(1, target, torch.where(some, 12.0, 0.0))
        target = target[:, 0]
        if T > 8:                                # padding tokens
            target = torch.where(torch.rand(T, generator=gen, device="cuda") < 0.03, -100, target)
        s["logits"], s["target"] = z.to(dt), target.contiguous()
        if case["kind"] == "logprob_grad":
            logp = torch.log_softmax(s["logits"].float() / case["tau"], 1)
            s["lse"] = torch.logsumexp(s["logits"].float() / case["tau"], 1)
            s["entropy"] = -torch.where(logp > -math.inf, logp.exp() * logp, 0.0).sum(1)
            s["dlogprob"] = _randn(gen, T) / T   # advantages over the tokens
            s["dentropy"] = torch.full((T,), 0.01 / T, device="cuda")
        return s
    n, rows, cols, dt = case["count"], case["rows"], case["cols"], DTYPES[case["dtype"]]
    if case["kind"] == "orthogonalise":
        s["g"] = list(_gradient(gen, n, rows, cols).to(dt))
        return s
    # flat buffers with the matrices in them one after another, as the bucket plan lays them out
    size = rows * cols
    pitch = (size + 127) // 128 * 128
    s["offsets"] = [i * pitch for i in range(n)]
    mean = _gradient(gen, n, rows, cols)
    s["grads"] = []
    for _ in range(case["replicas"]):
        flat = torch.zeros(n, pitch, device="cuda")
        flat[:, :size] = (mean + _randn(gen, n, rows, cols) * 1e-3).reshape(n, size)
        s["grads"].append(flat.reshape(-1).to(dt))
    s["param"], s["buf"] = torch.zeros(n * pitch, device="cuda"), torch.zeros(n * pitch, device="cuda")
    s["param"].view(n, pitch)[:, :size] = _randn(gen, n, size) * 0.04
    s["buf"].view(n, pitch)[:, :size] = (mean * 10 + _randn(gen, n, rows, cols) * 3e-3).reshape(n, size)
    s["scale"] = RMS * math.sqrt(max(rows, cols))
    return s


# ------------------------------------------------------------------ the plain form

def _plain_norm(s):
    dt = DTYPES[s["dtype"]]
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    mean = h.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((h - mean).square().mean(1, keepdim=True) + EPS)
    out = {"y": ((h - mean) * rstd * s["gamma"] + s["beta"]).to(dt), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if s["r"] is not None:
        out["h"] = h.to(dt)
    return out


def _plain_norm_grad(s):
    dt = DTYPES[s["dtype"]]
    dy, n = s["dy"].float(), (s["h"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dn = dy * s["gamma"]
    dx = s["rstd"][:, None] * (dn - dn.mean(1, keepdim=True) - n * (dn * n).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(dt), "dgamma": (dy * n).sum(0), "dbeta": dy.sum(0)}


def _plain_logprob(s):
    tau, V, k = s["tau"], s["V"], s["k"]
    z = s["logits"].float() / tau
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    inside = (s["target"] >= 0) & (s["target"] < V)
    at = torch.gather(z, 1, torch.where(inside, s["target"], 0)[:, None])
    out = {"logprob": torch.where(inside, (at - lse)[:, 0], 0.0), "lse": lse[:, 0]}
    # -sum p ln p, an entry of probability 0 counting as 0
    out["entropy"] = (torch.log(total) - torch.where(e > 0, e * (z - top), 0.0).sum(1, keepdim=True) / total)[:, 0]
    if k:
        # one whole number per entry: its value's order (0 and -0 alike), then the lower index first
        bits = (s["logits"].float() + 0.0).view(torch.int32).long()
        order = torch.where(bits < 0, -(bits & 0x7fffffff), bits)
        key = order * 2 ** 20 + (V - 1 - torch.arange(V, device="cuda"))
        index = torch.topk(key, k, dim=1).indices
        out["top_index"], out["top_logprob"] = index, torch.gather(z, 1, index) - lse
    return out


def _plain_logprob_grad(s):
    tau, V = s["tau"], s["V"]
    logp = s["logits"].float() / tau - s["lse"][:, None]
    p = torch.exp(logp)
    inside = (s["target"] >= 0) & (s["target"] < V)
    up = torch.where(inside, s["dlogprob"], 0.0)[:, None]
    surprise = torch.where(p > 0, p * (logp + s["entropy"][:, None]), 0.0)
    dz = -(p * up + surprise * s["dentropy"][:, None])
    dz.scatter_add_(1, torch.where(inside, s["target"], 0)[:, None], up)
    return (dz / tau).to(DTYPES[s["dtype"]])


def _plain_steps(x):
    """Newton-Schulz on a stack of matrices, in 32 bits."""
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    for _ in range(5):
        a = x @ x.transpose(1, 2)
        x = NS_A * x + (NS_B * a + NS_C * (a @ a)) @ x
    return x.transpose(1, 2) if tall else x


def _plain_orthogonalise(s):
    return list(_plain_steps(torch.stack(s["g"]).float()).to(torch.bfloat16))


def _plain_muon(s):
    n, size = s["count"], s["rows"] * s["cols"]
    mean = torch.stack([x.view(n, -1) for x in s["grads"]]).float().sum(0) / s["replicas"]
    buf = s["buf"].view(n, -1)
    buf.mul_(MOMENTUM).add_(mean)
    update = _plain_steps((mean + MOMENTUM * buf)[:, :size].reshape(n, s["rows"], s["cols"]))
    param = s["param"].view(n, -1)[:, :size]
    param.mul_(1 - LR * DECAY).sub_(update.reshape(n, size) * (LR * s["scale"]))
    return {"param": s["param"], "buf": s["buf"]}


# ------------------------------------------------------------------ the package's operators

def _kept(s, name, *shape, dtype):
    """A buffer that the caller keeps from call to call, as the package's callers do."""
    if name not in s:
        s[name] = torch.empty(shape, dtype=dtype, device="cuda")
    return s[name]


def _own_norm(s):
    import gradient_sync_ddp_gb300 as g
    T, D, dt = s["T"], s["D"], DTYPES[s["dtype"]]
    out = {n: _kept(s, "out_" + n, T, dtype=torch.float32) for n in ("mean", "rstd")}
    h = None
    if s["r"] is not None:
        out["h"] = h = _kept(s, "out_h", T, D, dtype=dt)
    out["y"] = _kept(s, "out_y", T, D, dtype=dt)
    g.layernorm_forward(s["x"], s["gamma"], s["beta"], out["y"], EPS, residual=s["r"], h_out=h, mean_out=out["mean"],
                        rstd_out=out["rstd"])
    return out


def _own_norm_grad(s):
    import gradient_sync_ddp_gb300 as g
    T, D = s["T"], s["D"]
    if "ws" not in s:
        s["ws"] = torch.empty(g.layernorm_backward_workspace_bytes(T, D), dtype=torch.uint8, device="cuda")
    out = {n: _kept(s, "out_" + n, D, dtype=torch.float32) for n in ("dgamma", "dbeta")}
    out["dx"] = _kept(s, "out_dx", T, D, dtype=DTYPES[s["dtype"]])
    g.layernorm_backward(s["dy"], s["h"], s["mean"], s["rstd"], s["gamma"], out["dx"], out["dgamma"], out["dbeta"],
                         s["ws"], dh=s["dh"])
    return out


def _own_logprob(s):
    import gradient_sync_ddp_gb300 as g
    T, k = s["T"], s["k"]
    out = {n: _kept(s, "out_" + n, T, dtype=torch.float32) for n in ("logprob", "entropy", "lse")}
    index = logprob = None
    if k:
        out["top_index"] = index = _kept(s, "out_index", T, k, dtype=torch.int64)
        out["top_logprob"] = logprob = _kept(s, "out_top", T, k, dtype=torch.float32)
    g.token_logprobs_forward(s["logits"], s["target"], out["logprob"], out["entropy"], out["lse"], index, logprob,
                             temperature=s["tau"])
    return out


def _own_logprob_grad(s):
    import gradient_sync_ddp_gb300 as g
    dz = _kept(s, "out_dlogits", s["T"], s["V"], dtype=DTYPES[s["dtype"]])
    g.token_logprobs_backward(s["logits"], s["target"], s["lse"], s["dlogprob"], dz, s["entropy"], s["dentropy"],
                              temperature=s["tau"])
    return dz


def _workspace(s, g):
    if "ws" not in s:
        s["ws"] = torch.empty(g.newton_schulz_workspace_bytes(s["count"], s["rows"], s["cols"]), dtype=torch.uint8,
                              device="cuda")
    return s["ws"]


def _own_orthogonalise(s):
    import gradient_sync_ddp_gb300 as g
    if "out" not in s:
        s["out"] = list(torch.empty(s["count"], s["rows"], s["cols"], dtype=torch.bfloat16, device="cuda"))
    g.newton_schulz(s["g"], s["out"], _workspace(s, g), steps=5, eps=NS_EPS)
    return s["out"]


def _own_muon(s):
    import gradient_sync_ddp_gb300 as g
    g.ddp_bucket_allreduce_muon(s["grads"], s["offsets"], s["rows"], s["cols"], s["param"], s["buf"], _workspace(s, g),
                                LR, MOMENTUM, DECAY, update_scale=s["scale"], nesterov=True, steps=5, eps=NS_EPS)
    return {"param": s["param"], "buf": s["buf"]}


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "logprob": _plain_logprob,
          "logprob_grad": _plain_logprob_grad, "orthogonalise": _plain_orthogonalise, "muon": _plain_muon}
_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "logprob": _own_logprob, "logprob_grad": _own_logprob_grad,
        "orthogonalise": _own_orthogonalise, "muon": _own_muon}


def run(state):
    return (_OWN if own else _PLAIN)[state["kind"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    kind = case["kind"]
    if kind in ("norm", "norm_grad"):
        n, b, res = case["T"] * case["D"], BYTES[case["dtype"]], int(case["residual"])
        if kind == "norm":               # x, residual in; h, y, mean, rstd out; gamma, beta
            return {"bytes": n * b * (2 + 2 * res) + 8 * case["T"] + 8 * case["D"], "flops": 8 * n}
        return {"bytes": n * b * (3 + res) + 8 * case["T"] + 12 * case["D"], "flops": 13 * n}
    if kind in ("logprob", "logprob_grad"):
        n, b, T = case["T"] * case["V"], BYTES[case["dtype"]], case["T"]
        if kind == "logprob":
            return {"bytes": n * b + 20 * T + 12 * T * case["k"], "flops": 5 * n}
        return {"bytes": 2 * n * b + 24 * T, "flops": 8 * n}
    n = case["count"] * case["rows"] * case["cols"]
    m = min(case["rows"], case["cols"])
    # a step: the two symmetric products by half of their entries, and the product with X
    flops = 5 * (3 * n * m + case["count"] * m ** 3)
    if kind == "orthogonalise":
        return {"bytes": n * (BYTES[case["dtype"]] + 2), "flops": flops}
    return {"bytes": n * (case["replicas"] * BYTES[case["dtype"]] + 16), "flops": flops}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_norm(s):
    h = s["x"].double() + (0 if s["r"] is None else s["r"].double())
    var, mean = torch.var_mean(h, 1, correction=0)
    y = torch.addcmul(s["beta"].double(), (h - mean[:, None]) / (var + EPS).sqrt()[:, None], s["gamma"].double())
    out = {"y": y, "mean": mean, "rstd": (var + EPS).pow(-0.5)}
    if s["r"] is not None:
        out["h"] = h
    return out


def _exact_norm_grad(s):
    dy, h, g, m, r = (s[n].double() for n in ("dy", "h", "gamma", "mean", "rstd"))
    h = h - m[:, None]
    inner, total = torch.einsum("td,td,d->t", dy, h, g), torch.einsum("td,d->t", dy, g)
    dx = torch.einsum("td,d,t->td", dy, g, r) - (r * total / s["D"])[:, None] - h * (r.pow(3) * inner / s["D"])[:, None]
    if s["dh"] is not None:
        dx = dx + s["dh"].double()
    return {"dx": dx, "dgamma": torch.einsum("td,td,t->d", dy, h, r), "dbeta": torch.einsum("td->d", dy)}


def _blocks(s):
    """Blocks of tokens: 64-bit logits of all of them are large."""
    return [slice(t, min(s["T"], t + 512)) for t in range(0, s["T"], 512)]


def _exact_logprob(s):
    rows = []
    for part in _blocks(s):
        z, target = s["logits"][part], s["target"][part]
        logp = torch.log_softmax(z.double() / s["tau"], 1)
        absent = (target < 0) | (target >= s["V"])
        one = {"logprob": logp.gather(1, target.masked_fill(absent, 0)[:, None])[:, 0].masked_fill(absent, 0.0),
               "lse": torch.logsumexp(z.double() / s["tau"], 1),
               "entropy": torch.special.entr(logp.exp()).sum(1)}
        if s["k"]:
            values, index = torch.sort(z.double(), dim=1, descending=True, stable=True)
            one["top_index"] = index[:, :s["k"]].contiguous()
            one["top_logprob"] = logp.gather(1, one["top_index"])
            del values, index
        rows.append(one)
    return {name: torch.cat([one[name] for one in rows]) for name in rows[0]}


def _exact_logprob_grad(s):
    rows = []
    for part in _blocks(s):
        logp = s["logits"][part].double() / s["tau"] - s["lse"][part].double()[:, None]
        target, dentropy = s["target"][part], s["dentropy"][part].double()[:, None]
        absent = (target < 0) | (target >= s["V"])
        up = s["dlogprob"][part].double().masked_fill(absent, 0.0)[:, None]
        p = logp.exp()
        dz = torch.zeros_like(p).scatter_(1, target.masked_fill(absent, 0)[:, None], up) - p * up
        dz += dentropy * (torch.special.entr(p) - p * s["entropy"][part].double()[:, None])
        # kept in 32 bits: the 64-bit gradient of the largest case would not fit beside the rest
        rows.append((dz / s["tau"]).float())
    return torch.cat(rows)


def _exact_steps(x):
    """On the shorter side, whichever it is, the polynomial of the Gram matrix: X X^T X = X (X^T X)."""
    x = x / (torch.linalg.matrix_norm(x) + NS_EPS)
    wide = x.shape[0] <= x.shape[1]
    for _ in range(5):
        gram = torch.mm(x, x.t()) if wide else torch.mm(x.t(), x)
        poly = torch.addmm(gram, gram, gram, beta=NS_B, alpha=NS_C)
        poly.diagonal().add_(NS_A)
        x = torch.mm(poly, x) if wide else torch.mm(x, poly)
    return x


def _exact_orthogonalise(s):
    return [_exact_steps(x.double()) for x in s["g"]]


def _exact_muon(s):
    size, grads = s["rows"] * s["cols"], [x.double() for x in s["grads"]]
    param, buf = s["param"].double(), s["buf"].double()
    mean = sum(grads) / len(grads)
    buf = buf * MOMENTUM + mean
    for o in s["offsets"]:
        part = slice(o, o + size)
        update = _exact_steps((mean[part] + buf[part] * MOMENTUM).view(s["rows"], s["cols"]))
        param[part] = param[part] * (1 - LR * DECAY) - LR * s["scale"] * update.reshape(-1)
    return {"param": param, "buf": buf}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "logprob": _exact_logprob,
            "logprob_grad": _exact_logprob_grad, "orthogonalise": _exact_orthogonalise,
            "muon": _exact_muon}[case["kind"]](s)
