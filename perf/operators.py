"""Cases that measure the operators of distilling a student from an 8-bit teacher.

norm      h = x + residual, rstd = 1/sqrt(mean(h^2) + eps), y = h * rstd * gamma;
          with q8 the output is 8-bit integers with one scale per token
norm_grad the gradient of norm with respect to x (= residual) and gamma
product   out[m, n] = (sum_k a[m, k] * w[n, k]) * sa[m] * sw[n] of 8-bit integers
distill   loss_t = tau^2 * KL(p || q) where p = softmax(teacher / tau) over a token's
          k teacher entries (an index outside the vocabulary is no entry; a token
          without entries has loss and gradient 0) and q = softmax(logits / tau) over
          the vocabulary; direction "loss", "grad" (from a kept log-sum-exp) or "both"

A case is a dict of plain values; ``own`` chooses between the plain form
(elementary torch operations in 32 bits, rounded once at the end) and the
package's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a GPT-2 small block (d = 768): what a decoding step pays, latency only
        {"name": "norm 1x768", "kind": "norm", "q8": False, "T": 1, "D": 768, "dtype": "bf16", "residual": True},
        # a training batch of 16 x 1024 tokens at a width of 4096
        {"name": "norm 16384x4096", "kind": "norm", "q8": False, "T": 16384, "D": 4096, "dtype": "bf16",
         "residual": True},
        # a few sequences' next tokens on their way into an 8-bit product
        {"name": "norm q8 24x4096", "kind": "norm", "q8": True, "T": 24, "D": 4096, "dtype": "bf16",
         "residual": True},
        # a ragged batch of teacher tokens into 8 bits
        {"name": "norm q8 10007x2560", "kind": "norm", "q8": True, "T": 10007, "D": 2560, "dtype": "bf16",
         "residual": True},
        # backward of a GPT-2 small batch: 8 x 1024 tokens
        {"name": "norm grad 8192x768", "kind": "norm_grad", "T": 8192, "D": 768, "dtype": "bf16", "residual": True},
        # the same in fp32 at an odd width: rows that are not whole vectors
        {"name": "norm grad 4099x2051 f32", "kind": "norm_grad", "T": 4099, "D": 2051, "dtype": "f32",
         "residual": True},
        # the teacher's head on one token (GPT-2 small vocabulary)
        {"name": "product 1x50257x768", "kind": "product", "M": 1, "N": 50257, "K": 768, "out": "f32"},
        # a projection on the next tokens of a ragged set of sequences
        {"name": "product 37x8192x4096", "kind": "product", "M": 37, "N": 8192, "K": 4096, "out": "bf16"},
        # a projection on a prompt batch: the largest product
        {"name": "product 8192x16384x4096", "kind": "product", "M": 8192, "N": 16384, "K": 4096, "out": "bf16"},
        # a validation loss on a few tokens of fp32 logits
        {"name": "distill loss 129x50257 f32", "kind": "distill", "direction": "loss", "T": 129, "V": 50257, "k": 50,
         "dtype": "f32", "tau": 1.0},
        # the backward pass of an autograd step, odd vocabulary
        {"name": "distill grad 2049x32003", "kind": "distill", "direction": "grad", "T": 2049, "V": 32003, "k": 100,
         "dtype": "bf16", "tau": 2.0},
        # a training step's loss and gradient: 8 x 1024 tokens of the GPT-2 small vocabulary
        {"name": "distill both 8192x50257", "kind": "distill", "direction": "both", "T": 8192, "V": 50257, "k": 64,
         "dtype": "bf16", "tau": 2.0},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "norm_grad", "product", "product", "distill", "distill"])
    if kind in ("norm", "norm_grad"):
        d = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            d = max(64, d // 64 * 64)
        t = _log_int(rng, 1, max(1, min(65536, 16384 * 4096 // d // 2)))
        case = {"kind": kind, "T": t, "D": d, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "residual": rng.random() < 0.75}
        if kind == "norm":
            case["q8"] = rng.random() < 0.5
        return case
    if kind == "product":
        n, k = _log_int(rng, 64, 50257), _log_int(rng, 64, 8192)
        if rng.random() < 0.7:
            k = max(64, k // 64 * 64)
        m = _log_int(rng, 1, max(1, min(8192, int(8192 * 16384 * 4096 / (n * k)))))
        return {"kind": kind, "M": m, "N": n, "K": k, "out": rng.choice(["bf16", "bf16", "f32"])}
    v = _log_int(rng, 1000, 160000)
    t = _log_int(rng, 1, max(1, min(16384, 8192 * 50257 // v // 2)))
    return {"kind": kind, "direction": rng.choice(["loss", "grad", "both"]), "T": t, "V": v,
            "k": _log_int(rng, 1, 256), "dtype": rng.choice(["bf16", "bf16", "f32"]),
            "tau": rng.choice([1.0, 2.0, 4.0])}


# ------------------------------------------------------------------ inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["kind"] in ("norm", "norm_grad"):
        T, D, dt = case["T"], case["D"], DTYPES[case["dtype"]]
        # activations: unit variance, one channel in 64 a few times larger
        chan = torch.where(torch.rand(D, generator=gen, device="cuda") < 1 / 64, 3.0, 1.0)
        s["gamma"] = 1 + 0.1 * _randn(gen, D)
        if case["kind"] == "norm":
            s["x"] = (_randn(gen, T, D) * chan).to(dt)
            s["r"] = (_randn(gen, T, D) * 2).to(dt) if case["residual"] else None
        else:
            h = (_randn(gen, T, D) * chan * 2).to(dt)
            s["h"], s["dy"] = h, (_randn(gen, T, D) * 0.1).to(dt)
            s["dh"] = (_randn(gen, T, D) * 0.1).to(dt) if case["residual"] else None
            s["rstd"] = torch.rsqrt((h.float() * h.float()).mean(1) + EPS)
        return s
    if case["kind"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        for name, rows in (("a", M), ("w", N)):
            x = _randn(gen, rows, K)
            scale = x.abs().amax(1) / 127
            s[name] = torch.round(x / scale[:, None]).to(torch.int8)
            s["s" + name] = scale
        return s
    T, V, k, dt = case["T"], case["V"], case["k"], DTYPES[case["dtype"]]
    logits = _randn(gen, T, V) * 2.5
    # the teacher agrees in part with the student; its k largest logits, in descending order
    top = torch.topk(logits * 0.6 + _randn(gen, T, V) * 1.5, k, dim=1)
    s["logits"] = logits.to(dt)
    s["teacher"], s["index"] = top.values.contiguous(), top.indices.contiguous()
    # ragged lists: the tail of some tokens' entries is absent, padding tokens have none
    kept = torch.randint(1, k + 1, (T, 1), generator=gen, device="cuda")
    kept = torch.where(torch.rand(T, 1, generator=gen, device="cuda") < 0.7, k, kept)
    if T > 8:
        kept = torch.where(torch.rand(T, 1, generator=gen, device="cuda") < 0.03, 0, kept)
    s["index"] = torch.where(torch.arange(k, device="cuda") < kept, s["index"], -1)
    s["dloss"] = torch.full((T,), 1.0 / T, device="cuda")
    s["lse"] = torch.logsumexp(s["logits"].float() / case["tau"], 1) if case["direction"] == "grad" else None
    return s


# ------------------------------------------------------------------ the plain form

def _plain_norm(s):
    dt = DTYPES[s["dtype"]]
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    rstd = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    y = h * rstd * s["gamma"]
    out = {"rstd": rstd[:, 0]}
    if s["r"] is not None:
        out["h"] = h.to(dt)
    if s["q8"]:
        scale = y.abs().amax(1, keepdim=True) / 127
        q = torch.where(scale > 0, torch.round(y / scale), 0.0).clamp(-127, 127)
        out["values"], out["scale"] = (q * scale).to(torch.bfloat16), scale[:, 0]
    else:
        out["y"] = y.to(dt)
    return out


def _plain_norm_grad(s):
    dt = DTYPES[s["dtype"]]
    dy, n = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
    dn = dy * s["gamma"]
    dx = s["rstd"][:, None] * (dn - n * (dn * n).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(dt), "dgamma": (dy * n).sum(0)}


def _plain_product(s):
    acc = s["a"].float() @ s["w"].float().T
    return (acc * s["sa"][:, None] * s["sw"]).to(DTYPES[s["out"]])


def _plain_distill(s):
    tau, V = s["tau"], s["V"]
    z = s["logits"].float() / tau
    valid = (s["index"] >= 0) & (s["index"] < V)
    some = valid.any(1)
    at = torch.where(valid, s["index"], 0)
    t = torch.where(valid, s["teacher"].float() / tau, -math.inf)
    t = t - torch.where(some[:, None], t.amax(1, keepdim=True), 0.0)
    e = torch.exp(t)
    total = e.sum(1, keepdim=True)
    p = torch.where(some[:, None], e / total, 0.0)
    out = {}
    if s["direction"] == "grad":
        lse = s["lse"][:, None]
    else:
        top = z.amax(1, keepdim=True)
        lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
        log_p = torch.where(p > 0, t - torch.log(total), 0.0)
        log_q = torch.where(p > 0, torch.gather(z, 1, at) - lse, 0.0)
        out["loss"] = torch.where(some, (p * (log_p - log_q)).sum(1), 0.0) * (tau * tau)
        out["lse"] = lse[:, 0]
    if s["direction"] != "loss":
        g = torch.where(some, s["dloss"] * tau, 0.0)[:, None]
        dz = torch.exp(z - lse) * g
        out["dlogits"] = dz.scatter_add_(1, at, -p * g).to(DTYPES[s["dtype"]])
    return out


# ------------------------------------------------------------------ the package's operators

def _kept(s, name, *shape, dtype):
    """A buffer that the caller keeps from call to call, as the package's callers do."""
    if name not in s:
        s[name] = torch.empty(shape, dtype=dtype, device="cuda")
    return s[name]


def _own_norm(s):
    import gradient_sync_ddp_gb300 as g
    T, D, dt = s["T"], s["D"], DTYPES[s["dtype"]]
    out = {"rstd": _kept(s, "out_rstd", T, dtype=torch.float32)}
    h = None
    if s["r"] is not None:
        out["h"] = h = _kept(s, "out_h", T, D, dtype=dt)
    if s["q8"]:
        q, scale = _kept(s, "out_q", T, D, dtype=torch.int8), _kept(s, "out_scale", T, dtype=torch.float32)
        g.rmsnorm_forward_q8(s["x"], s["gamma"], q, scale, EPS, residual=s["r"], h_out=h, rstd_out=out["rstd"])
        out["scale"] = scale
        out["values"] = torch.mul(q, scale[:, None], out=_kept(s, "out_values", T, D, dtype=torch.bfloat16))
    else:
        out["y"] = _kept(s, "out_y", T, D, dtype=dt)
        g.rmsnorm_forward(s["x"], s["gamma"], out["y"], EPS, residual=s["r"], h_out=h, rstd_out=out["rstd"])
    return out


def _own_norm_grad(s):
    import gradient_sync_ddp_gb300 as g
    T, D = s["T"], s["D"]
    if "ws" not in s:
        s["ws"] = torch.empty(g.rmsnorm_backward_workspace_bytes(T, D), dtype=torch.uint8, device="cuda")
    dx, dgamma = _kept(s, "out_dx", T, D, dtype=DTYPES[s["dtype"]]), _kept(s, "out_dgamma", D, dtype=torch.float32)
    g.rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["gamma"], dx, dgamma, s["ws"], dh=s["dh"])
    return {"dx": dx, "dgamma": dgamma}


def _own_product(s):
    import gradient_sync_ddp_gb300 as g
    M, N, K = s["M"], s["N"], s["K"]
    if "ws" not in s:
        s["ws"] = torch.empty(g.q8_matmul_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    out = _kept(s, "out_buf", M, N, dtype=DTYPES[s["out"]])
    g.q8_matmul(s["a"], s["sa"], s["w"], s["sw"], out, s["ws"])
    return out


def _own_distill(s):
    import gradient_sync_ddp_gb300 as g
    T, V, tau = s["T"], s["V"], s["tau"]
    out = {}
    if s["direction"] != "grad":
        out["loss"], out["lse"] = (_kept(s, "out_" + n, T, dtype=torch.float32) for n in ("loss", "lse"))
    if s["direction"] != "loss":
        out["dlogits"] = _kept(s, "out_dlogits", T, V, dtype=DTYPES[s["dtype"]])
    if s["direction"] == "loss":
        g.distill_topk_forward(s["logits"], s["index"], s["teacher"], out["loss"], out["lse"], temperature=tau)
    elif s["direction"] == "grad":
        g.distill_topk_backward(s["logits"], s["index"], s["teacher"], s["lse"], s["dloss"], out["dlogits"],
                                temperature=tau)
    else:
        g.distill_topk_forward_backward(s["logits"], s["index"], s["teacher"], s["dloss"], out["loss"], out["lse"],
                                        out["dlogits"], temperature=tau)
    return out


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "product": _plain_product, "distill": _plain_distill}
_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "product": _own_product, "distill": _own_distill}


def run(state):
    return (_OWN if own else _PLAIN)[state["kind"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["kind"] in ("norm", "norm_grad"):
        n, b = case["T"] * case["D"], BYTES[case["dtype"]]
        res = int(case["residual"])
        if case["kind"] == "norm":       # x, residual in; h, y (or 8 bits and scales), rstd out; gamma
            out = n + 4 * case["T"] if case["q8"] else n * b
            return {"bytes": n * b * (1 + 2 * res) + out + 4 * case["T"] + 4 * case["D"], "flops": 6 * n}
        return {"bytes": n * b * (3 + res) + 4 * case["T"] + 8 * case["D"], "flops": 11 * n}
    if case["kind"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + M * N * BYTES[case["out"]] + 4 * (M + N), "flops": 2 * M * N * K}
    n = case["T"] * case["V"]
    passes = 1 if case["direction"] == "loss" else 2
    return {"bytes": n * BYTES[case["dtype"]] * passes + 12 * case["T"] * case["k"] + 8 * case["T"],
            "flops": n * 4 * passes}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_norm(s):
    h = s["x"].double() + (0 if s["r"] is None else s["r"].double())
    ms = torch.einsum("td,td->t", h, h) / s["D"] + EPS
    y = h / ms.sqrt()[:, None] * s["gamma"].double()
    out = {"rstd": ms.pow(-0.5)}
    if s["r"] is not None:
        out["h"] = h
    if s["q8"]:
        # the 8-bit values themselves have the integers' step; only the scale has an exact value
        out["scale"], out["values"] = y.abs().max(dim=1).values / 127, None
    else:
        out["y"] = y
    return out


def _exact_norm_grad(s):
    dy, h, g, r = (s[n].double() for n in ("dy", "h", "gamma", "rstd"))
    inner = torch.einsum("td,td,d->t", dy, h, g)
    dx = torch.einsum("td,d,t->td", dy, g, r) - h * (r.pow(3) * inner / s["D"])[:, None]
    if s["dh"] is not None:
        dx = dx + s["dh"].double()
    return {"dx": dx, "dgamma": torch.einsum("td,td,t->d", dy, h, r)}


def _exact_product(s):
    # sums of at most 1024 products of 8-bit integers are whole numbers up to 2^24, which fp32 holds
    acc = torch.zeros(s["M"], s["N"], dtype=torch.float64, device="cuda")
    for k in range(0, s["K"], 1024):
        acc += s["a"][:, k:k + 1024].float() @ s["w"][:, k:k + 1024].float().T
    return torch.einsum("mn,m,n->mn", acc, s["sa"].double(), s["sw"].double())


def _exact_distill(s):
    tau, rows = s["tau"], []
    for t0 in range(0, s["T"], 512):     # blocks of tokens: 64-bit logits of all of them are large
        part = slice(t0, min(s["T"], t0 + 512))
        log_q = torch.log_softmax(s["logits"][part].double() / tau, 1)
        index, teacher = s["index"][part], s["teacher"][part].double() / tau
        absent = (index < 0) | (index >= s["V"])
        empty = absent.all(1)
        log_p = torch.log_softmax(teacher.masked_fill(absent & ~empty[:, None], -math.inf), 1)
        p = log_p.exp().masked_fill(empty[:, None], 0.0)
        one = {}
        if s["direction"] != "grad":
            terms = p * (log_p - log_q.gather(1, index.clamp(0, s["V"] - 1)))
            one["loss"] = tau ** 2 * terms.masked_fill(p == 0, 0.0).sum(1)
            one["lse"] = torch.logsumexp(s["logits"][part].double() / tau, 1)
        if s["direction"] != "loss":
            target = torch.zeros_like(log_q).scatter_add_(1, index.clamp(0, s["V"] - 1), p)
            q = log_q.exp().masked_fill(empty[:, None], 0.0)
            # kept in 32 bits: the 64-bit gradient of the largest case would not fit beside the rest
            one["dlogits"] = ((q - target) * (s["dloss"][part].double() * tau)[:, None]).float()
        rows.append(one)
    return {name: torch.cat([one[name] for one in rows]) for name in rows[0]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "product": _exact_product,
            "distill": _exact_distill}[case["kind"]](s)
