"""The training and serving operators around a fused product: what is measured, and their plain forms.

Three operators, each with its gradient:

linear         D = act(X W^T + bias) + residual, Z = X W^T + bias kept for the gradient on request.
               X (M, K), W (N, K), bias (N,), residual, D, Z (M, N).
               Gradient: dZ = dD act'(Z), dX = dZ W, dW = dZ^T X, dbias = sum of dZ over rows (fp32).
linear_xent    softmax cross entropy of the logits X W^T, which are never kept: X (T, K), W (V, K), target (T,) int64,
               lse[t] = log sum_v exp(logit[t, v]), loss[t] = lse[t] - logit[t, target[t]], 0 where the target is
               IGNORE.  Gradient: P[t, v] = (exp(logit[t, v] - lse[t]) - [v == target[t]]) dloss[t], 0 in ignored
               rows, dX = P W, dW = P^T X.
norm_residual  the residual step between two blocks: H' = H + scale * gate * norm_post(Y), X = norm_pre(H'), with
               root-mean-square or mean-and-variance norms over the rows, one gate row for each run of T / G rows.
               Gradient from (dX, dH'): dH, dY, and fp32 dw_post, dw_pre, dgate.
"""
import math

import torch

own = False

IGNORE = -100
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token through a projection of a decoder: bound by reading W once, and by latency
        {"name": "linear_token", "op": "linear", "dir": "fwd", "M": 1, "N": 8192, "K": 4096, "act": "silu",
         "dtype": "bf16"},
        # a prompt through the framework's 2400 x 3232 x 4096 shape, not tile multiples, with Z kept
        {"name": "linear_prompt", "op": "linear", "dir": "fwd", "M": 2400, "N": 3232, "K": 4096, "act": "gelu",
         "dtype": "f16"},
        # the framework's headline size
        {"name": "linear_8192", "op": "linear", "dir": "fwd", "M": 8192, "N": 8192, "K": 8192, "act": "gelu",
         "dtype": "bf16"},
        # the gradient of an up projection over a training batch
        {"name": "linear_grad", "op": "linear", "dir": "bwd", "M": 8192, "N": 8192, "K": 2048, "act": "silu",
         "dtype": "bf16"},
        # odd and ragged: no size is a multiple of 8, every row starts at an odd offset
        {"name": "linear_grad_odd", "op": "linear", "dir": "bwd", "M": 1001, "N": 1003, "K": 999, "act": "relu",
         "dtype": "f16"},
        # the log probability of one token over a large vocabulary of odd size
        {"name": "xent_token", "op": "xent", "dir": "fwd", "T": 1, "V": 100003, "K": 4096, "dtype": "bf16"},
        # loss and gradients over a small batch, every size odd in its way
        {"name": "xent_train_small", "op": "xent", "dir": "train", "T": 333, "V": 9999, "K": 1000, "dtype": "f16"},
        # loss and gradients over training batches: the usual and the largest
        {"name": "xent_train", "op": "xent", "dir": "train", "T": 2048, "V": 32768, "K": 2048, "dtype": "bf16"},
        {"name": "xent_train_large", "op": "xent", "dir": "train", "T": 4096, "V": 100003, "K": 4096,
         "dtype": "bf16"},
        # one token between two blocks: latency alone
        {"name": "norm_token", "op": "norm", "dir": "fwd", "T": 1, "H": 4096, "G": 1, "post": "rms", "pre": "rms",
         "dtype": "bf16", "stream": "bf16"},
        # a batch with a gate row for each of 8 sequences, the residual stream held in fp32
        {"name": "norm_batch", "op": "norm", "dir": "fwd", "T": 8192, "H": 8192, "G": 8, "post": "rms", "pre": "rms",
         "dtype": "bf16", "stream": "f32"},
        # its gradient, with means subtracted and a width that is no multiple of 8
        {"name": "norm_grad", "op": "norm", "dir": "bwd", "T": 8190, "H": 4100, "G": 1, "post": "layer",
         "pre": "layer", "dtype": "f16", "stream": "f16"},
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over the logarithm; a third of them multiples of 64, a third of 8."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    m = rng.choice((1, 8, 64))
    return max(lo, v // m * m) if v >= m else v


def draw(rng):
    op = rng.choice(("linear", "xent", "norm"))
    dtype = rng.choice(("bf16", "f16"))
    if op == "linear":
        return {"op": op, "dir": rng.choice(("fwd", "bwd")), "M": _spread(rng, 1, 8192), "N": _spread(rng, 64, 8192),
                "K": _spread(rng, 64, 8192), "act": rng.choice(("identity", "relu", "gelu", "silu")), "dtype": dtype}
    if op == "xent":
        return {"op": op, "dir": rng.choice(("fwd", "train")), "T": _spread(rng, 1, 4096),
                "V": _spread(rng, 1000, 100003), "K": _spread(rng, 64, 4096), "dtype": dtype}
    t = _spread(rng, 1, 8192)
    g = rng.choice([d for d in (1, 2, 4, 8, t) if t % d == 0])
    return {"op": op, "dir": rng.choice(("fwd", "bwd")), "T": t, "H": _spread(rng, 64, 8192), "G": g,
            "post": rng.choice(("rms", "layer", "none")), "pre": rng.choice(("rms", "layer")), "dtype": dtype,
            "stream": rng.choice((dtype, "f32"))}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, to=t, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(to)

    s = dict(case)
    if case["op"] == "linear":
        m, n, k = case["M"], case["N"], case["K"]
        s["x"] = normal(m, k)
        s["w"] = normal(n, k, std=k ** -0.5)
        if case["dir"] == "fwd":
            s["bias"], s["residual"] = normal(n, std=0.5), normal(m, n)
        else:
            s["z"], s["dd"] = normal(m, n), normal(m, n)
    elif case["op"] == "xent":
        n, v, k = case["T"], case["V"], case["K"]
        s["x"] = normal(n, k)
        s["w"] = normal(v, k, std=2.0 * k ** -0.5)
        target = torch.randint(0, v, (n,), generator=g, device="cuda")
        if n > 1:  # a tenth of the rows (padding, prompts) does not count
            target = torch.where(torch.rand(n, generator=g, device="cuda") < 0.1, IGNORE, target)
        s["target"] = target
        # the mean over a batch; fp16 gradients come with a loss scale
        s["dloss"] = torch.full((n,), (4096.0 if case["dtype"] == "f16" else 1.0) / n, device="cuda")
    else:
        n, h, u = case["T"], case["H"], TYPES[case["stream"]]
        s["y"] = normal(n, h, std=3.0, mean=0.25)
        s["gate"] = normal(case["G"], h, std=0.3, mean=0.5)
        s["w_post"] = normal(h, std=0.1, mean=1.0)
        s["w_pre"] = normal(h, std=0.1, mean=1.0)
        s["scale"] = 0.7
        if case["dir"] == "fwd":
            s["h"] = normal(n, h, std=2.0, to=u, mean=-0.5)
        else:
            s["h_out"] = normal(n, h, std=2.0, to=u, mean=-0.5)
            s["dx"], s["dh_out"] = normal(n, h), normal(n, h, to=u)
    return s


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "xent": _plain_xent, "norm": _plain_norm}[state["op"]](state)


def _own(s):
    import dense_gemm_elementwise_amd as ops
    if s["op"] == "linear":
        if s["dir"] == "fwd":
            if s["M"] == 1:  # serving keeps no Z
                return ops.linear(s["x"], s["w"], s["bias"], s["residual"], act=s["act"])
            return ops.linear(s["x"], s["w"], s["bias"], s["residual"], act=s["act"], save_z=True)
        return ops.linear_backward(s["dd"], s["x"], s["w"], s["z"], act=s["act"])
    if s["op"] == "xent":
        loss, lse = ops.linear_xent(s["x"], s["w"], s["target"], ignore_index=IGNORE)
        if s["dir"] == "fwd":
            return loss, lse
        dx, dw = ops.linear_xent_backward(s["dloss"], s["x"], s["w"], s["target"], lse, ignore_index=IGNORE)
        return loss, lse, dx, dw
    w_post = s["w_post"] if s["post"] != "none" else None
    kw = dict(w_post=w_post, w_pre=s["w_pre"], gate=s["gate"], scale=s["scale"], post=s["post"], pre=s["pre"],
              eps=EPS)
    if s["dir"] == "fwd":
        return ops.norm_residual(s["h"], s["y"], **kw)
    return ops.norm_residual_backward(s["dx"], s["dh_out"], s["h_out"], s["y"], **kw)


# The plain forms: elementary operations on fp32 copies, rounded once at the end.

def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    return torch.ones_like(z)


def _plain_linear(s):
    t, x, w = s["x"].dtype, s["x"].float(), s["w"].float()
    if s["dir"] == "fwd":
        z = x @ w.t() + s["bias"].float()
        d = (_act(z, s["act"]) + s["residual"].float()).to(t)
        return d if s["M"] == 1 else (d, z.to(t))
    dz = s["dd"].float() * _act_grad(s["z"].float(), s["act"])
    return (dz @ w).to(t), (dz.t() @ x).to(t), dz.sum(0)


def _plain_xent(s):
    t, x, w, target = s["x"].dtype, s["x"].float(), s["w"].float(), s["target"]
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    lse = (logits - top).exp().sum(1).log() + top[:, 0]
    counts = target != IGNORE
    at = torch.where(counts, target, 0)[:, None]
    loss = torch.where(counts, lse - logits.gather(1, at)[:, 0], 0.0)
    if s["dir"] == "fwd":
        return loss, lse
    scale = torch.where(counts, s["dloss"], 0.0)[:, None]
    p = logits.sub_(lse[:, None]).exp_().mul_(scale)
    p.scatter_add_(1, at, -scale)
    return loss, lse, (p @ w).to(t), (p.t() @ x).to(t)


def _norm(v, kind):
    """The normalised rows and the reciprocal of their scale."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * r, r


def _norm_grad(dn, n, r, kind):
    dn = dn - n * (dn * n).mean(1, keepdim=True)
    if kind == "layer":
        dn = dn - dn.mean(1, keepdim=True)
    return dn * r


def _plain_norm(s):
    post, pre, scale = s["post"], s["pre"], s["scale"]
    rows = s["T"] // s["G"]
    y = s["y"].float()
    gate = s["gate"].float().repeat_interleave(rows, 0)
    w_pre = s["w_pre"].float()
    yn, yr = _norm(y, post) if post != "none" else (y, None)
    yw = yn * s["w_post"].float() if post != "none" else yn
    if s["dir"] == "fwd":
        h = s["h"].float() + scale * gate * yw
        return h.to(s["h"].dtype), (_norm(h, pre)[0] * w_pre).to(s["y"].dtype)
    hn, hr = _norm(s["h_out"].float(), pre)
    dx = s["dx"].float()
    dh = s["dh_out"].float() + _norm_grad(dx * w_pre, hn, hr, pre)
    dyw = scale * gate * dh
    dgate = (scale * yw * dh).view(s["G"], rows, -1).sum(1)
    dw_pre = (dx * hn).sum(0)
    if post == "none":
        return dh.to(s["h_out"].dtype), dyw.to(s["y"].dtype), None, dw_pre, dgate
    dy = _norm_grad(dyw * s["w_post"].float(), yn, yr, post)
    return dh.to(s["h_out"].dtype), dy.to(s["y"].dtype), (dyw * yn).sum(0), dw_pre, dgate


def work(case):
    """Inputs read once, outputs written once, and the products that no form can do without."""
    if case["op"] == "linear":
        m, n, k = case["M"], case["N"], case["K"]
        operands = m * k + n * k
        if case["dir"] == "fwd":
            return {"bytes": 2 * (operands + n + m * n * (2 if m == 1 else 3)), "flops": 2 * m * n * k}
        return {"bytes": 2 * (2 * operands + 2 * m * n) + 4 * n, "flops": 4 * m * n * k}
    if case["op"] == "xent":
        n, v, k = case["T"], case["V"], case["K"]
        train = case["dir"] == "train"
        return {"bytes": 2 * (n + v) * k * (2 if train else 1) + (20 if train else 16) * n,
                "flops": (6 if train else 2) * n * v * k}
    n, h = case["T"], case["H"]
    e = 4 if case["stream"] == "f32" else 2
    weights = 2 * (case["G"] + (1 if case["post"] == "none" else 2)) * h
    if case["dir"] == "fwd":
        return {"bytes": n * h * (2 * e + 4) + weights, "flops": 12 * n * h}
    return {"bytes": n * h * (3 * e + 6) + 3 * weights, "flops": 30 * n * h}


def exact(case, seed):
    """The definitions in 64 bits; the gradients by differentiating the definition, not by its formulas."""
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    with torch.enable_grad():
        if case["op"] == "linear":
            f = {"identity": lambda z: z, "relu": torch.nn.functional.relu, "silu": torch.nn.functional.silu,
                 "gelu": torch.nn.functional.gelu}[case["act"]]
            if case["dir"] == "fwd":
                z = torch.mm(d["x"], d["w"].t()) + d["bias"][None, :]
                out = f(z) + d["residual"]
                return out if case["M"] == 1 else (out, z)
            z = d["z"].requires_grad_()
            dz, = torch.autograd.grad(f(z), z, d["dd"])
            return torch.mm(dz, d["w"]), torch.mm(dz.t(), d["x"]), dz.sum(0)
        if case["op"] == "xent":
            logits = torch.mm(d["x"], d["w"].t()).requires_grad_(case["dir"] == "train")
            lse = torch.logsumexp(logits, 1)
            loss = torch.nn.functional.cross_entropy(logits, s["target"], reduction="none", ignore_index=IGNORE)
            if case["dir"] == "fwd":
                return loss, lse
            p, = torch.autograd.grad(loss, logits, d["dloss"])
            return loss.detach(), lse.detach(), torch.mm(p, d["w"]), torch.mm(p.t(), d["x"])

        def norm(v, kind):
            if kind == "none":
                return v
            if kind == "layer":
                return (v - v.mean(1, keepdim=True)) / torch.sqrt(v.var(1, unbiased=False, keepdim=True) + EPS)
            return v / torch.sqrt(v.pow(2).mean(1, keepdim=True) + EPS)

        rows = case["T"] // case["G"]
        leaves = {k: d[k].requires_grad_() for k in ("y", "gate", "w_post", "w_pre")}
        w_post = leaves["w_post"] if case["post"] != "none" else 1.0
        step = s["scale"] * torch.repeat_interleave(leaves["gate"], rows, 0) * (norm(leaves["y"], case["post"]) * w_post)
        if case["dir"] == "fwd":
            h = d["h"] + step
            return h.detach(), (norm(h, case["pre"]) * leaves["w_pre"]).detach()
        # H' is given: its gradient is dH' and what comes back through X, and goes on to H and to the step
        h = d["h_out"].requires_grad_()
        x = norm(h, case["pre"]) * leaves["w_pre"]
        back, dw_pre = torch.autograd.grad(x, (h, leaves["w_pre"]), d["dx"])
        dh = d["dh_out"] + back
        if case["post"] == "none":
            dy, dgate = torch.autograd.grad(step, (leaves["y"], leaves["gate"]), dh)
            return dh, dy, None, dw_pre, dgate
        dy, dw_post, dgate = torch.autograd.grad(step, (leaves["y"], leaves["w_post"], leaves["gate"]), dh)
        return dh, dy, dw_post, dw_pre, dgate
