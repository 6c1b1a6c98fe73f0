"""The training and serving operators on the GPU against their definitions in
64 bits, with elementwise bounds that are derived from the roundings each
operator makes:

 * u(t) = eps(t) / 2 relative for the one rounding of an output (plus half the
   smallest subnormal for fp16);
 * fp32 sums of n products: at most (n + 2) 2^-24 of the sum of magnitudes;
 * an activation or its derivative: 4e-6 of its magnitude, and 1.13 times the
   error of its argument (the largest slope of gelu);
 * an intermediate that is an MFMA operand (dZ, P): u(t) of its magnitude,
   summed with the magnitudes of the other operand.
"""
import math

import pytest
import torch

import dense_gemm_elementwise_amd as ge

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E24 = 2.0 ** -24
IGNORE = -100


def log(*a):
    print(*a, flush=True)


def u(t):
    return torch.finfo(t).eps / 2


def floor_of(t):
    return {F16: 2.0 ** -25, BF16: 2.0 ** -134, F32: 2.0 ** -150}[t]


def rnd(g, *shape, std=1.0, mean=0.0, t=BF16):
    return (torch.randn(shape, generator=g, dtype=torch.float32) * std + mean).to(t).to(DEV)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def close(name, got, want, bound):
    """|got - want| <= bound everywhere, `bound` a float64 tensor without the output's own rounding."""
    got64 = got.double().cpu()
    want, bound = want.cpu(), bound.cpu() if isinstance(bound, torch.Tensor) else bound
    assert got64.shape == want.shape, name
    assert not got64.isnan().any(), f"{name}: NaN"
    lim = u(got.dtype) * want.abs() + floor_of(got.dtype) + bound * (1 + u(got.dtype))
    bad = (got64 - want).abs() > lim
    if bad.any():
        i = int(bad.flatten().nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{got64.flatten()[i]} want {want.flatten()[i]} bound {lim.flatten()[i]}")


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z * 0.5 ** 0.5)
    return z


def act_grad64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        return torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
    if act == "gelu":
        return 0.5 * torch.erfc(-z * 0.5 ** 0.5) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def linear_ref(x, w, bias, residual, act):
    """(D, Z) in 64 bits and the bounds of their errors before the last rounding."""
    x, w = x.double().cpu(), w.double().cpu()
    z = x @ w.t()
    mag = x.abs() @ w.abs().t()
    if bias is not None:
        z = z + bias.double().cpu()
        mag = mag + bias.double().cpu().abs()
    bz = (x.shape[1] + 3) * E24 * mag
    a = act64(z, act)
    d, bd = a, 1.13 * bz + 4e-6 * a.abs()
    if residual is not None:
        d = d + residual.double().cpu()
        bd = bd + E24 * d.abs()
    return d, bd, z, bz


SHAPES = [(1, 64, 64), (1, 1, 1), (1, 1003, 999), (3, 40, 8), (16, 520, 300), (17, 64, 64), (17, 1, 1), (33, 7, 5),
          (64, 129, 72), (128, 128, 32), (129, 257, 33), (200, 264, 520), (257, 255, 264), (300, 1000, 1001)]


@pytest.mark.parametrize("t", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear(shape, t):
    M, N, K = shape
    for n, act in enumerate(("identity", "relu", "gelu", "silu")):
        log(f"[linear] {shape} {t} {act}")
        g = gen(M * 31 + N + K + n)
        x, w = rnd(g, M, K, t=t), rnd(g, N, K, std=K ** -0.5, t=t)
        bias = rnd(g, N, std=0.5, t=t) if n != 1 else None
        residual = rnd(g, M, N, t=t) if n != 2 else None
        d, bd, z, bz = linear_ref(x, w, bias, residual, act)
        got = ge.linear(x, w, bias, residual, act=act, save_z=True)
        close("D", got[0], d, bd)
        close("Z", got[1], z, bz)
        assert torch.equal(ge.linear(x, w, bias, residual, act=act), got[0])


# every tile and the split form: grids and depths that the plan gives them
@pytest.mark.parametrize("shape", [(2048, 2048, 96), (2304, 3232, 128), (1280, 4400, 64), (4400, 1290, 72),
                                   (512, 768, 4096), (40, 128, 8192), (130, 136, 2056)], ids=str)
@pytest.mark.parametrize("t", [BF16, F16], ids=["bf16", "f16"])
def test_linear_tiles(shape, t):
    M, N, K = shape
    log(f"[linear tiles] {shape} {t}")
    g = gen(M + N + K)
    x, w = rnd(g, M, K, t=t), rnd(g, N, K, std=K ** -0.5, t=t)
    bias, residual = rnd(g, N, t=t), rnd(g, M, N, t=t)
    got = ge.linear(x, w, bias, residual, act="silu", save_z=True)
    d, bd, z, bz = linear_ref(x, w, bias, residual, "silu")
    close("D", got[0], d, bd)
    close("Z", got[1], z, bz)


@pytest.mark.parametrize("M", [2, 70])
def test_linear_strides(M):
    """Column slices of wider tensors at odd offsets, read in place."""
    g = gen(5)
    N, K = 72, 48
    for off in (0, 1, 8):
        log(f"[linear strides] M={M} off={off}")
        x = rnd(g, M, K + 24)[:, off:off + K]
        w = rnd(g, N, K + 16, std=K ** -0.5)[:, off:off + K]
        residual = rnd(g, M, N + 9)[:, off:off + N]
        d, bd, z, bz = linear_ref(x, w, None, residual, "gelu")
        got = ge.linear(x, w, None, residual, act="gelu", save_z=True)
        close("D", got[0], d, bd)
        close("Z", got[1], z, bz)
        dd = rnd(g, M, N + 9)[:, off:off + N]
        a, b = (ge.linear_backward(dd.contiguous(), x.contiguous(), w.contiguous(), got[1], act="gelu"),
                ge.linear_backward(dd, x, w, got[1], act="gelu"))
        for p, q in zip(a, b):
            assert torch.equal(p, q)


@pytest.mark.parametrize("t", [BF16, F16], ids=["bf16", "f16"])
def test_linear_special_values(t):
    """Infinities and NaN stay in their own row or column; the tiles' padding stays out."""
    g = gen(9)
    for M in (3, 40):
        x, w = rnd(g, M, 72, t=t), rnd(g, 24, 72, t=t)
        clean = ge.linear(x, w, act="silu")
        x[1, 3], x[2, 5], w[7, 0] = float("nan"), float("inf"), float("-inf")
        got = ge.linear(x, w, act="silu")
        assert got[1].isnan().all()
        keep = [i for i in range(M) if i not in (1, 2)]
        cols = [i for i in range(24) if i != 7]
        assert torch.equal(got[keep][:, cols], clean[keep][:, cols])
        # relu keeps a NaN, and clears negatives to +0
        z = ge.linear(x, w, act="relu")
        assert z[1].isnan().all() and (z[keep][:, cols] >= 0).all()


def linear_grad_ref(dd, x, w, z, act):
    dd, x, w, z = (v.double().cpu() for v in (dd, x, w, z))
    dz = dd * act_grad64(z, act)
    e = 4e-6 * (dd.abs() * (1 + z.abs()) if act in ("gelu", "silu") else dz.abs())  # of the factor, fp32
    t = dz, e
    return t, x, w


@pytest.mark.parametrize("t", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 64, 64), (1, 1, 1), (5, 9, 3), (64, 64, 64), (65, 130, 72), (31, 257, 33),
                                   (300, 70, 1000), (1001, 203, 99), (128, 2048, 136), (2100, 1100, 264),
                                   (8, 4096, 96), (4096, 40, 48)], ids=str)
def test_linear_backward(shape, t):
    M, N, K = shape
    for n, act in enumerate(("identity", "relu", "gelu", "silu")):
        log(f"[linear_backward] {shape} {t} {act}")
        g = gen(M + 7 * N + K + n)
        x, w = rnd(g, M, K, t=t), rnd(g, N, K, std=K ** -0.5, t=t)
        z, dd = rnd(g, M, N, std=2.0, t=t), rnd(g, M, N, t=t)
        (dz, e), x64, w64 = linear_grad_ref(dd, x, w, z, act)
        dx, dw, db = ge.linear_backward(dd, x, w, z, act=act)
        ez = e + (u(t) * dz.abs() + floor_of(t) if act != "identity" else 0)
        close("dX", dx, dz @ w64, ez @ w64.abs() + (N + 2) * E24 * (dz.abs() @ w64.abs()))
        close("dW", dw, dz.t() @ x64, ez.t() @ x64.abs() + (M + 2) * E24 * (dz.abs().t() @ x64.abs()))
        close("dbias", db, dz.sum(0), e.sum(0) + (M + 2) * E24 * dz.abs().sum(0))
        # each alone gives the same bits
        one = ge.linear_backward(dd, x, w, z, act=act, need_dx=False, need_dbias=False)
        assert one[0] is None and one[2] is None and torch.equal(one[1], dw)
        one = ge.linear_backward(dd, x, w, z, act=act, need_dw=False, need_dbias=False)
        assert one[1] is None and torch.equal(one[0], dx)
        one = ge.linear_backward(dd, x, w, z, act=act, need_dw=False, need_dx=False)
        assert torch.equal(one[2], db)


@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
def test_act_gradient_everywhere(act):
    """act'(z) at every finite bf16 z and at the infinities, through an identity product."""
    log(f"[act'] {act}")
    z = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
    z = z[~z.isnan()][:65024].reshape(-1, 64).to(DEV)
    eye = torch.eye(64, dtype=BF16, device=DEV)
    dx, _, _ = ge.linear_backward(torch.ones_like(z), torch.zeros_like(z), eye, z, act=act, need_dw=False)
    z64 = z.double().cpu().clamp(-300, 300)
    want = act_grad64(z64, act)
    close("act'", dx, want, 4e-6 * (1 + z64.abs()) * torch.sigmoid(z64 + 3))


def test_linear_gradient_against_differences():
    """The gradient of sum(D * c) by central differences of the 64-bit forward."""
    g = gen(3)
    M, N, K = 4, 6, 8
    for act in ("gelu", "silu"):
        x, w, c = rnd(g, M, K, t=F16), rnd(g, N, K, std=0.3, t=F16), rnd(g, M, N, t=F16)
        _, z = ge.linear(x, w, act=act, save_z=True)
        dx, dw, db = ge.linear_backward(c, x, w, z, act=act)
        x64, w64, c64 = x.double().cpu(), w.double().cpu(), c.double().cpu()

        def f(xv, wv, bv):
            return (act64(xv @ wv.t() + bv, act) * c64).sum()
        zero, h = torch.zeros(N, dtype=torch.float64), 1e-5

        def diff(i, args):
            out = torch.zeros_like(args[i])
            for j in range(out.numel()):
                lo, hi = [a.clone() for a in args], [a.clone() for a in args]
                lo[i].view(-1)[j] -= h
                hi[i].view(-1)[j] += h
                out.view(-1)[j] = (f(*hi) - f(*lo)) / (2 * h)
            return out
        args = (x64, w64, zero)
        # Z's rounding moves act' by at most 1.2 u |z|, dZ's by u: 3 roundings of magnitudes up to 4
        for got, i, other in ((dx, 0, w64), (dw, 1, x64), (db, 2, torch.ones(N, 1, dtype=torch.float64))):
            scale = (c64.abs().sum() * other.abs().max()).item()
            assert (got.double().cpu() - diff(i, args)).abs().max() < 8 * u(F16) * scale, (act, i)


# ---- cross entropy ------------------------------------------------------------
def xent_ref(x, w, target):
    x, w = x.double().cpu(), w.double().cpu()
    logits = x @ w.t()
    be = (x.shape[1] + 2) * E24 * (x.abs() @ w.abs().t())  # of every logit
    lse = torch.logsumexp(logits, 1)
    t = target.cpu()
    live = t != IGNORE
    at = torch.where(live, t, 0)[:, None]
    loss = torch.where(live, lse - logits.gather(1, at)[:, 0], 0.0)
    return logits, be, lse, loss, live, at


XSHAPES = [(1, 1000, 64), (1, 1, 1), (1, 5, 3), (7, 129, 33), (16, 2000, 520), (17, 1000, 64), (130, 257, 72),
           (300, 1003, 99), (256, 4100, 264), (40, 20000, 48), (600, 9000, 40)]


@pytest.mark.parametrize("t", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", XSHAPES, ids=str)
def test_linear_xent(shape, t):
    T, V, K = shape
    log(f"[xent] {shape} {t}")
    g = gen(T + V + K)
    x, w = rnd(g, T, K, t=t), rnd(g, V, K, std=2 * K ** -0.5, t=t)
    target = torch.randint(0, V, (T,), generator=g)
    target[:: 5] = IGNORE if T > 1 else target[0]
    if T > 4:
        target[1], target[2] = 0, V - 1
    dloss = torch.rand(T, generator=g) * (4096.0 if t == F16 else 1.0) / T
    target, dloss = target.to(DEV), dloss.to(DEV)
    logits, be, lse, loss, live, at = xent_ref(x, w, target)
    got_loss, got_lse = ge.linear_xent(x, w, target, ignore_index=IGNORE)
    # of lse: the largest error of a logit, the sums (a tree under 64 deep), the exponentials and the logarithm
    bl = be.amax(1) + 1e-5 + lse.abs() * 2.0 ** -23
    close("lse", got_lse, lse, bl)
    close("loss", got_loss, loss, torch.where(live, bl + be.gather(1, at)[:, 0] + 2 * E24 * logits.abs().amax(1), 0.0))
    assert (got_loss[~live.to(DEV)] == 0).all()

    dx, dw = ge.linear_xent_backward(dloss, x, w, target, got_lse, ignore_index=IGNORE)
    p = torch.exp(logits - lse[:, None])
    one = torch.zeros_like(p).scatter_(1, at, 1.0)
    scale = torch.where(live, dloss.double().cpu(), 0.0)[:, None]
    P = (p - one) * scale
    eP = p * scale * (be + bl[:, None] + 2e-6 * (1 + (logits - lse[:, None]).abs())) + (u(t) + 4 * E24) * P.abs() \
        + scale.max() * 2.0 ** -40  # fp16 subnormals of the scaled P
    x64, w64 = x.double().cpu(), w.double().cpu()
    close("dX", dx, P @ w64, eP @ w64.abs() + (V + 9) * E24 * (P.abs() @ w64.abs()))
    close("dW", dw, P.t() @ x64, eP.t() @ x64.abs() + (T + 9) * E24 * (P.abs().t() @ x64.abs()))
    only = ge.linear_xent_backward(dloss, x, w, target, got_lse, ignore_index=IGNORE, need_dx=False)
    assert only[0] is None and torch.equal(only[1], dw)
    only = ge.linear_xent_backward(dloss, x, w, target, got_lse, ignore_index=IGNORE, need_dw=False)
    assert only[1] is None and torch.equal(only[0], dx)


def test_xent_several_pieces():
    """A batch large enough for several pieces of the vocabulary: the fp32 accumulator between them."""
    log("[xent pieces]")
    g = gen(21)
    T, V, K = 9000, 16500, 24
    x, w = rnd(g, T, K), rnd(g, V, K, std=2 * K ** -0.5)
    target = torch.randint(0, V, (T,), generator=g).to(DEV)
    loss, lse = ge.linear_xent(x, w, target)
    dloss = torch.full((T,), 1.0 / T, device=DEV)
    dx, dw = ge.linear_xent_backward(dloss, x, w, target, lse)
    # the same in fp32 on the GPU; bounds of both: sums in fp32, P in bf16
    p = x.float() @ w.float().t()
    ref_lse = torch.logsumexp(p, 1)
    assert (lse - ref_lse).abs().max() < 1e-4
    p = (p - ref_lse[:, None]).exp_()
    p[torch.arange(T, device=DEV), target] -= 1
    p /= T
    ref_dx, ref_dw = p @ w.float(), p.t() @ x.float()
    for name, got, ref, mag in (("dX", dx, ref_dx, p.abs() @ w.float().abs()),
                                ("dW", dw, ref_dw, p.abs().t() @ x.float().abs())):
        bad = (got.float() - ref).abs() > u(BF16) * ref.abs() + (u(BF16) + 2e-4) * mag
        assert not bad.any(), name


def test_xent_masks():
    log("[xent masks]")
    g = gen(8)
    for T in (5, 40):
        V, K = 300, 64
        x, w = rnd(g, T, K), rnd(g, V, K, std=0.3)
        none = torch.full((T,), IGNORE, device=DEV)
        loss, lse = ge.linear_xent(x, w, none)
        assert (loss == 0).all() and lse.isfinite().all()
        dl = torch.ones(T, device=DEV)
        dx, dw = ge.linear_xent_backward(dl, x, w, none, lse)
        assert (dx == 0).all() and (dw == 0).all()
        # a zero incoming gradient
        tgt = torch.randint(0, V, (T,), generator=g).to(DEV)
        _, lse = ge.linear_xent(x, w, tgt)
        dx, dw = ge.linear_xent_backward(dl * 0, x, w, tgt, lse)
        assert (dx == 0).all() and (dw == 0).all()
        # out of range: NaN, in its own row only; an ignore index inside the range masks too
        bad = tgt.clone()
        bad[0], bad[1] = V, -1
        loss, _ = ge.linear_xent(x, w, bad)
        good, _ = ge.linear_xent(x, w, tgt)
        assert loss[:2].isnan().all() and torch.equal(loss[2:], good[2:])
        loss, lse = ge.linear_xent(x, w, tgt, ignore_index=int(tgt[2]))
        assert (loss[tgt == tgt[2]] == 0).all()
        dx, _ = ge.linear_xent_backward(dl, x, w, tgt, lse, ignore_index=int(tgt[2]))
        assert (dx[tgt == tgt[2]] == 0).all()
        # an ignored row's NaN stays out of the other rows and of dX
        x2 = x.clone()
        x2[3] = float("nan")
        masked = tgt.clone()
        masked[3] = IGNORE
        l2, lse2 = ge.linear_xent(x2, w, masked)
        assert l2[3] == 0 and torch.equal(l2[4:], good[4:])
        dx, _ = ge.linear_xent_backward(dl, x2, w, masked, lse2)
        assert (dx[3] == 0).all() and dx.isfinite().all()


def test_xent_extreme_logits():
    """Logits at 3e4, where exp overflows, and all-equal rows."""
    log("[xent extremes]")
    for T in (3, 40):
        K, V = 16, 700
        x = torch.full((T, K), 40.0, dtype=F16, device=DEV)
        w = torch.full((V, K), 47.0, dtype=F16, device=DEV)
        w[5] = -47.0
        tgt = torch.full((T,), 5, device=DEV)
        loss, lse = ge.linear_xent(x, w, tgt)
        top = 40.0 * 47.0 * K
        assert (lse.double().cpu() - (top + math.log(V - 1))).abs().max() <= top * 2.0 ** -23 + 1e-5
        assert (loss.double().cpu() - (2 * top + math.log(V - 1))).abs().max() <= 4 * top * 2.0 ** -23
        tgt[:] = 6
        loss, lse = ge.linear_xent(x, w, tgt)
        dx, dw = ge.linear_xent_backward(torch.ones(T, device=DEV), x, w, tgt, lse)
        assert dx.isfinite().all() and dw.isfinite().all()


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1.0, 2.0 ** 20])
def test_xent_gradient_scales(scale):
    """P keeps its digits in 16 bits whatever the incoming gradient's size."""
    log(f"[xent scale] {scale}")
    g = gen(4)
    T, V, K = 33, 500, 32
    t = BF16
    x, w = rnd(g, T, K, t=t), rnd(g, V, K, t=t, std=0.3)
    tgt = torch.randint(0, V, (T,), generator=g).to(DEV)
    _, lse = ge.linear_xent(x, w, tgt)
    a = ge.linear_xent_backward(torch.full((T,), 1.0, device=DEV), x, w, tgt, lse)
    s = 2.0 ** round(math.log2(scale))
    b = ge.linear_xent_backward(torch.full((T,), s, device=DEV), x, w, tgt, lse)
    for p, q in zip(a, b):
        assert torch.equal((p.float() * s).to(t), q)


# ---- norms ----------------------------------------------------------------------
def norm64(v, kind, eps):
    """(normalised rows, reciprocal scale, mean)"""
    mu = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros(v.shape[0], 1, dtype=torch.float64)
    c = v - mu
    r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    return c * r, r, mu


NSHAPES = [(1, 64, 1), (1, 1, 1), (4, 5, 2), (3, 100, 3), (17, 513, 1), (8, 1024, 4), (30, 1030, 30), (12, 2048, 2),
           (9, 4100, 3), (5, 8192, 1), (6, 8200, 2), (2, 16384, 1), (700, 72, 7), (2050, 40, 1025), (1200, 136, 1)]
NKINDS = [("rms", "rms"), ("layer", "layer"), ("none", "rms"), ("rms", "layer")]


@pytest.mark.parametrize("t,s", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)],
                         ids=["bf16", "f16", "bf16-f32", "f16-f32"])
@pytest.mark.parametrize("shape", NSHAPES, ids=str)
def test_norm_residual(shape, t, s):
    T, H, G = shape
    eps = 1e-5
    for n, (post, pre) in enumerate(NKINDS):
        log(f"[norm] {shape} {t} {s} {post} {pre}")
        g = gen(T + H + G + n)
        h, y = rnd(g, T, H, std=2.0, mean=-0.5, t=s), rnd(g, T, H, std=3.0, mean=0.25, t=t)
        gate = rnd(g, G, H, std=0.3, mean=0.5, t=t) if n != 3 else None
        wo = rnd(g, H, std=0.1, mean=1.0, t=t) if post != "none" else None
        wi = rnd(g, H, std=0.1, mean=1.0, t=t) if n != 2 else None
        kw = dict(w_post=wo, w_pre=wi, gate=gate, scale=0.7, post=post, pre=pre, eps=eps)
        ho, x = ge.norm_residual(h, y, **kw)
        one = torch.ones(H, dtype=torch.float64)
        y64, h64 = y.double().cpu(), h.double().cpu()
        g64 = gate.double().cpu().repeat_interleave(T // G, 0) if gate is not None else one
        wo64 = wo.double().cpu() if wo is not None else one
        wi64 = wi.double().cpu() if wi is not None else one
        # of fp32 norms: 4e-6 of the value (sums of squares, rsqrt, three products) and the mean's
        # rounding, 2^-22 of the largest element
        if post != "none":
            yn, ry, _ = norm64(y64, post, eps)
            eyn = 4e-6 * yn.abs() + ry * y64.abs().amax(1, keepdim=True) * 2.0 ** -22
        else:
            yn, eyn = y64, y64.abs() * E24
        step = 0.7 * g64 * wo64 * yn
        hh = h64 + step
        eh = 0.7 * (g64 * wo64).abs() * eyn + 4 * E24 * (step.abs() + hh.abs())
        close("H'", ho, hh, eh)
        hn, rh, _ = norm64(hh, pre, eps)
        # every element of the row enters the scale: the relative error of the largest
        ehn = rh * eh + hn.abs() * (4e-6 + (eh * rh).amax(1, keepdim=True)) \
            + rh * hh.abs().amax(1, keepdim=True) * 2.0 ** -22 + (eh * rh).mean(1, keepdim=True)
        if H == 1 and pre == "layer":  # a single element less its mean: 0 times 1 / sqrt(eps)
            ehn = ehn + (hh.abs() * 2.0 ** -22 + eh) / math.sqrt(eps)
        close("X", x, hn * wi64, ehn * wi64.abs())

        if H > 8192:  # the gradient's limit
            continue
        # the gradient at the stored H'
        dx, dho = rnd(g, T, H, t=t), rnd(g, T, H, t=s)
        got = ge.norm_residual_backward(dx, dho, ho, y, **kw)
        H64 = ho.double().cpu()
        hn, rh, _ = norm64(H64, pre, eps)
        dx64, dho64 = dx.double().cpu(), dho.double().cpu()
        dn = dx64 * wi64
        c_h = (dn * hn).mean(1, keepdim=True)
        dm = dn.mean(1, keepdim=True) if pre == "layer" else 0.0
        dh = dho64 + (dn - hn * c_h - dm) * rh
        big = rh * H64.abs().amax(1, keepdim=True) * 2.0 ** -22 + 4e-6 * hn.abs()  # of hn
        mag = dn.abs() + hn.abs() * (dn * hn).abs().mean(1, keepdim=True) + dn.abs().mean(1, keepdim=True)
        edh = rh * (1e-5 * mag + big * c_h.abs() + hn.abs() * (dn.abs() * big).mean(1, keepdim=True)) \
            + 4 * E24 * dh.abs() + E24 * dho64.abs()
        close("dH", got[0], dh, edh)
        dyw = 0.7 * g64 * dh
        edyw = 0.7 * g64.abs() * edh + 3 * E24 * dyw.abs()
        d = dyw * wo64
        if post != "none":
            yn, ry, _ = norm64(y64, post, eps)
            c_y = (d * yn).mean(1, keepdim=True)
            m_y = d.mean(1, keepdim=True) if post == "layer" else 0.0
            dy = (d - yn * c_y - m_y) * ry
            ed = edyw * wo64.abs()
            magy = d.abs() + yn.abs() * (d * yn).abs().mean(1, keepdim=True) + d.abs().mean(1, keepdim=True)
            edy = ry * (1e-5 * magy + ed + yn.abs() * ((ed * yn.abs()).mean(1, keepdim=True)
                                                       + (d.abs() * eyn).mean(1, keepdim=True))
                        + eyn * c_y.abs() + ed.mean(1, keepdim=True))
        else:
            yn, dy, edy = y64, dyw, edyw
        close("dY", got[1], dy, edy)
        rows = (T + 4) * E24
        if wo is not None:
            close("dw_post", got[2], (dyw * yn).sum(0),
                  (edyw * yn.abs() + dyw.abs() * eyn).sum(0) + rows * (dyw * yn).abs().sum(0))
        else:
            assert got[2] is None
        if wi is not None:
            close("dw_pre", got[3], (dx64 * hn).sum(0), (dx64.abs() * big).sum(0) + rows * (dx64 * hn).abs().sum(0))
        else:
            assert got[3] is None
        if gate is not None:
            yw = 0.7 * yn * wo64
            v, e = yw * dh, yw.abs() * edh + 0.7 * wo64.abs() * eyn * dh.abs() + 4 * E24 * (yw * dh).abs()
            close("dgate", got[4], v.view(G, T // G, H).sum(1),
                  e.view(G, T // G, H).sum(1) + rows * v.abs().view(G, T // G, H).sum(1))
        else:
            assert got[4] is None


def test_norm_large_mean():
    """A mean of 1000 deviations costs the LAYER norm no more than the input's own rounding."""
    log("[norm mean]")
    g = gen(6)
    h = torch.zeros(4, 512, device=DEV)
    y = rnd(g, 4, 512, t=F16, std=1.0, mean=1000.0)
    _, x = ge.norm_residual(h, y, post="layer", pre="layer")
    want = norm64(norm64(y.double().cpu(), "layer", 1e-5)[0], "layer", 1e-5)[0]
    assert (x.double().cpu() - want).abs().max() < 5 * u(F16) * 4 + 1000 * 2.0 ** -21


def test_norm_gradient_against_differences():
    g = gen(13)
    T, H, G, eps, h = 4, 6, 2, 1e-3, 1e-5
    for post, pre in (("rms", "rms"), ("layer", "layer"), ("rms", "layer")):
        H0, y = rnd(g, T, H, t=F32), rnd(g, T, H, t=F16)
        gate, wo, wi = rnd(g, G, H, t=F16), rnd(g, H, t=F16), rnd(g, H, t=F16)
        kw = dict(w_post=wo, w_pre=wi, gate=gate, scale=0.7, post=post, pre=pre, eps=eps)
        ho, _ = ge.norm_residual(H0, y, **kw)
        cx, ch = rnd(g, T, H, t=F16), rnd(g, T, H, t=F32)
        got = ge.norm_residual_backward(cx, ch, ho, y, **kw)
        leaves = [v.double().cpu() for v in (H0, y, wo, wi, gate)]

        def f(h0, yv, wov, wiv, gv):
            hh = h0 + 0.7 * gv.repeat_interleave(T // G, 0) * norm64(yv, post, eps)[0] * wov
            return (hh * ch.double().cpu()).sum() + (norm64(hh, pre, eps)[0] * wiv * cx.double().cpu()).sum()
        for i, gr in enumerate(got):
            out = torch.zeros_like(leaves[i])
            for j in range(out.numel()):
                lo, hi = [a.clone() for a in leaves], [a.clone() for a in leaves]
                lo[i].view(-1)[j] -= h
                hi[i].view(-1)[j] += h
                out.view(-1)[j] = (f(*hi) - f(*lo)) / (2 * h)
            # dY is rounded to fp16; the rest fp32 from an fp32 H'
            lim = (u(F16) if gr.dtype == F16 else 0) * out.abs() + 2e-5 * (1 + out.abs().max())
            assert ((gr.double().cpu() - out).abs() <= lim).all(), (post, pre, i)


# ---- calls ------------------------------------------------------------------------
def test_empty_batches():
    log("[empty]")
    x, w = torch.empty(0, 64, dtype=BF16, device=DEV), torch.ones(48, 64, dtype=BF16, device=DEV)
    d, z = ge.linear(x, w, act="gelu", save_z=True)
    assert d.shape == z.shape == (0, 48)
    dx, dw, db = ge.linear_backward(d, x, w, z, act="gelu")
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    t = torch.empty(0, dtype=torch.int64, device=DEV)
    loss, lse = ge.linear_xent(x, w, t)
    assert loss.shape == lse.shape == (0,)
    dx, dw = ge.linear_xent_backward(loss, x, w, t, lse)
    assert dx.shape == (0, 64) and (dw == 0).all()
    v = torch.ones(64, dtype=BF16, device=DEV)
    ho, xo = ge.norm_residual(x, x, w_post=v, w_pre=v)
    assert ho.shape == xo.shape == (0, 64)
    out = ge.norm_residual_backward(x, x, x, x, w_post=v, w_pre=v)
    assert (out[2] == 0).all() and (out[3] == 0).all()


def test_refusals_on_the_gpu():
    x = torch.zeros(4, 8, dtype=F16, device=DEV)
    w = torch.zeros(6, 8, dtype=F16, device=DEV)
    for bad, err in (((x, w.to(BF16)), TypeError), ((x, w[:, :7]), ValueError), ((x, w.t()), ValueError),
                     ((x, w.cpu()), ValueError), ((x[None], w), ValueError),
                     ((x, w, torch.zeros(5, dtype=F16, device=DEV)), ValueError),
                     ((x, w, None, torch.zeros(6, 4, dtype=F16, device=DEV).t()), ValueError)):
        with pytest.raises(err):
            ge.linear(*bad)
    with pytest.raises(ValueError, match="act"):
        ge.linear(x, w, act="tanh")
    with pytest.raises(ValueError, match="needs z"):
        ge.linear_backward(torch.zeros(4, 6, dtype=F16, device=DEV), x, w, act="gelu")
    with pytest.raises(ValueError, match="requires grad"):
        ge.linear(x, w.clone().requires_grad_())
    with torch.no_grad():
        ge.linear(x, w.clone().requires_grad_())
    with pytest.raises(TypeError):
        ge.linear_xent(x, w, torch.zeros(4, device=DEV))
    with pytest.raises(ValueError):
        ge.linear_xent(x, w, torch.zeros(5, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError, match="divide"):
        ge.norm_residual(x, x, gate=torch.zeros(3, 8, dtype=F16, device=DEV))
    with pytest.raises(ValueError, match="overlap"):
        ge.norm_residual(x, x[:1].expand(4, 8))
    with pytest.raises(ValueError, match="pre"):
        ge.norm_residual(x, x, pre="none")
    with pytest.raises(ValueError, match="w_post"):
        ge.norm_residual(x, x, post="none", w_post=x[0])
    wide = torch.zeros(1, 16385, dtype=F16, device=DEV)
    with pytest.raises(ge.GemmEpiError):
        ge.norm_residual(wide, wide)


def operators_of(M, t=BF16):
    """A set of calls covering every operator, on fresh inputs: f() -> tuple of outputs."""
    g = gen(M)
    N, K, V = 264, 128, 1000
    x, w, b, r = rnd(g, M, K, t=t), rnd(g, N, K, t=t, std=0.1), rnd(g, N, t=t), rnd(g, M, N, t=t)
    wv = rnd(g, V, N, t=t, std=0.1)
    tgt = torch.randint(0, V, (M,), generator=g).to(DEV)
    v = rnd(g, N, t=t, mean=1.0, std=0.1)
    dl = torch.full((M,), 1.0 / M, device=DEV)
    ins = [x, w, b, r, wv, tgt, v, dl]

    def f(stream=None):
        k = dict(stream=stream)
        d, z = ge.linear(x, w, b, r, act="gelu", save_z=True, **k)
        ho, xo = ge.norm_residual(r, d, w_post=v, w_pre=v, **k)
        loss, lse = ge.linear_xent(xo, wv, tgt, **k)
        dxo, dwv = ge.linear_xent_backward(dl, xo, wv, tgt, lse, **k)
        dh, dd, dwo, dwi, _ = ge.norm_residual_backward(dxo, torch.zeros_like(ho) if stream is None else ho, ho, d,
                                                        w_post=v, w_pre=v, **k)
        dx, dw, db = ge.linear_backward(dd, x, w, z, act="gelu", **k)
        return d, z, ho, xo, loss, lse, dxo, dwv, dh, dd, dwo, dwi, dx, dw, db
    return f, ins


@pytest.mark.parametrize("M", [1, 200])
def test_repeats_and_streams(M):
    """The same bits every time, on the current stream, on a given one and on a current side stream."""
    log(f"[streams] M={M}")
    f, ins = operators_of(M)
    a, b = f(), f()
    torch.cuda.synchronize()
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = f()
    d1, d2 = f(side), f(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for p, q in zip(a, c):
        assert torch.equal(p, q)
    for p, q in zip(d1, d2):
        assert torch.equal(p, q)


@pytest.mark.parametrize("M", [1, 200])
def test_graph_capture(M):
    """Recorded into a HIP graph and replayed on changed inputs, with eager work between the replays."""
    log(f"[graph] M={M}")
    f, ins = operators_of(M)
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    for rep in range(4):
        ins[0].mul_(-0.5)
        ins[3].add_(0.25)
        for o in out:
            o.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        want = f()
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(got, want)):
            assert torch.equal(p, q), (rep, i)


def test_guards():
    """Nothing is written outside the outputs (ragged sizes, rows past every tile)."""
    import struct
    from dense_gemm_elementwise_amd import operators as o
    log("[guards]")
    g = gen(2)
    M, N, K = 150, 133, 40
    x, w = rnd(g, M, K), rnd(g, N, K)
    for ld in (N, N + 3, 136):
        buf = torch.full((M * ld + 512,), 3.0, dtype=BF16, device=DEV)
        d = buf[256:256 + M * ld].view(M, ld)
        args = o._LINEAR.pack(M, N, K, x.data_ptr(), K, w.data_ptr(), K, 0, 0, 0, d.data_ptr(), ld, 0, 0, 0, 1)
        s = torch.cuda.current_stream().cuda_stream
        rc, need = o.workspace_bytes("ge_linear", args + struct.pack("@3q", 0, 0, s))
        assert rc == 0
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
        assert o._functions()["ge_linear"](args + struct.pack("@3q", ws.data_ptr(), need, s)) == 0
        torch.cuda.synchronize()
        assert (buf[:256] == 3).all() and (buf[256 + M * ld:] == 3).all()
        assert (d[:, N:] == 3).all()
        assert torch.equal(d[:, :N], ge.linear(x, w))


def test_in_place():
    """D on top of the residual and H' on top of H, through the C entry points, give the same bits."""
    import struct
    from dense_gemm_elementwise_amd import operators as o
    log("[in place]")
    g = gen(15)
    s = torch.cuda.current_stream().cuda_stream
    for M, N, K in ((1, 520, 300), (9, 61, 64), (40, 200, 2304), (300, 264, 72), (300, 263, 72)):
        x, w, r = rnd(g, M, K), rnd(g, N, K, std=K ** -0.5), rnd(g, M, N)
        want = ge.linear(x, w, None, r, act="silu")
        args = o._LINEAR.pack(M, N, K, x.data_ptr(), K, w.data_ptr(), K, 0, r.data_ptr(), N, r.data_ptr(), N, 0, 0, 3, 1)
        rc, need = o.workspace_bytes("ge_linear", args + struct.pack("@3q", 0, 0, s))
        assert rc == 0
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
        assert o._functions()["ge_linear"](args + struct.pack("@3q", ws.data_ptr(), need, s)) == 0
        torch.cuda.synchronize()
        assert torch.equal(r, want)
    for H in (513, 4096):
        h, y = rnd(g, 7, H, t=F32), rnd(g, 7, H)
        ho, xo = ge.norm_residual(h, y)
        x = torch.empty_like(y)
        args = o._NORM.pack(7, H, 1, h.data_ptr(), H, y.data_ptr(), H, 0, 0, 0, 1, 1, 1.0, 1e-5, h.data_ptr(), H,
                            x.data_ptr(), H, 1, 2)
        assert o._functions()["ge_norm_residual"](args + struct.pack("@q", s)) == 0
        torch.cuda.synchronize()
        assert torch.equal(h, ho) and torch.equal(x, xo)


# ---- offsets past 32 bits (operands of more than 4 GiB) ---------------------------
@pytest.mark.parametrize("T", [2, 9, 40])
def test_weights_past_32_bits(T):
    log(f"[past 32 bits] T={T}")
    g = gen(31)
    V, K = 530000, 4104  # 4.35 GB
    x = rnd(g, T, K, std=0.5)
    w = torch.zeros(V, K, dtype=BF16, device=DEV)
    w[-64:] = rnd(g, 64, K, std=2 * K ** -0.5)
    tail = (x.double() @ w[-64:].double().t()).cpu()  # the other logits are 0

    d = ge.linear(x, w)
    assert (d[:, :-64] == 0).all()
    close("D", d[:, -64:], tail, (K + 2) * E24 * (x.double().abs() @ w[-64:].double().abs().t()).cpu())
    dd = torch.zeros_like(d)
    dd[:, -64:] = rnd(g, T, 64)
    dx, dw, db = ge.linear_backward(dd, x, w)
    dd64, x64, w64 = dd[:, -64:].double().cpu(), x.double().cpu(), w[-64:].double().cpu()
    close("dX", dx, dd64 @ w64, 70 * E24 * (dd64.abs() @ w64.abs()))
    close("dW", dw[-64:], dd64.t() @ x64, (T + 2) * E24 * (dd64.abs().t() @ x64.abs()))
    assert (dw[:-64] == 0).all()
    del dw, d, dd

    target = torch.randint(V - 64, V, (T,), generator=g).to(DEV)
    loss, lse = ge.linear_xent(x, w, target)
    want = torch.logsumexp(torch.cat([tail, torch.full((T, 1), math.log(V - 64), dtype=torch.float64)], 1), 1)
    assert (lse.double().cpu() - want).abs().max() < 1e-4
    at = (target - (V - 64)).cpu()
    assert (loss.double().cpu() - (want - tail[torch.arange(T), at])).abs().max() < 1e-4
    dx, dw = ge.linear_xent_backward(torch.ones(T, device=DEV), x, w, target, lse)
    P = torch.exp(tail - want[:, None])
    P[torch.arange(T), at] -= 1
    close("dX", dx, P @ w64, (u(BF16) + 1e-4) * (P.abs() @ w64.abs()))
    close("dW", dw[-64:], P.t() @ x64, (u(BF16) + 1e-4) * (P.abs().t() @ x64.abs()))
    rest = torch.exp(-want) @ x64  # any other row of dW
    for v in (0, V // 2, V - 65):
        close("dW row", dw[v], rest, (u(BF16) + 1e-4) * (torch.exp(-want) @ x64.abs()))


def test_norms_past_32_bits():
    log("[past 32 bits] norms")
    g = gen(32)
    T, H = 270000, 8192  # 4.4 GB a tensor
    h = torch.zeros(T, H, dtype=F16, device=DEV)
    y, dx, dh = torch.zeros_like(h), torch.zeros_like(h), torch.zeros_like(h)
    for t in (h, y, dx, dh):
        t[-3:] = rnd(g, 3, H, t=F16)
    w = rnd(g, H, t=F16, mean=1.0, std=0.1)
    a = ge.norm_residual(h, y, w_post=w, w_pre=w)
    b = ge.norm_residual(h[-3:], y[-3:], w_post=w, w_pre=w)
    for p, q in zip(a, b):
        assert torch.equal(p[-3:], q) and (p[:-3] == 0).all()
    a = ge.norm_residual_backward(dx, dh, h, y, w_post=w, w_pre=w)
    b = ge.norm_residual_backward(dx[-3:], dh[-3:], h[-3:], y[-3:], w_post=w, w_pre=w)
    for p, q in zip(a[:2], b[:2]):
        assert torch.equal(p[-3:], q) and (p[:-3] == 0).all()
    for p, q in zip(a[2:4], b[2:4]):
        assert (p - q).abs().max() <= 1e-5 * q.abs().max()


def test_rows_past_one_grid_axis():
    """2^26 rows of a wave each are 2^32 threads: more than a launch takes along x."""
    log("[many rows] norms")
    g = gen(33)
    T, H = (1 << 26) + 35, 2
    h = torch.zeros(T, H, dtype=F16, device=DEV)
    y = torch.zeros_like(h)
    some = torch.tensor([0, 1, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, 1 << 25, T - 2, T - 1], device=DEV)
    for t in (h, y):
        t[some] = rnd(g, len(some), H, t=F16)
    a = ge.norm_residual(h, y)
    b = ge.norm_residual(h[some], y[some])
    for p, q in zip(a, b):
        assert torch.equal(p[some], q)
        p[some] = 0
        assert (p == 0).all()
    log("[many rows] cross entropy")
    T, K, V = (1 << 26) + 35, 8, 24
    x = torch.zeros(T, K, dtype=F16, device=DEV)
    x[-100:] = rnd(g, 100, K, t=F16)
    w = rnd(g, V, K, t=F16)
    target = torch.zeros(T, dtype=torch.int64, device=DEV)
    target[-100:] = torch.arange(100, device=DEV) % V
    a = ge.linear_xent(x, w, target)
    b = ge.linear_xent(x[-100:], w, target[-100:])
    # (another tile may add the 24 exponentials in another order: some 30 roundings
    # of 2^-24 on values below 64)
    for p, q in zip(a, b):
        assert (p[-100:] - q).abs().max() <= 30 * 64 * 2.0 ** -24
        assert (p[:-100] - math.log(V)).abs().max() <= 30 * 4 * 2.0 ** -24


@pytest.mark.parametrize("t,s", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)],
                         ids=["bf16", "f16", "bf16-f32", "f16-f32"])
@pytest.mark.parametrize("shape", [(9, 4104, 1), (520, 5120, 2), (6, 6143, 3), (300, 6144, 1), (3, 6145, 1),
                                   (7, 4097, 7)], ids=str)
def test_norm_residual_wide(shape, t, s):
    test_norm_residual(shape, t, s)


# ---- long vocabularies, long batches ----------------------------------------------
@pytest.mark.parametrize("T", [1, 9, 17])
def test_xent_few_rows_several_pieces(T):
    """Few rows over a vocabulary longer than a row of P may be: two pieces, the second one short."""
    log(f"[xent few rows, pieces] T={T}")
    g = gen(34 + T)
    V, K = 2100011, 8
    x, w = rnd(g, T, K), rnd(g, V, K, std=0.7).abs()  # (weights of one sign: a piece left out of dX would show)
    target = torch.randint(0, V, (T,), generator=g)
    target[0] = V - 1
    if T > 2:
        target[1], target[2] = 0, IGNORE
    target, dloss = target.to(DEV), torch.linspace(0.25, 1.0, T, device=DEV)
    loss, lse = ge.linear_xent(x, w, target)
    dx, dw = ge.linear_xent_backward(dloss, x, w, target, lse)
    x64, w64 = x.double(), w.double()
    logits = x64 @ w64.t()
    be = (K + 2) * E24 * (x64.abs() @ w64.abs().t())
    want = torch.logsumexp(logits, 1)
    # of lse: a logit's error, and under 400 joins of partial sums of 3 roundings each
    bl = be.amax(1) + 1200 * E24 + want.abs() * 2.0 ** -23
    close("lse", lse, want, bl)
    live = target != IGNORE
    at = torch.where(live, target, 0)[:, None]
    scale = torch.where(live, dloss.double(), 0.0)[:, None]
    p = torch.exp(logits - want[:, None]) * scale
    ep = p * (be + bl[:, None] + 2e-6 * (1 + (logits - want[:, None]).abs()))
    P = p.scatter_add_(1, at, -scale)
    ep = ep + (u(BF16) + 4 * E24) * P.abs()
    # fp32 sums over V entries: their roundings have either sign, 8 standard deviations
    close("dX", dx, P @ w64, ep @ w64 + 8 * math.sqrt(V) * E24 * (P.abs() @ w64))
    close("dW", dw, P.t() @ x64, ep.t() @ x64.abs() + (T + 9) * E24 * (P.abs().t() @ x64.abs()))


def test_empty_batches_one_gradient():
    """Each gradient of an empty batch alone: an empty dX, zeros for the rest."""
    log("[empty, one gradient]")
    x, w = torch.empty(0, 64, dtype=BF16, device=DEV), torch.ones(48, 64, dtype=BF16, device=DEV)
    d, t = torch.empty(0, 48, dtype=BF16, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    f = torch.empty(0, device=DEV)
    for act in ("identity", "gelu"):
        for need in ((1, 0, 0), (0, 1, 0), (0, 0, 1)):
            got = ge.linear_backward(d, x, w, d, act=act, need_dx=need[0], need_dw=need[1], need_dbias=need[2])
            for o, n, shape in zip(got, need, ((0, 64), (48, 64), (48,))):
                assert (o is not None and o.shape == shape and (o == 0).all()) if n else o is None
    dx, dw = ge.linear_xent_backward(f, x, w, t, f, need_dw=False)
    assert dx.shape == (0, 64) and dw is None
    dx, dw = ge.linear_xent_backward(f, x, w, t, f, need_dx=False)
    assert dx is None and (dw == 0).all()


LONGEST = 2 ** 31 - 257  # the longest vocabulary and batch that the calls take


def longest_vocabulary(T, V=LONGEST, std=8.0, joins=1000):
    """Loss and lse of T rows over V columns of K = 1; all but 64 logits are 0."""
    g = gen(35 + T)
    x = rnd(g, T, 1)
    w = torch.zeros(V, 1, dtype=BF16, device=DEV)
    some = torch.cat([torch.arange(32), torch.arange(V - 32, V)]).to(DEV)
    w[some] = rnd(g, 64, 1, std=std)
    at = (torch.arange(T, device=DEV) * 7 + 31) % 64  # targets from both ends
    target = some[at]
    loss, lse = ge.linear_xent(x, w, target)
    logits = x.double() @ w[some].double().t()
    rest = torch.full((T, 1), math.log(V - 64), dtype=torch.float64, device=DEV)
    want = torch.logsumexp(torch.cat([logits, rest], 1), 1)
    # sums of ones are exact up to 2^24 (a wave's 2^18 rows); every join of partial sums
    # leaves 3 roundings
    b = 3 * joins * E24 + want.abs() * 2.0 ** -22
    close("lse", lse, want, b)
    close("loss", loss, want - logits.gather(1, at[:, None])[:, 0], b + 2 * E24 * logits.abs().amax(1))


@pytest.mark.parametrize("T", [1, 2])
def test_xent_longest_vocabulary_row_dot(T):
    log(f"[longest vocabulary] T={T}")
    longest_vocabulary(T)


@pytest.mark.parametrize("T,V", [(3, LONGEST), (16, LONGEST), (3, (1 << 30) + 64), (3, (1 << 27) + 1)])
def test_xent_longest_vocabulary_skinny(T, V):
    """Blocks of 64 columns past one grid axis (2^21 of them) and past 2^32 threads (2^24)."""
    log(f"[longest vocabulary] T={T} V={V}")
    # 256 threads join the V / 64 partial sums of a row
    longest_vocabulary(T, V, std=1.0, joins=1000 + V // 2 ** 14)


def test_linear_backward_longest_batch_dbias():
    """The last strip of rows ends past 2^31 before it is cut to the batch."""
    log("[longest batch] dbias")
    g = gen(36)
    M, N, K = LONGEST, 8, 1
    dd = torch.zeros(M, N, dtype=BF16, device=DEV)  # 34 GB
    some = torch.tensor([0, 1, 1 << 30, M - (1 << 20), M - 4096, M - 2, M - 1], device=DEV)
    dd[some] = rnd(g, len(some), N)
    x = torch.zeros(M, K, dtype=BF16, device=DEV)
    w = torch.zeros(N, K, dtype=BF16, device=DEV)
    _, _, db = ge.linear_backward(dd, x, w, need_dx=False, need_dw=False)
    v = dd[some].double()
    close("dbias", db, v.sum(0), len(some) * E24 * v.abs().sum(0))  # (zeros add no rounding)


def test_norm_gradient_longest_batch_of_gates():
    """A gate row for each of 2^31 - 1 rows: the last workgroup's share ends past 2^31 before it is cut."""
    log("[longest batch] norm gates")
    g = gen(37)
    T, H = 2 ** 31 - 1, 1
    some = torch.tensor([0, 1, 1 << 21, 1 << 30, T - (1 << 21), T - 12345, T - 2, T - 1], device=DEV)
    dx, dh, h, y, gate = (torch.zeros(T, H, dtype=F16, device=DEV) for _ in range(5))
    for t in (dx, dh, h, y, gate):
        t[some] = rnd(g, len(some), H, t=F16)
    kw = dict(scale=0.7, post="none", pre="rms")
    a = ge.norm_residual_backward(dx, dh, h, y, gate=gate, **kw)
    b = ge.norm_residual_backward(dx[some], dh[some], h[some], y[some], gate=gate[some], **kw)
    for i in (0, 1, 4):
        assert torch.equal(a[i][some], b[i]), i
        a[i][some] = 0
        assert a[i].count_nonzero() == 0, i


def test_linear_backward_longest_batch_dw():
    """The contraction's last part ends past 2^31 before it is cut to the batch."""
    log("[longest batch] dW")
    g = gen(38)
    M, N, K = LONGEST, 8, 8
    some = torch.tensor([0, 1, 1 << 30, M - (1 << 20), M - 4096, M - 2, M - 1], device=DEV)
    dd, x = (torch.zeros(M, 8, dtype=BF16, device=DEV) for _ in range(2))  # 34 GB each
    dd[some], x[some] = rnd(g, len(some), N), rnd(g, len(some), K)
    _, dw, _ = ge.linear_backward(dd, x, torch.zeros(N, K, dtype=BF16, device=DEV), need_dx=False, need_dbias=False)
    d64, x64 = dd[some].double(), x[some].double()
    close("dW", dw, d64.t() @ x64, len(some) * E24 * (d64.abs().t() @ x64.abs()))  # (zeros add no rounding)


def test_linear_backward_longest_batch():
    """All three gradients of 2^31 - 257 rows: the two products together have more workgroups than
    one launch takes."""
    log("[longest batch] linear_backward")
    g = gen(38)
    M, N, K = LONGEST, 8, 8
    some = torch.tensor([0, 1, 1 << 30, M - (1 << 20), M - 4096, M - 2, M - 1], device=DEV)
    dd, x = (torch.zeros(M, 8, dtype=BF16, device=DEV) for _ in range(2))  # 34 GB each
    dd[some], x[some] = rnd(g, len(some), N), rnd(g, len(some), K)
    w = rnd(g, N, K)
    dx, dw, db = ge.linear_backward(dd, x, w)
    d64, x64, w64 = dd[some].double(), x[some].double(), w.double()
    n = len(some)  # (zeros add no rounding)
    close("dX", dx[some], d64 @ w64, (N + 2) * E24 * (d64.abs() @ w64.abs()))
    close("dW", dw, d64.t() @ x64, n * E24 * (d64.abs().t() @ x64.abs()))
    close("dbias", db, d64.sum(0), n * E24 * d64.abs().sum(0))
    dx[some] = 0
    for part in dx.split(1 << 28):
        assert part.count_nonzero() == 0


@pytest.mark.parametrize("T", [17, 256])
def test_xent_longest_vocabulary_tiles(T):
    """2^24 tiles of 128 columns, and 256 rows, where only the larger tile is few enough workgroups."""
    log(f"[longest vocabulary] T={T}")
    # 256 threads join the V / 128 or V / 256 partial sums of a row
    longest_vocabulary(T, std=1.0, joins=1000 + LONGEST // 2 ** 15)


def test_forward_mode_tangents():
    """Every call refuses an input with a forward-mode tangent, and takes its primal."""
    from torch.autograd import forward_ad
    x, w = torch.ones(4, 8, dtype=F16, device=DEV), torch.ones(8, 8, dtype=F16, device=DEV)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    f = torch.ones(4, device=DEV)
    calls = [lambda v: ge.linear(v, w), lambda v: ge.linear(x, w, None, v), lambda v: ge.linear_backward(v, x, w),
             lambda v: ge.linear_xent(v, w, t), lambda v: ge.linear_xent_backward(f, v, w, t, f),
             lambda v: ge.norm_residual(x, v), lambda v: ge.norm_residual_backward(x, v, x, x)]
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        for call in calls:
            with pytest.raises(ValueError, match="tangent"):
                call(dual)
            a, b = call(forward_ad.unpack_dual(dual).primal), call(x)
            for p, q in zip(a, b) if isinstance(a, tuple) else ((a, b),):
                assert (p is None and q is None) or torch.equal(p, q)


@pytest.mark.parametrize("t,s", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)],
                         ids=["bf16", "f16", "bf16-f32", "f16-f32"])
@pytest.mark.parametrize("H", [3, 40, 513, 1000, 2052, 4101, 5000, 6148, 8191])
def test_norm_gradient_large_means(H, t, s):
    """Rows whose mean is 20 deviations, of H', of Y and of both: the gradient then takes its sums
    about the mean in a second pass."""
    log(f"[norm gradient, means] {H} {t} {s}")
    T, G, eps = 6, 2, 1e-5
    for n, (mh, my, post, pre) in enumerate(((40.0, 0.25, "layer", "layer"), (-0.5, -60.0, "layer", "layer"),
                                             (40.0, -60.0, "layer", "layer"), (-40.0, 60.0, "rms", "layer"),
                                             (40.0, 60.0, "layer", "rms"), (40.0, 60.0, "none", "layer"))):
        g = gen(40 + H + n)
        h, y = rnd(g, T, H, std=2.0, mean=mh, t=s), rnd(g, T, H, std=3.0, mean=my, t=t)
        h[1], y[2] = h[1] - mh, y[2] - my  # a row without one between the others
        gate, wi = rnd(g, G, H, std=0.3, mean=0.5, t=t), rnd(g, H, std=0.1, mean=1.0, t=t)
        wo = rnd(g, H, std=0.1, mean=1.0, t=t) if post != "none" else None
        dx, dho = rnd(g, T, H, t=t), rnd(g, T, H, t=s)
        got = ge.norm_residual_backward(dx, dho, h, y, w_post=wo, w_pre=wi, gate=gate, scale=0.7, post=post, pre=pre,
                                        eps=eps)
        one = torch.ones(H, dtype=torch.float64)
        h64, y64, dx64, dho64 = (v.double().cpu() for v in (h, y, dx, dho))
        g64, wi64 = gate.double().cpu().repeat_interleave(T // G, 0), wi.double().cpu()
        wo64 = wo.double().cpu() if wo is not None else one

        def normed(v, kind):
            """(rows, reciprocal scale, error of the rows): the mean is off by at most 24 roundings of the
            largest element (12 terms a thread, 10 steps across the workgroup), the scale by 4e-6."""
            if kind == "none":
                return v, None, v.abs() * E24
            vn, r, _ = norm64(v, kind, eps)
            return vn, r, 4e-6 * vn.abs() + r * v.abs().amax(1, keepdim=True) * 24 * E24

        hn, rh, ehn = normed(h64, pre)
        dn = dx64 * wi64
        c_h = (dn * hn).mean(1, keepdim=True)
        m_d = dn.mean(1, keepdim=True) if pre == "layer" else 0.0
        dh = dho64 + (dn - hn * c_h - m_d) * rh
        mag = dn.abs() + hn.abs() * (dn * hn).abs().mean(1, keepdim=True) + dn.abs().mean(1, keepdim=True)
        edh = rh * (1e-5 * mag + ehn * c_h.abs() + hn.abs() * (dn.abs() * ehn).mean(1, keepdim=True)) \
            + 4 * E24 * dh.abs() + E24 * dho64.abs()
        close("dH", got[0], dh, edh)
        yn, ry, eyn = normed(y64, post)
        dyw = 0.7 * g64 * dh
        edyw = 0.7 * g64.abs() * edh + 3 * E24 * dyw.abs()
        d, ed = dyw * wo64, edyw * wo64.abs()
        dy, edy = dyw, edyw
        if post != "none":
            c_y = (d * yn).mean(1, keepdim=True)
            m_y = d.mean(1, keepdim=True) if post == "layer" else 0.0
            dy = (d - yn * c_y - m_y) * ry
            magy = d.abs() + yn.abs() * (d * yn).abs().mean(1, keepdim=True) + d.abs().mean(1, keepdim=True)
            edy = ry * (1e-5 * magy + ed + ed.mean(1, keepdim=True) + eyn * c_y.abs()
                        + yn.abs() * (ed * yn.abs() + d.abs() * eyn).mean(1, keepdim=True))
            close("dw_post", got[2], (dyw * yn).sum(0), (edyw * yn.abs() + dyw.abs() * eyn).sum(0)
                  + (T + 4) * E24 * (dyw * yn).abs().sum(0))
        close("dY", got[1], dy, edy)
        close("dw_pre", got[3], (dx64 * hn).sum(0), (dx64.abs() * ehn).sum(0) + (T + 4) * E24 * (dx64 * hn).abs().sum(0))
        v = 0.7 * yn * wo64 * dh
        e = 0.7 * wo64.abs() * (yn.abs() * edh + eyn * dh.abs()) + 4 * E24 * v.abs()
        close("dgate", got[4], v.view(G, T // G, H).sum(1),
              e.view(G, T // G, H).sum(1) + (T + 4) * E24 * v.abs().view(G, T // G, H).sum(1))


@pytest.mark.parametrize("t", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("M", [1, 3, 20])
def test_activation_everywhere(M, act, t):
    """act(z) at every finite z, through the bias of a product of zeros: each of the three paths."""
    log(f"[act] M={M} {act} {t}")
    z = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(t)
    z = z[z.isfinite()]
    x, w = torch.zeros(M, 8, dtype=t, device=DEV), torch.zeros(len(z), 8, dtype=t, device=DEV)
    d, kept = ge.linear(x, w, z.to(DEV), act=act, save_z=True)
    assert torch.equal(kept, z.to(DEV).expand(M, -1))
    z64 = z.double()
    want, a = act64(z64, act), z64.abs()
    if act == "gelu":
        # |z| Q(|z|) by a fit to 2e-6, with four roundings and an exponent z^2 / 4 that is off by 3
        # half units in fp32, twice
        bound = (4e-6 + 1.5 * E24 * a * a) * 0.5 * a * torch.erfc(a * 0.5 ** 0.5) + 2 * E24 * want.abs()
    else:
        # e^-|z| from an exponent |z| / 2 that is off by 2 half units, twice; exponential and
        # reciprocal to a unit, four roundings
        bound = (1e-6 + 2 * E24 * a) * want.abs()
    close(act, d, want.expand(M, -1), bound.nan_to_num(nan=0.0).expand(M, -1))


@pytest.mark.parametrize("t", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("T", [12, 40])
def test_xent_gradient_unequal_rows(T, t):
    """Incoming gradients from 2^12 down to 2^-12 of either sign in one batch: P is held with one
    factor for all rows."""
    log(f"[xent unequal rows] T={T} {t}")
    g = gen(41)
    V, K = 1003, 64
    x, w = rnd(g, T, K, t=t), rnd(g, V, K, std=2 * K ** -0.5, t=t)
    target = torch.randint(0, V, (T,), generator=g).to(DEV)
    dloss = (torch.tensor([(-1.0) ** i * 2.0 ** (12 - 24 * i / (T - 1)) for i in range(T)])).to(DEV)
    logits, be, lse, _, _, at = xent_ref(x, w, target)
    _, got_lse = ge.linear_xent(x, w, target)
    dx, dw = ge.linear_xent_backward(dloss, x, w, target, got_lse)
    # of lse: as in test_linear_xent; of P: its logit's, lse's and the exponential's errors, the
    # rounding to the element type, and in fp16 half the smallest subnormal at 2^14 over the largest
    bl = be.amax(1) + 1e-5 + lse.abs() * 2.0 ** -23
    scale = dloss.double().cpu()[:, None]
    p = torch.exp(logits - lse[:, None])
    P = (p - torch.zeros_like(p).scatter_(1, at, 1.0)) * scale
    eP = p * scale.abs() * (be + bl[:, None] + 2e-6 * (1 + (logits - lse[:, None]).abs())) \
        + (u(t) + 4 * E24) * P.abs() + (2.0 ** -39 * scale.abs().max() if t == F16 else 0.0)
    x64, w64 = x.double().cpu(), w.double().cpu()
    close("dX", dx, P @ w64, eP @ w64.abs() + (V + 9) * E24 * (P.abs() @ w64.abs()))
    close("dW", dw, P.t() @ x64, eP.t() @ x64.abs() + (T + 9) * E24 * (P.abs().t() @ x64.abs()))


@pytest.mark.parametrize("t", [BF16, F16], ids=["bf16", "f16"])
def test_relu_gradient_masks(t):
    """What arrives where relu is 0 does not pass, an infinity or a NaN neither; a NaN z, which the
    forward keeps, does not count as masked."""
    log(f"[relu masks] {t}")
    g = gen(42)
    M, N, K = 40, 24, 16
    x, w, dd = rnd(g, M, K, t=t), rnd(g, N, K, t=t), rnd(g, M, N, t=t)
    z = rnd(g, M, N, t=t)
    z[3, 5], z[4, 6], z[5, 7] = -1.0, 0.0, -0.5
    want = ge.linear_backward(torch.where(z > 0, dd, 0.0), x, w)  # the identity's
    dd[3, 5], dd[4, 6], dd[5, 7] = float("inf"), float("nan"), float("-inf")
    got = ge.linear_backward(dd, x, w, z, act="relu")
    for p, q in zip(got, want):
        assert q.isfinite().all() and torch.equal(p, q)
    # the same rows through autograd's relu
    z32 = z.float().requires_grad_()
    dz, = torch.autograd.grad(torch.relu(z32), z32, dd.float())
    assert torch.equal(dz, torch.where(z > 0, dd, 0.0).float())
    z[7, 2] = float("nan")
    dx, dw, db = ge.linear_backward(torch.where(dd.isfinite(), dd, 0.0), x, w, z, act="relu")
    want = ge.linear_backward(torch.where((z > 0) | z.isnan(), dd, 0.0), x, w)
    for p, q in zip((dx, dw, db), want):
        assert torch.equal(p, q)


@pytest.mark.parametrize("t", [BF16, F16], ids=["bf16", "f16"])
def test_two_rows(t):
    """Two rows of X: fp16 in multiply-adds, bf16 in one MFMA block."""
    for shape in ((2, 64, 64), (2, 1003, 999), (2, 520, 300), (2, 5, 3), (2, 1, 1), (2, 4104, 2056)):
        test_linear(shape, t)
    for shape in ((2, 1000, 64), (2, 257, 33), (2, 33000, 520), (2, 1, 1)):
        test_linear_xent(shape, t)


def test_xent_longest_vocabulary_two_rows_f16():
    """The second row's loop past 2^31 - 8192 columns in the type that still takes it."""
    log("[longest vocabulary] two rows, f16")
    g = gen(43)
    V = LONGEST
    x, w = rnd(g, 2, 1, t=F16), torch.zeros(V, 1, dtype=F16, device=DEV)
    w[-32:] = rnd(g, 32, 1, t=F16)
    target = torch.tensor([V - 1, 5], device=DEV)
    loss, lse = ge.linear_xent(x, w, target)
    logits = x.double() @ w[-32:].double().t()
    rest = torch.full((2, 1), math.log(V - 32), dtype=torch.float64, device=DEV)
    want = torch.logsumexp(torch.cat([logits, rest], 1), 1)
    b = 3000 * E24 + want.abs() * 2.0 ** -22  # as in longest_vocabulary
    close("lse", lse, want, b)
    close("loss", loss, want - torch.stack([logits[0, -1], 0 * logits[1, 0]]), b + 2 * E24 * logits.abs().max())
