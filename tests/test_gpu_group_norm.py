"""Group norm with an activation, channels last: forward, codes and gradients
against the definitions in 64 bits.

Tolerances, with u = 2^-24 (half a step of fp32, relative):
  * a group's mean is a sum of fp32 values in chains of at most some hundred
    additions whose roundings are independent: 64 u (|mean| + max|x|) covers it;
    the deviations and rstd likewise carry 64 u relative;
  * z = (x - mean) a + b then is off by 64 u (|a| (|mean| + max|x|) + |z| + |b|),
    the activations (slope below 1.13) add the fast exponential's and quotient's
    error, (|z| + 4) 2^-22 relative;
  * the output's rounding: half a step of its type, eps / 2 relative.
"""
import math

import pytest
import torch

import post_quantized_linear_b200 as pq

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def half_step(t):
    return torch.finfo(t).eps / 2


def act64(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z


def reference(x, G, gamma, beta, eps, act):
    """(y, bound on |y - fp32 evaluation|, mean, rstd) in float64, x [B, S, C]."""
    B, S, C = x.shape
    v = x.double().view(B, S, G, C // G)
    mean = v.mean((1, 3), keepdim=True)
    var = ((v - mean) ** 2).mean((1, 3), keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    ga = torch.ones(C, dtype=torch.float64, device=x.device) if gamma is None else gamma.double()
    be = torch.zeros(C, dtype=torch.float64, device=x.device) if beta is None else beta.double()
    z = ((v - mean) * rstd).view(B, S, C) * ga + be
    a = (rstd.expand(B, 1, G, C // G).reshape(B, 1, C) * ga).abs()
    far = (mean.abs() + v.abs().amax((1, 3), keepdim=True)).expand(B, 1, G, C // G).reshape(B, 1, C)
    bound = 1.13 * 64 * U * (a * far + z.abs() + be.abs())
    y = act64(z, act)
    if act != "none":
        bound = bound + (z.abs() + 4) * 2.0 ** -22 * y.abs() + U * z.abs()
    return y, bound, mean.view(B, G), rstd.view(B, G)


def make(B, S, C, dtype, seed=0, wide=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, S, C, generator=g, device="cuda") * (0.5 + torch.rand(B, 1, C, generator=g, device="cuda"))
    x = x + torch.randn(B, 1, C, generator=g, device="cuda") * (30.0 if wide else 0.7)
    gamma = 1 + 0.2 * torch.randn(C, generator=g, device="cuda")
    beta = 0.2 * torch.randn(C, generator=g, device="cuda")
    return x.to(dtype), gamma, beta, g


def check(y, ref, bound):
    tol = bound + half_step(y.dtype) * (ref.abs() + bound) + 1e-38
    err = (y.double() - ref).abs()
    assert torch.isfinite(y.float()).all()
    assert (err <= tol).all(), f"worst {(err / tol).max().item():.2f} of the tolerance"


SHAPES = [
    # B, S, C, G: one position; one channel a group; odd maps; groups that straddle
    # 16-byte vectors; one group; wide groups; maps of the two-pass form
    (1, 1, 8, 1), (2, 1, 64, 8), (3, 7, 64, 64), (2, 64, 1280, 32), (3, 1023, 320, 32), (2, 257, 72, 24),
    (1, 100, 4096, 1), (5, 33, 1152, 128), (1, 4097, 960, 32), (1, 70001, 64, 8), (2, 66049, 40, 4),
    (70, 16, 16, 2), (1, 3001, 2304, 9),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_matches_definition(shape, dtype):
    B, S, C, G = shape
    act = ("none", "silu", "gelu")[(S + C) % 3]
    x, gamma, beta, _ = make(B, S, C, dtype, seed=S)
    if C // G * x.element_size() > 8192:                   # a group wider than the kernels' blocks
        with pytest.raises(pq.SegQuantError, match="SQ_ERR_UNSUPPORTED"):
            pq.group_norm_act(x, G, gamma, beta)
        return
    for out_dtype in (BF, F32):
        y, stats = pq.group_norm_act(x, G, gamma, beta, eps=1e-5, act=act, out_dtype=out_dtype, return_stats=True)
        ref, bound, mean, rstd = reference(x, G, gamma, beta, 1e-5, act)
        check(y, ref, bound)
        far = mean.abs() + x.double().abs().amax()
        assert ((stats[..., 0] - mean).abs() <= 64 * U * far).all()
        assert ((stats[..., 1] / rstd - 1).abs() <= 64 * U * (1 + far * rstd)).all()
    again = pq.group_norm_act(x, G, gamma, beta, eps=1e-5, act=act, out_dtype=out_dtype)
    assert torch.equal(y, again)
    assert pq.stream_status() == 0


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_forward_defaults_wide_means_and_in_place(act):
    x, gamma, beta, _ = make(2, 129, 320, F32, seed=5, wide=True)
    ref, bound, _, _ = reference(x, 32, None, None, 1e-5, act)
    check(pq.group_norm_act(x, 32, act=act), ref, bound)
    ref, bound, _, _ = reference(x, 32, gamma, None, 0.25, act)
    check(pq.group_norm_act(x, 32, gamma, eps=0.25, act=act), ref, bound)
    out = x.clone()
    assert pq.group_norm_act(out, 32, gamma, eps=0.25, act=act, out=out) is out
    check(out, ref, bound)
    big = torch.cat([x, x.repeat(1, 600, 1)], 1)          # the two-pass form, in place
    ref, bound, _, _ = reference(big, 32, gamma, beta, 1e-5, act)
    pq.group_norm_act(big, 32, gamma, beta, act=act, out=big)
    check(big, ref, bound)


def test_forward_strided_maps():
    """Maps inside larger ones: other position and image strides, rows around them untouched."""
    x, gamma, beta, _ = make(4, 50, 96, BF, seed=9)
    xv = x[1:, 3:40, 16:80]                                # C = 64 of 96, images 50 positions apart
    buf = torch.full((3, 39, 72), 7.0, device="cuda")
    out = buf[:, 1:38, 4:68]
    pq.group_norm_act(xv, 8, gamma[:64].contiguous(), beta[:64].contiguous(), act="silu", out=out)
    ref, bound, _, _ = reference(xv.contiguous(), 8, gamma[:64], beta[:64], 1e-5, "silu")
    check(out, ref, bound)
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[:, 1:38, 4:68] = False
    assert (buf[keep] == 7).all()
    # an NCHW tensor in the channels_last format, and images in reverse order of memory are not needed:
    t = torch.randn(2, 64, 9, 11, device="cuda").to(memory_format=torch.channels_last)
    m = t.permute(0, 2, 3, 1).flatten(1, 2)
    ref, bound, _, _ = reference(m, 8, None, None, 1e-5, "gelu")
    check(pq.group_norm_act(m, 8, act="gelu"), ref, bound)


def test_constant_groups_outliers_and_non_finite_values():
    x, gamma, beta, _ = make(1, 300, 64, F32, seed=3)
    x[:, :, 0:8] = 3.0                                     # variance zero: z = beta
    x[:, 0, 8:16] = 1e4                                    # the first position far off the rest
    ref, bound, _, _ = reference(x, 8, gamma, beta, 1e-5, "none")
    y = pq.group_norm_act(x, 8, gamma, beta)
    check(y, ref, bound)
    clean = y.clone()
    x[0, 5, 20] = float("nan")
    x[0, 7, 30] = float("inf")
    y = pq.group_norm_act(x, 8, gamma, beta)
    assert torch.isnan(y[:, :, 16:32]).all()
    assert torch.equal(y[:, :, :16], clean[:, :, :16]) and torch.equal(y[:, :, 32:], clean[:, :, 32:])


@pytest.mark.parametrize("shape", [(2, 64, 1152, 32), (1, 1, 16, 2), (3, 37, 2304, 32), (1, 70001, 64, 8)], ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_codes_equal_the_quantizer_of_the_norm(shape, dtype, act):
    B, S, C, G = shape
    x, gamma, beta, _ = make(B, S, C, dtype, seed=S + 1)
    kseg = (0, C) if C < 256 else (0, 256, C)
    y16 = pq.group_norm_act(x, G, gamma, beta, act=act, out_dtype=BF).view(B * S, C)
    sp, sn = pq.calibrate(y16, kseg)
    want = pq.quantize_activations(y16, kseg, sp, sn)
    qp, qn, y = pq.quantize_activations_norm(x, G, gamma, beta, kseg, sp, sn, act=act, return_y=True)
    assert torch.equal(qp, want[0]) and torch.equal(qn, want[1]) and torch.equal(y, y16)
    wide = torch.full((2, B * S, C + 32), 99, dtype=torch.int8, device="cuda")
    pq.quantize_activations_norm(x, G, gamma, beta, kseg, sp, sn, act=act, out=(wide[0, :, :C], wide[1, :, :C]))
    for w, t in zip(wide, want):
        assert torch.equal(w[:, :C], t) and (w[:, C:] == 99).all()
    assert pq.stream_status() == 0


@pytest.mark.parametrize("S", [37, 70001])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_codes_of_non_finite_values_equal_the_quantizer(dtype, S):
    """Groups with NaN, values that overflow to infinities, and segments whose scales are zero:
    the fused codes are those that the quantizer gives for the same bf16 values."""
    x, gamma, beta, _ = make(1, S, 256, dtype, seed=S)
    x[0, 5, 20], x[0, S - 1, 130] = float("nan"), float("inf")
    gamma[64:80] = 3e38
    gamma[192:208] = -3e38
    y16 = pq.group_norm_act(x, 32, gamma, beta, out_dtype=BF).view(S, 256)
    assert torch.isnan(y16).any() and (y16 == float("inf")).any() and (y16 == float("-inf")).any()
    kseg = (0, 128, 256)
    for sp, sn in (((0.05, 0.04), (0.03, 0.06)), ((0.0, 0.04), (0.03, 0.0)), ((0.05, 0.0), (0.0, 0.06)),
                   ((0.0, 0.0), (0.0, 0.0))):
        sp, sn = torch.tensor(sp, device="cuda"), torch.tensor(sn, device="cuda")
        want = pq.quantize_activations(y16, kseg, sp, sn)
        got = pq.quantize_activations_norm(x, 32, gamma, beta, kseg, sp, sn)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ gradients
def slope64(z, act):
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def reference_grads(dy, x, stats, gamma, beta, act):
    """((dx, dgamma, dbeta), their bounds) in float64.  The forward's mean and rstd are
    inputs; xhat is off by 4 u (|x| + |mean|) rstd, dz by the slope's change over that
    (second derivatives below 1.2) and the fast exponential's (|z| + 4) 2^-22 relative to
    1.13 |dy|; sums add 64 u of their absolute terms."""
    B, S, C = x.shape
    G = stats.shape[1]
    w = C // G
    mean = stats[..., 0].double().repeat_interleave(w, 1)[:, None]
    rstd = stats[..., 1].double().repeat_interleave(w, 1)[:, None]
    hat = (x.double() - mean) * rstd
    e_hat = 4 * U * (x.double().abs() + mean.abs()) * rstd
    z = hat * gamma.double() + beta.double()
    dz = dy.double() * slope64(z, act)
    e_dz = dy.double().abs() * (1.2 * (e_hat * gamma.double().abs() + 4 * U * z.abs())
                                + 1.13 * (z.abs() + 4) * 2.0 ** -22) * (act != "none")
    group = lambda t: t.view(B, S, G, w).mean((1, 3)).repeat_interleave(w, 1)[:, None]  # noqa: E731
    dbeta, dgamma = dz.sum((0, 1)), (dz * hat).sum((0, 1))
    e_t = e_dz * hat.abs() + dz.abs() * e_hat
    b_dbeta = (e_dz + 64 * U * dz.abs()).sum((0, 1))
    b_dgamma = (e_t + 64 * U * (dz * hat).abs()).sum((0, 1))
    ga = gamma.double().abs()
    dh = dz * gamma.double()
    m1, m2 = group(dh), group(dh * hat)
    e1, e2 = group((e_dz + 64 * U * dz.abs()) * ga), group((e_t + 64 * U * (dz * hat).abs()) * ga)
    dx = rstd * (dh - m1 - hat * m2)
    b_dx = rstd * (e_dz * ga + e1 + hat.abs() * e2 + e_hat * m2.abs()
                   + 8 * U * (dh.abs() + m1.abs() + (hat * m2).abs()))
    return (dx, dgamma, dbeta), (b_dx, b_dgamma, b_dbeta)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients_match_the_formula(shape, dtype):
    B, S, C, G = shape
    act = ("silu", "none", "gelu")[(S + C) % 3]
    x, gamma, beta, g = make(B, S, C, dtype, seed=S + 2)
    dy = torch.randn(B, S, C, generator=g, device="cuda").to(dtype)
    if C // G * x.element_size() > 8192:
        with pytest.raises(pq.SegQuantError, match="SQ_ERR_UNSUPPORTED"):
            pq.group_norm_act_backward(dy, x, torch.zeros(B, G, 2, device="cuda"), gamma, beta)
        return
    _, stats = pq.group_norm_act(x, G, gamma, beta, act=act, return_stats=True)
    got = pq.group_norm_act_backward(dy, x, stats, gamma, beta, act=act)
    want, bounds = reference_grads(dy, x, stats, gamma, beta, act)
    for y, r, b in zip(got, want, bounds):
        check(y, r, b)
    again = pq.group_norm_act_backward(dy, x, stats, gamma, beta, act=act)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert pq.stream_status() == 0


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_gradients_match_differences_and_autograd(act):
    """Central differences of the 64-bit definition along random directions: with steps of
    1e-4 they are off by about 1e-8 of the terms; the kernel's fp32 gradients by 1e-5."""
    x, gamma, beta, g = make(2, 21, 48, F32, seed=11)
    dy = torch.randn(2, 21, 48, generator=g, device="cuda")
    _, stats = pq.group_norm_act(x, 6, gamma, beta, act=act, return_stats=True)
    grads = pq.group_norm_act_backward(dy, x, stats, gamma, beta, act=act)

    def f(x, gamma, beta):
        return (reference(x, 6, gamma, beta, 1e-5, act)[0] * dy.double()).sum()

    at = [x.double(), gamma.double(), beta.double()]
    for i in range(3):
        v = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        lo, hi = list(at), list(at)
        lo[i], hi[i] = at[i] - 1e-4 * v, at[i] + 1e-4 * v
        want = ((f(*hi) - f(*lo)) / 2e-4).item()
        got = (grads[i].double() * v).sum().item()
        terms = (grads[i].double() * v).abs().sum().item()
        assert abs(got - want) <= 1e-5 * terms
    leaves = [t.clone().requires_grad_() for t in at]
    auto = torch.autograd.grad(f(*leaves), leaves)
    for a, b in zip(grads, auto):
        assert ((a.double() - b).abs() <= 1e-5 * (1 + b.abs().amax())).all()


def test_gradients_strided_in_place_and_defaults():
    x, gamma, beta, g = make(3, 45, 96, BF, seed=21)
    xv, dyv = x[:, :, 32:96], torch.randn(3, 45, 128, generator=g, device="cuda").to(BF)[:, :, 8:72]
    _, stats = pq.group_norm_act(xv, 8, act="silu", return_stats=True)
    one, zero = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    want, bounds = reference_grads(dyv, xv, stats, one, zero, "silu")
    got = pq.group_norm_act_backward(dyv, xv, stats, act="silu")
    for y, r, b in zip(got, want, bounds):
        check(y, r, b)
    dx, _, _ = pq.group_norm_act_backward(dyv, xv, stats, act="silu", dx=dyv)
    assert dx is dyv and torch.equal(dyv, got[0])


# --------------------------------------------------- the activations themselves
# A map of zeros has z = beta exactly, and with mean 0, rstd 1 and dy = 1 at a single
# position dbeta is the slope at beta: one value of z a channel.
def activation_of(z, act, out_dtype=F32):
    C = z.numel()
    return pq.group_norm_act(torch.zeros(1, 1, C, device="cuda"), C // 8, None, z, act=act, out_dtype=out_dtype).view(C)


def slope_of(z, act):
    C = z.numel()
    stats = torch.tensor([0.0, 1.0], device="cuda").expand(1, C // 8, 2).contiguous()
    zero, one = torch.zeros(1, 1, C, device="cuda"), torch.ones(1, 1, C, device="cuda")
    return pq.group_norm_act_backward(one, zero, stats, None, z, act=act)[2]


def z_values(kind):
    g = torch.Generator(device="cuda").manual_seed(7)
    if kind == "normal":
        return torch.randn(65536, generator=g, device="cuda")
    if kind == "wide":
        return torch.linspace(-13, 13, 65536, device="cuda")
    return torch.linspace(-86, 86, 65536, device="cuda")


@pytest.mark.parametrize("act,kind", [("silu", "normal"), ("silu", "wide"), ("silu", "far"), ("gelu", "normal"),
                                      ("gelu", "wide")])     # beyond |z| = 13 GELU's tail leaves the fp32 range
def test_activations_keep_their_tails(act, kind):
    """Relative to the value itself.  GELU below zero is |z| / 2 erfc: the exponential is off by
    2^-22, t P(t) by 2^-23 (the reciprocal), 2^-22 (its sums) and 2^-26 (the fit), four products
    by 2^-24 each, 2^-20 together, and the exponent z^2 / 2 by three roundings of 2^-24 (z^2, the
    constant, their product), below z^2 2^-23; above zero |z| / 2 erfc is at most z.  SiLU: the
    exponential by 2^-22 and |z| 2^-24 (its argument), the quotient by 2^-22, three products:
    (|z| + 4) 2^-22 covers it.  bf16: half a step more.  The reference takes the tail from
    erfc: 1 + erf, as ndtr has it, leaves nothing of it in 64 bits either."""
    z = z_values(kind)
    zd = z.double()
    if act == "gelu":
        rel = 2.0 ** -20 + zd * zd * 2.0 ** -23
        ref = 0.5 * zd * torch.special.erfc(-zd * math.sqrt(0.5))
    else:
        rel = (zd.abs() + 4) * 2.0 ** -22
        ref = act64(zd, act)
    y = activation_of(z, act)
    assert ((y.double() - ref).abs() <= rel * ref.abs()).all()
    y16 = activation_of(z, act, BF)
    assert ((y16.double() - ref).abs() <= (half_step(BF) * (1 + rel) + rel) * ref.abs()).all()


@pytest.mark.parametrize("kind", ["normal", "wide", "far"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_slopes_of_the_activations(act, kind):
    """Off by the errors of the two terms, each as in the test above, and their sum's rounding."""
    z = z_values(kind)
    zd = z.double()
    p = torch.sigmoid(zd) if act == "silu" else torch.special.ndtr(zd)
    second = zd * p * (1 - p) if act == "silu" else zd * torch.exp(-zd * zd / 2) / math.sqrt(2 * math.pi)
    rel = 2.0 ** -20 + zd * zd * 2.0 ** -23 if act == "gelu" else (zd.abs() + 4) * 2.0 ** -22
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-zd * math.sqrt(0.5))
    s = slope_of(z, act)
    assert ((s.double() - (p + second)).abs() <= rel * (p + second.abs()) + 1e-37).all()


def test_gelu_errors_are_those_of_fp32_arithmetic():
    """Root mean squares over normal z.  The slope is a sum of about five roundings of at most
    2^-24 each, 2^-24 sqrt(5 / 3) = 7.7e-8 if they are independent; of the activation they
    reach |z| / 2 erfc <= 0.17, and the sum's own rounding stays: 0.75 * 2^-24 = 4.5e-8."""
    z = z_values("normal")
    rms = lambda e: e.double().square().mean().sqrt().item()  # noqa: E731
    assert rms(activation_of(z, "gelu").double() - act64(z.double(), "gelu")) <= 4.5e-8
    assert rms(slope_of(z, "gelu").double() - slope64(z.double(), "gelu")) <= 7.7e-8


@pytest.mark.parametrize("shape", [(2, 257, 320, 32), (1, 70001, 64, 8)], ids=str)
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_fp32_results_are_as_close_as_elementary_fp32(act, shape):
    """Root mean square errors of fp32 results against the 64-bit definition, beside those of the
    same formulas in elementary fp32 operations: each side rounds every element a handful of
    times, the kernels up to twice as often (two constants of z, the tail's factors), so up to
    sqrt 2 of that error is theirs; 2 leaves room for the sums' different orders."""
    B, S, C, G = shape
    x, gamma, beta, g = make(B, S, C, F32, seed=C + S)
    dy = torch.randn(B, S, C, generator=g, device="cuda")
    half = math.sqrt(0.5)

    def forward(x, gamma, beta):
        v = x.view(B, S, G, C // G)
        mean = v.mean((1, 3), keepdim=True)
        rstd = 1 / torch.sqrt((v - mean).square().mean((1, 3), keepdim=True) + 1e-5)
        hat = ((v - mean) * rstd).view(B, S, C)
        z = hat * gamma + beta
        p = 1 / (1 + torch.exp(-z)) if act == "silu" else 0.5 * (1 + torch.erf(z * half))
        return hat, rstd, z, p

    def backward(x, dy, gamma, beta):
        hat, rstd, z, p = forward(x, gamma, beta)
        d = {"none": lambda: torch.ones_like(z), "silu": lambda: p * (1 + z * (1 - p)),
             "gelu": lambda: p + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)}[act]()
        dz = dy * d
        dh = (dz * gamma).view(B, S, G, -1)
        h = hat.view(B, S, G, -1)
        dx = rstd * (dh - dh.mean((1, 3), keepdim=True) - h * (dh * h).mean((1, 3), keepdim=True))
        return dx.reshape(B, S, C), (dz * hat).sum((0, 1)), dz.sum((0, 1))

    def value(x, gamma, beta):
        _, _, z, p = forward(x, gamma, beta)
        return z if act == "none" else z * p

    rms = lambda t, r: (t.double() - r).square().mean().sqrt().item()  # noqa: E731
    ref = value(x.double(), gamma.double(), beta.double())
    y, stats = pq.group_norm_act(x, G, gamma, beta, act=act, return_stats=True)
    assert rms(y, ref) <= 2 * rms(value(x, gamma, beta), ref)
    want = backward(x.double(), dy.double(), gamma.double(), beta.double())
    for got, plain, r in zip(pq.group_norm_act_backward(dy, x, stats, gamma, beta, act=act),
                             backward(x, dy, gamma, beta), want):
        assert rms(got, r) <= 2 * rms(plain, r)


def test_activations_of_infinities_and_nan():
    """GELU of +infinity is +infinity and of -infinity zero, its slopes are 1 and 0; a NaN reaches
    no other channel, not the one that shares its reciprocal either (whose last bits may
    follow the NaN's place, (|z| + 4) 2^-21 for two results within their bounds)."""
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([inf, -inf, 1e30, -1e30, 40.0, -40.0, 3.0, -3.0], device="cuda").repeat(4)
    y, s = activation_of(z, "gelu"), slope_of(z, "gelu")
    assert (y[0::8] == inf).all() and (y[2::8] == 1e30).all() and (y[4::8] == 40).all()
    assert (y[1::8] == 0).all() and (y[3::8] == 0).all() and (y[5::8] == 0).all()
    assert (s[0:6:2] == 1).all() and (s[1:6:2] == 0).all()
    assert (activation_of(z, "silu")[2::8] == 1e30).all() and (activation_of(z, "silu")[3::8] == 0).all()
    z = z_values("normal")[:4096]
    for act in ("silu", "gelu"):
        clean = activation_of(z, act), slope_of(z, act)
        for part in (0, 1):
            bad = z.clone()
            bad[part::2] = nan
            for want, got in zip(clean, (activation_of(bad, act), slope_of(bad, act))):
                assert torch.isnan(got[part::2]).all()
                w, v = want[1 - part::2].double(), got[1 - part::2].double()
                tol = (z[1 - part::2].double().abs() + 4) * 2.0 ** -21 * w.abs().clamp(min=1)
                assert ((w - v).abs() <= tol).all()


# ------------------------------------------------------------- streams, graphs
def test_other_stream_and_graph_replay():
    x, gamma, beta, g = make(2, 300, 320, BF, seed=31)
    big, _, _, _ = make(1, 70000, 64, BF, seed=32)
    dy = torch.randn(2, 300, 320, generator=g, device="cuda").to(BF)
    want, stats = pq.group_norm_act(x, 32, gamma, beta, act="silu", return_stats=True)
    want_big = pq.group_norm_act(big, 8, act="gelu")
    want_g = pq.group_norm_act_backward(dy, x, stats, gamma, beta, act="silu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = pq.group_norm_act(big, 8, act="gelu", stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want_big)

    xs, bs = torch.zeros_like(x), torch.zeros_like(big)
    graphs = []
    with torch.cuda.stream(s):
        for _ in range(2):                                 # two graphs, each with its own workspaces
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                y1, st = pq.group_norm_act(xs, 32, gamma, beta, act="silu", return_stats=True)
                y2 = pq.group_norm_act(bs, 8, act="gelu")
                gr = pq.group_norm_act_backward(dy, xs, st, gamma, beta, act="silu")
            graphs.append((graph, y1, y2, gr))
    torch.cuda.synchronize()
    xs.copy_(x)
    bs.copy_(big)
    for graph, y1, y2, gr in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for graph, y1, y2, gr in graphs:
        assert torch.equal(y1, want) and torch.equal(y2, want_big)
        assert all(torch.equal(a, b) for a, b in zip(gr, want_g))


def calls_with_results():
    """Calls of every entry point that allocates: name -> (f(stream) -> results)."""
    x, gamma, beta, g = make(2, 300, 320, BF, seed=33)
    big, _, _, _ = make(1, 70000, 64, BF, seed=34)         # two passes: a workspace, too
    dy = torch.randn(2, 300, 320, generator=g, device="cuda").to(BF)
    _, stats = pq.group_norm_act(x, 32, gamma, beta, act="silu", return_stats=True)
    scale = torch.full((1,), 0.05, device="cuda")
    rows, out = x.view(600, 320), torch.randn(600, 256, generator=g, device="cuda").to(BF)
    ad = pq.Adapters((torch.randn(2, 16, 320, generator=g, device="cuda") / 18).to(BF),
                     (torch.randn(2, 256, 16, generator=g, device="cuda") / 4).to(BF))
    bounds = torch.tensor([0, 200, 600], dtype=torch.int32, device="cuda")
    index = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    _, hidden = pq.adapter_add(out.clone(), rows, ad, bounds, index, return_hidden=True)
    return {
        "norm": lambda s: pq.group_norm_act(x, 32, gamma, beta, act="silu", return_stats=True, stream=s),
        "norm of a large map": lambda s: (pq.group_norm_act(big, 8, act="gelu", stream=s),),
        "norm to fp32": lambda s: (pq.group_norm_act(x, 32, out_dtype=F32, stream=s),),
        "codes": lambda s: pq.quantize_activations_norm(x, 32, gamma, beta, (0, 320), scale, scale, return_y=True,
                                                        stream=s),
        "norm gradients": lambda s: pq.group_norm_act_backward(dy, x, stats, gamma, beta, act="silu", stream=s),
        "hidden": lambda s: pq.adapter_add(torch.zeros_like(out), rows, ad, bounds, index, return_hidden=True,
                                           stream=s)[1:],
        "adapter gradients": lambda s: pq.adapter_backward(out, rows, hidden, ad, bounds, index, stream=s),
    }


@pytest.mark.parametrize("name", ["norm", "norm of a large map", "norm to fp32", "codes", "norm gradients", "hidden",
                                  "adapter gradients"])
def test_results_on_an_explicit_stream_take_no_block_in_use(name):
    """Blocks that were freed on the current stream while its kernels still wait to write them
    are not given to a call on another stream, which would run ahead of those kernels."""
    f = calls_with_results()[name]
    want = [t.clone() for t in f(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    blocks = [torch.empty_like(t) for t in want for _ in range(2)]
    torch.cuda._sleep(100_000_000)                         # about 50 ms
    for b in blocks:
        b.fill_(77)
    del blocks, b
    got = f(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_empty_maps():
    for shape in ((0, 5, 64), (2, 0, 64)):
        x = torch.empty(shape, device="cuda", dtype=BF)
        y, stats = pq.group_norm_act(x, 8, return_stats=True)
        assert y.shape == x.shape
        dx, dgamma, dbeta = pq.group_norm_act_backward(x, x, torch.zeros(shape[0], 8, 2, device="cuda"))
        assert dx.shape == x.shape and (dgamma == 0).all() and (dbeta == 0).all()


@pytest.mark.parametrize("shape", [(8, 1024, 640, 32), (2, 16129, 320, 32), (1, 65536, 256, 32)], ids=str)
def test_results_repeat_under_load(shape):
    """The same call over and over, calls of another size in flight around it, gives the same bits."""
    B, S, C, G = shape
    x, gamma, beta, g = make(B, S, C, BF, seed=3)
    dy = torch.randn(B, S, C, generator=g, device="cuda").to(BF)
    small, _, _, _ = make(2, 64, C, BF, seed=4)
    want, stats = pq.group_norm_act(x, G, gamma, beta, act="silu", return_stats=True)
    grads = pq.group_norm_act_backward(dy, x, stats, gamma, beta, act="silu")
    for _ in range(20):
        pq.group_norm_act(small, G, gamma, beta)
        y, st = pq.group_norm_act(x, G, gamma, beta, act="silu", return_stats=True)
        again = pq.group_norm_act_backward(dy, x, st, gamma, beta, act="silu")
        assert torch.equal(y, want) and torch.equal(st, stats)
        assert all(torch.equal(a, b) for a, b in zip(again, grads))
