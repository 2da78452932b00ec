"""Low-rank adapters of many requests beside a shared projection, and the run
norm -> codes -> quantized linear -> adapters, against 64-bit definitions.

Tolerances: products of bf16 values are exact in fp32; sums over K or N run in fp32
(64 roundings of 2^-24 of the absolute terms cover chains whose roundings are
independent).  Between the two products of a row, h (or u) is fp32; the tensor-core
form multiplies it as a sum of bf16 parts, off by at most 2^-17 of itself for bf16
outputs and 2^-24 for fp32 outputs.  The output's rounding: eps / 2 relative.
"""
import types

import pytest
import torch

import post_quantized_linear_b200 as pq

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def half_step(t):
    return torch.finfo(t).eps / 2


def make(M, K, N, L, R, dtype=BF, ydtype=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rn(M, K).to(dtype)
    y = rn(M, N).to(ydtype or dtype)
    ad = pq.Adapters((rn(L, R, K) / K ** 0.5).to(BF), (rn(L, N, R) / R ** 0.5).to(BF),
                     0.5 + torch.rand(L, generator=g, device="cuda"))
    return x, y, ad, g


def requests(lengths, index, first=0):
    b = torch.tensor([first] + lengths, dtype=torch.int32).cumsum(0).to(torch.int32)
    return b.cuda(), torch.tensor(index, dtype=torch.int32).cuda()


def rows_of(bounds, index):
    b = bounds.tolist()
    return [(slice(b[q], b[q + 1]), l) for q, l in enumerate(index.tolist()) if l >= 0 and b[q + 1] > b[q]]


def forward64(y, x, ad, bounds, index):
    """(y, hidden) and bounds on the fp32 errors."""
    out, e = y.double().clone(), torch.zeros_like(y, dtype=torch.float64)
    R = ad.a.shape[1]
    hid = torch.zeros(x.shape[0], R, dtype=torch.float64, device="cuda")
    e_h = torch.zeros_like(hid)
    part = 2.0 ** -17 if y.dtype == BF else U
    for m, l in rows_of(bounds, index):
        A, B, s = ad.a[l].double(), ad.b[l].double(), 1.0 if ad.scale is None else ad.scale[l].double()
        hid[m] = x[m].double() @ A.t()
        e_h[m] = 64 * U * (x[m].double().abs() @ A.abs().t())
        out[m] += s * (hid[m] @ B.t())
        e[m] = s * ((e_h[m] + (64 * U + part) * hid[m].abs()) @ B.abs().t()) + U * y[m].double().abs()
    return (out, hid), (e, e_h)


def backward64(dy, x, hidden, ad, bounds, index):
    dx = torch.zeros_like(x, dtype=torch.float64)
    da, db = torch.zeros_like(ad.a, dtype=torch.float64), torch.zeros_like(ad.b, dtype=torch.float64)
    e_dx, e_da, e_db = torch.zeros_like(dx), torch.zeros_like(da), torch.zeros_like(db)
    part = 2.0 ** -17 if x.dtype == BF else U
    for m, l in rows_of(bounds, index):
        A, B, s = ad.a[l].double(), ad.b[l].double(), 1.0 if ad.scale is None else ad.scale[l].double()
        g, v, h = dy[m].double(), x[m].double(), hidden[m].double()
        u = s * (g @ B)
        e_u = 64 * U * s * (g.abs() @ B.abs())
        dx[m] = u @ A
        e_dx[m] = (e_u + (64 * U + part) * u.abs()) @ A.abs()
        da[l] += u.t() @ v
        e_da[l] += (e_u + 64 * U * u.abs()).t() @ v.abs()
        db[l] += s * (g.t() @ h)
        e_db[l] += 64 * U * s * (g.abs().t() @ h.abs())
    return (dx, da, db), (e_dx, e_da, e_db)


def check(got, ref, bound):
    assert got.shape == ref.shape
    tol = bound + half_step(got.dtype) * (ref.abs() + bound) + 1e-38
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.float()).all()
    assert (err <= tol).all(), f"worst {(err / tol).max().item():.2f} of the tolerance"


# M, K, N, L, R, lengths, index, first row
CASES = {
    "one_row": (1, 128, 64, 1, 8, [1], [0], 0),
    "single_rows": (37, 1152, 3456, 5, 16, [1] * 37, [(3 * i) % 5 for i in range(37)], 0),
    "few_rows_each": (61, 768, 256, 4, 24, [3, 0, 9, 1, 17, 8, 16], [1, 2, -1, 3, 0, 0, 1], 5),
    "one_request": (300, 512, 400, 1, 64, [300], [0], 0),
    "ragged": (777, 1152, 2304, 3, 40, [128, 1, 0, 127, 129, 200, 31], [0, 2, 1, -1, 2, 0, 0], 100),
    "largest_rank": (260, 272, 1040, 2, 128, [130, 130], [1, 0], 0),
    "narrow": (200, 16, 16, 2, 8, [100, 99], [1, 1], 0),
    "many_requests": (1500, 256, 128, 7, 32, [1, 2] * 500, [i % 8 - 1 for i in range(1000)], 0),
    "long": (2500, 640, 1920, 2, 16, [2300, 7], [1, 0], 33),
    "none": (40, 128, 64, 2, 8, [20, 20], [-1, -3], 0),
    "single_rows_many": (613, 128, 96, 4, 8, [1] * 600, [i % 5 - 1 for i in range(600)], 7),
    "tiles_of_many_requests": (2700, 192, 208, 3, 24, [9, 0, 17] * 100, [i % 4 - 1 for i in range(300)], 3),
    "middle_rank": (900, 320, 336, 2, 72, [513, 130, 64], [1, 0, 1], 11),
}


@pytest.mark.parametrize("dtype,ydtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)], ids=str)
@pytest.mark.parametrize("case", CASES)
def test_forward_matches_definition(case, dtype, ydtype):
    M, K, N, L, R, lengths, index, first = CASES[case]
    x, y, ad, _ = make(M, K, N, L, R, dtype, ydtype, seed=M)
    bounds, idx = requests(lengths, index, first)
    (ref, hid), (e, e_h) = forward64(y, x, ad, bounds, idx)
    before = y.clone()
    out, hidden = pq.adapter_add(y, x, ad, bounds, idx, return_hidden=True)
    assert out is y
    check(y, ref, e)
    check(hidden, hid, e_h)
    untouched = torch.ones(M, dtype=torch.bool, device="cuda")
    for m, _ in rows_of(bounds, idx):
        untouched[m] = False
    assert torch.equal(y[untouched], before[untouched])
    again = pq.adapter_add(before, x, ad, bounds, idx)
    assert torch.equal(again, y)
    assert pq.stream_status() == 0


@pytest.mark.parametrize("dtype,dydtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)], ids=str)
@pytest.mark.parametrize("case", CASES)
def test_gradients_match_the_formula(case, dtype, dydtype):
    M, K, N, L, R, lengths, index, first = CASES[case]
    x, dy, ad, _ = make(M, K, N, L, R, dtype, dydtype, seed=M + 1)
    bounds, idx = requests(lengths, index, first)
    _, hidden = pq.adapter_add(torch.zeros_like(dy), x, ad, bounds, idx, return_hidden=True)
    got = pq.adapter_backward(dy, x, hidden, ad, bounds, idx)
    want, e = backward64(dy, x, hidden, ad, bounds, idx)
    for a, b, c in zip(got, want, e):
        check(a, b, c)
    again = pq.adapter_backward(dy, x, hidden, ad, bounds, idx)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert pq.stream_status() == 0


def test_gradients_match_differences():
    """Central differences of the 64-bit term: exact but for roundings, the term is linear
    in each argument; the kernel's fp32 sums are off by about 1e-6 of the terms."""
    x, dy, ad, g = make(90, 128, 96, 2, 16, F32, F32, seed=4)
    bounds, idx = requests([40, 30, 20], [1, 0, 1])
    zero = torch.zeros_like(dy)
    _, hidden = pq.adapter_add(zero.clone(), x, ad, bounds, idx, return_hidden=True)
    grads = pq.adapter_backward(dy, x, hidden, ad, bounds, idx)

    def f(x, a, b):
        t = types.SimpleNamespace(a=a, b=b, scale=ad.scale)
        return (forward64(zero, x, t, bounds, idx)[0][0] * dy.double()).sum()

    at = [x.double(), ad.a.double(), ad.b.double()]
    for i in range(3):
        v = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        lo, hi = list(at), list(at)
        lo[i], hi[i] = at[i] - 0.5 * v, at[i] + 0.5 * v
        want = (f(*hi) - f(*lo)).item()
        terms = (grads[i].double() * v).abs().sum().item()
        assert abs((grads[i].double() * v).sum().item() - want) <= 1e-5 * terms


@pytest.mark.parametrize("dtype", [BF, F32], ids=str)
@pytest.mark.parametrize("case", CASES)
def test_forward_into_another_output_rounds_once(case, dtype):
    """y fp32 into a bf16 out: y + the term within one half step, y's values rounded where there
    is no adapter, nothing around out and nothing of y changed."""
    M, K, N, L, R, lengths, index, first = CASES[case]
    x, y, ad, _ = make(M, K, N, L, R, dtype, F32, seed=M + 2)
    bounds, idx = requests(lengths, index, first)
    (ref, hid), (_, e_h) = forward64(y, x, ad, bounds, idx)
    _, (e, _) = forward64(y.to(BF), x, ad, bounds, idx)    # h in two parts, as for a bf16 y
    before = y.clone()
    room = torch.full((M, N + 24), 7.0, device="cuda", dtype=BF)
    out = room[:, 8:N + 8]
    got, hidden = pq.adapter_add(y, x, ad, bounds, idx, return_hidden=True, out=out)
    assert got is out and torch.equal(y, before)
    check(out, ref, e)
    check(hidden, hid, e_h)
    none = torch.ones(M, dtype=torch.bool, device="cuda")
    for m, _ in rows_of(bounds, idx):
        none[m] = False
    assert torch.equal(out[none], y[none].to(BF))
    assert (room[:, :8] == 7).all() and (room[:, N + 8:] == 7).all()
    assert torch.equal(pq.adapter_add(y, x, ad, bounds, idx, out=torch.empty(M, N, device="cuda", dtype=BF)), out)
    assert pq.stream_status() == 0


def test_forward_into_another_output_refusals_and_empty_batches():
    x, y, ad, _ = make(20, 128, 64, 2, 8, BF, F32)
    bounds, idx = requests([20], [1])
    out = torch.empty(20, 64, device="cuda", dtype=BF)
    with pytest.raises(TypeError, match="float32 and out bfloat16"):
        pq.adapter_add(y.to(BF), x, ad, bounds, idx, out=out)
    with pytest.raises(TypeError, match="float32 and out bfloat16"):
        pq.adapter_add(y, x, ad, bounds, idx, out=torch.empty_like(y))
    with pytest.raises(ValueError, match="out must be"):
        pq.adapter_add(y, x, ad, bounds, idx, out=out[:, :32])
    with pytest.raises(ValueError, match="out must be"):
        pq.adapter_add(y, x, ad, bounds, idx, out=out.cpu())
    none, start = idx[:0], bounds[:1]
    assert torch.equal(pq.adapter_add(y, x, ad, start, none, out=out), y.to(BF))
    assert pq.adapter_add(y[:0], x[:0], ad, start, none, out=out[:0]).shape == (0, 64)
    # a request that is left out: its rows are rows without an adapter
    bad = torch.tensor([0, 12, 30], dtype=torch.int32, device="cuda")
    two = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    pq.adapter_add(y, x, ad, bad, two, out=out)
    assert pq.stream_status() == pq._lib.SQ_ERR_RANGE
    assert torch.equal(out[12:], y[12:].to(BF)) and not torch.equal(out[:12], y[:12].to(BF))


def test_column_slices_strides_and_no_scale():
    """A fused q | k | v output with adapters of its own per part, in a padded buffer."""
    x0, y0, ad, g = make(150, 272, 3 * 128 + 16, 2, 16, seed=8)
    x, y = x0[:, 8:264], y0[:, 8:392]
    bounds, idx = requests([70, 5, 70], [0, 1, 1], 2)
    parts = [pq.Adapters(ad.a[:, :, i * 8:i * 8 + 256].contiguous(), ad.b[:, 128 * i:128 * i + 128].contiguous())
             for i in range(2)]
    want = y0.double().clone()
    err = torch.zeros_like(want)
    for i, p in enumerate(parts):
        cols = slice(8 + 128 * i, 8 + 128 * i + 128)
        (want[:, cols], _), (err[:, cols], _) = forward64(y0[:, cols], x, p, bounds, idx)
    for i, p in enumerate(parts):
        pq.adapter_add(y[:, 128 * i:128 * i + 128], x, p, bounds, idx)
    check(y0, want, err)


def test_non_finite_rows_of_other_requests():
    """Infinities and NaN in rows of no request, or of another one, reach nothing else."""
    for lengths in ([60, 100, 90], [1, 1, 1]):
        M = sum(lengths) + 6
        x, y, ad, g = make(M, 256, 192, 3, 16, seed=6)
        dy = torch.randn(M, 192, generator=g, device="cuda").to(BF)
        bounds, idx = requests(lengths, [0, 1, 2], 3)
        b = bounds.tolist()
        y2, want_h = pq.adapter_add(y.clone(), x, ad, bounds, idx, return_hidden=True)
        want_g = pq.adapter_backward(dy, x, want_h, ad, bounds, idx)
        bad = torch.zeros(M, dtype=torch.bool, device="cuda")
        bad[:b[0]] = bad[b[3]:] = bad[b[1]:b[2]] = True
        xb, dyb = x.clone(), dy.clone()
        xb[bad], dyb[bad] = float("nan"), float("inf")
        yb, hb = pq.adapter_add(y.clone(), xb, ad, bounds, idx, return_hidden=True)
        assert torch.equal(yb[~bad], y2[~bad]) and torch.equal(hb[~bad], want_h[~bad])
        assert torch.equal(yb[:b[0]], y[:b[0]]) and torch.equal(yb[b[3]:], y[b[3]:])
        dx, da, db = pq.adapter_backward(dyb, xb, hb, ad, bounds, idx)
        assert torch.equal(dx[~bad], want_g[0][~bad])
        for l in (0, 2):
            assert torch.equal(da[l], want_g[1][l]) and torch.equal(db[l], want_g[2][l])


@pytest.mark.parametrize("dtype", [BF, F32], ids=str)
@pytest.mark.parametrize("R", [8, 72, 128])
@pytest.mark.parametrize("lengths", [[1, 2, 3, 0, 1] * 15, [1, 70, 3, 130, 2, 61, 64, 1, 5], [2, 1, 1] * 100],
                         ids=["one to three rows", "uneven", "300 requests"])
def test_short_requests_share_steps(lengths, R, dtype):
    """Requests of a row or two, whose rows share a step of the gradients' sums, beside long
    ones that are cut in its middle; up to two rows a request on average, and more."""
    M = sum(lengths) + 3
    x, dy, ad, _ = make(M, 272, 208, 3, R, dtype, seed=M + R)
    bounds, idx = requests(lengths, [(i * 7 + i // 5) % 4 - 1 for i in range(len(lengths))])
    y = torch.zeros_like(dy)
    (ref, hid), (e, e_h) = forward64(y, x, ad, bounds, idx)
    _, hidden = pq.adapter_add(y, x, ad, bounds, idx, return_hidden=True)
    check(y, ref, e)
    check(hidden, hid, e_h)
    got = pq.adapter_backward(dy, x, hidden, ad, bounds, idx)
    want, e = backward64(dy, x, hidden, ad, bounds, idx)
    for a, b, c in zip(got, want, e):
        check(a, b, c)
    again = pq.adapter_backward(dy, x, hidden, ad, bounds, idx)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert pq.stream_status() == 0


@pytest.mark.parametrize("M,Q", [(70000, 70000), (70000, 5000), (3000, 100000)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=str)
def test_a_hundred_thousand_requests(M, Q, dtype):
    """One row each, fourteen, and mostly empty ones."""
    x, dy, ad, g = make(M, 64, 48, 5, 8, dtype, seed=Q)
    cuts = torch.randint(0, M + 1, (Q + 1,), generator=g, device="cuda").sort().values
    bounds = (torch.arange(Q + 1, device="cuda") if Q == M else cuts).to(torch.int32)
    idx = torch.randint(-1, 5, (Q,), generator=g, device="cuda", dtype=torch.int32)
    # the adapter of each row; then one request per adapter, of its rows in order
    which = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    rows = bounds[1:] - bounds[:-1]
    which[bounds[0]:bounds[-1]] = idx.repeat_interleave(rows)
    order = torch.argsort(which, stable=True)
    b = torch.searchsorted(which[order], torch.arange(6, device="cuda", dtype=torch.int32)).to(torch.int32)
    l = torch.arange(5, device="cuda", dtype=torch.int32)
    y = torch.zeros_like(dy)
    _, hidden = pq.adapter_add(y, x, ad, bounds, idx, return_hidden=True)
    (ref, hid), (e, e_h) = forward64(torch.zeros_like(dy), x[order], ad, b, l)
    check(y[order], ref, e)
    check(hidden[order], hid, e_h)
    dx, da, db = pq.adapter_backward(dy, x, hidden, ad, bounds, idx)
    want, e = backward64(dy[order], x[order], hidden[order], ad, b, l)
    for got, r, t in zip((dx[order], da, db), want, e):
        check(got, r, t)
    assert pq.stream_status() == 0


@pytest.mark.parametrize("rows", [1, 90])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_non_finite_adapters_of_other_requests(rows, dtype):
    """Infinities and NaN in another adapter reach nothing else: ranks, columns and rows of
    this one that do not fill the kernels' tiles meet zeros, not their neighbours."""
    x, y, ad, g = make(3 * rows, 272, 400, 3, 24, dtype, seed=5)
    dy = torch.randn(3 * rows, 400, generator=g, device="cuda").to(dtype)
    bounds, idx = requests([rows] * 3, [0, 1, 2])
    want, h = pq.adapter_add(y.clone(), x, ad, bounds, idx, return_hidden=True)
    grads = pq.adapter_backward(dy, x, h, ad, bounds, idx)
    a, b = ad.a.clone(), ad.b.clone()
    a[1], b[1] = float("nan"), float("inf")
    bad = pq.Adapters(a, b, ad.scale)
    got, h2 = pq.adapter_add(y.clone(), x, bad, bounds, idx, return_hidden=True)
    again = pq.adapter_backward(dy, x, h2, bad, bounds, idx)
    keep = torch.ones(3 * rows, dtype=torch.bool, device="cuda")
    keep[rows:2 * rows] = False
    assert torch.equal(got[keep], want[keep]) and torch.equal(again[0][keep], grads[0][keep])
    for l in (0, 2):
        assert torch.equal(again[1][l], grads[1][l]) and torch.equal(again[2][l], grads[2][l])


def test_two_streams_at_once():
    """Calls in flight on two streams share nothing."""
    sets = []
    for k in range(2):
        x, y, ad, g = make(3000, 768, 512, 3, 32, seed=20 + k)
        dy = torch.randn(3000, 512, generator=g, device="cuda").to(BF)
        bounds, idx = requests([1000, 900, 1100], [k, 1, 2])
        want, h = pq.adapter_add(y.clone(), x, ad, bounds, idx, return_hidden=True)
        sets.append((x, y, ad, dy, bounds, idx, want, h, pq.adapter_backward(dy, x, h, ad, bounds, idx)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for k, (x, y, ad, dy, bounds, idx, _, h, _) in enumerate(sets):
            with torch.cuda.stream(streams[k]):
                got[k].append((pq.adapter_add(y.clone(), x, ad, bounds, idx), pq.adapter_backward(dy, x, h, ad, bounds, idx)))
    torch.cuda.synchronize()
    for k in range(2):
        for out, grads in got[k]:
            assert torch.equal(out, sets[k][6])
            assert all(torch.equal(a, b) for a, b in zip(grads, sets[k][8]))
    assert pq.stream_status() == 0


def test_starved_rings_time_out_and_the_context_recovers(dev_lib):
    """No copy arrives (a host switch of the development library): every wait of the two
    kernels runs out, the status says so, and the next calls are right."""
    x, y, ad, g = make(700, 512, 320, 2, 16, seed=30)
    bounds, idx = requests([300, 400], [0, 1])
    want, h = pq.adapter_add(y.clone(), x, ad, bounds, idx, return_hidden=True)
    grads = pq.adapter_backward(y, x, h, ad, bounds, idx)
    assert pq.stream_status() == 0
    pq.set_wait_budget(2_000_000)
    pq.debug_starve_pipeline(True)
    try:
        pq.adapter_add(y.clone(), x, ad, bounds, idx)
        assert pq.stream_status() == pq._lib.SQ_ERR_TIMEOUT
        pq.adapter_backward(y, x, h, ad, bounds, idx)
        assert pq.stream_status() == pq._lib.SQ_ERR_TIMEOUT
    finally:
        pq.debug_starve_pipeline(False)
        pq.set_wait_budget(0)
    assert torch.equal(pq.adapter_add(y.clone(), x, ad, bounds, idx), want)
    assert all(torch.equal(a, b) for a, b in zip(pq.adapter_backward(y, x, h, ad, bounds, idx), grads))
    assert pq.stream_status() == 0


@pytest.mark.parametrize("lengths", [[300, 400], [130] * 40], ids=["clusters of eight", "more pieces"])
def test_rings_starved_in_the_middle_time_out_too(dev_lib, lengths):
    """The copies end after some steps of the first or the second product: every wait has a
    limit there as well, the two warps that share a quarter's barriers leave the loop over the
    output tiles together, the status reports it, and the next calls are right."""
    M = sum(lengths)
    x, y, ad, g = make(M, 1344, 1344, 2, 40, seed=31)
    bounds, idx = requests(lengths, [i % 2 for i in range(len(lengths))])
    want, h = pq.adapter_add(y.clone(), x, ad, bounds, idx, return_hidden=True)
    grads = pq.adapter_backward(y, x, h, ad, bounds, idx)
    assert pq.stream_status() == 0
    starve = dev_lib.sq_debug_starve_pipeline
    pq.set_wait_budget(2_000_000)
    try:
        for copies in range(1, 13):
            assert starve(1 + copies) == 0
            pq.adapter_backward(y, x, h, ad, bounds, idx)
            assert pq.stream_status() == pq._lib.SQ_ERR_TIMEOUT
            if copies < 4:                       # fewer than any CTA's share of both products
                pq.adapter_add(y.clone(), x, ad, bounds, idx)
                assert pq.stream_status() == pq._lib.SQ_ERR_TIMEOUT
    finally:
        pq.debug_starve_pipeline(False)
        pq.set_wait_budget(0)
    assert torch.equal(pq.adapter_add(y.clone(), x, ad, bounds, idx), want)
    assert all(torch.equal(a, b) for a, b in zip(pq.adapter_backward(y, x, h, ad, bounds, idx), grads))
    assert pq.stream_status() == 0


def test_bad_requests_are_left_out_and_reported():
    """Bounds outside the batch and an unknown adapter: the kernels' own checks leave those
    requests out and raise the range status; falling bounds raise it, and which rows of
    the batch then receive their term is not specified."""
    x, y, ad, _ = make(100, 128, 64, 2, 8, seed=2)
    for b, i in (([0, 50, 300], [0, 1]), ([0, 50, 100], [0, 2]), ([0, 50, 20, 100], [0, 1, -1])):
        bounds, idx = torch.tensor(b, dtype=torch.int32).cuda(), torch.tensor(i, dtype=torch.int32).cuda()
        good = slice(0, 50)
        (ref, _), (e, _) = forward64(y[good], x[good], ad, bounds[:2], idx[:1])
        out = pq.adapter_add(y.clone(), x, ad, bounds, idx)
        if b == sorted(b):
            check(out[good], ref, e)
            assert torch.equal(out[50:], y[50:])
        assert pq.stream_status() == pq._lib.SQ_ERR_RANGE
    assert pq.stream_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32], ids=str)
@pytest.mark.parametrize("lengths", [[50, 50], [1] * 60, [9] * 20, [9] * 400], ids=lambda v: f"{len(v)} requests")
def test_a_bound_far_outside_the_batch_costs_no_other_request(lengths, dtype):
    """The first bound below zero, or the last one behind the batch: that request is left out
    and the status says so; every other one gets its term, whichever form takes the batch."""
    M = sum(lengths)
    x, y, ad, _ = make(M, 128, 64, 3, 16, dtype, seed=M)
    bounds, idx = requests(lengths, [i % 3 for i in range(len(lengths))])
    for at, value, rows in ((0, -1000, slice(0, lengths[0])), (-1, M + 100000, slice(M - lengths[-1], M)),
                            (0, -2 ** 31, slice(0, lengths[0])), (-1, 2 ** 31 - 1, slice(M - lengths[-1], M))):
        good = idx.clone()
        good[at] = -1
        want = pq.adapter_add(y.clone(), x, ad, bounds, good)
        assert pq.stream_status() == 0
        bad = bounds.clone()
        bad[at] = value
        out = pq.adapter_add(y.clone(), x, ad, bad, idx)
        assert pq.stream_status() == pq._lib.SQ_ERR_RANGE
        assert torch.equal(out, want) and torch.equal(out[rows], y[rows])


@pytest.mark.parametrize("dtype", [BF, F32], ids=str)
@pytest.mark.parametrize("lengths", [[50, 50], [100, 30, 70, 100], [1] * 60, [9] * 400],
                         ids=lambda v: f"{len(v)} requests")
def test_requests_left_out_of_the_gradients(lengths, dtype):
    """A request with a bound outside the batch or an unknown adapter, beside good ones of the
    same adapter: its rows of hidden and dx are zeros, and the gradients are those of the other
    requests alone, whatever the workspace and its rows of hidden held before."""
    M, K, N, R = sum(lengths), 128, 64, 24
    x, dy, ad, _ = make(M, K, N, 2, R, dtype, seed=M)
    n = len(lengths)
    bounds, idx = requests(lengths, [1] * n)
    first, last = slice(0, lengths[0]), slice(M - lengths[-1], M)
    nan = float("nan")
    for what, at, value, rows in (("bound", 0, -3, first), ("bound", n, M + 200, last), ("index", n - 1, 2, last),
                                  ("index", 0, 2 ** 31 - 1, first)):
        good, bad_b, bad_i = idx.clone(), bounds.clone(), idx.clone()
        good[0 if rows is first else -1] = -1
        (bad_b if what == "bound" else bad_i)[at] = value
        _, hidden = pq.adapter_add(torch.zeros_like(dy), x, ad, bounds, good, return_hidden=True)
        want = pq.adapter_backward(dy, x, hidden, ad, bounds, good)
        # the C entries, so that every buffer can hold NaN before the calls
        lib = pq._lib.load()
        h = torch.full((M, R), nan, device="cuda")
        dx = torch.full((M, K), nan, device="cuda", dtype=dtype)
        da, db = torch.full_like(want[1], nan), torch.full_like(want[2], nan)
        wn = pq._adapter_workspace_size(M, R)
        ws = torch.full((wn // 4,), nan, device="cuda")
        t, c = pq._dtype_code(dtype), ad.c_struct()
        s = torch.cuda.current_stream().cuda_stream
        assert lib.sq_adapter_add(x.data_ptr(), t, M, K, c, bad_b.data_ptr(), bad_i.data_ptr(), n,
                                  torch.zeros_like(dy).data_ptr(), t, N, h.data_ptr(), s) == 0
        assert pq.stream_status() == pq._lib.SQ_ERR_RANGE
        assert torch.equal(h, hidden) and (h[rows] == 0).all()
        h[rows] = nan
        assert lib.sq_adapter_backward(dy.data_ptr(), t, M, N, x.data_ptr(), t, K, h.data_ptr(), c, bad_b.data_ptr(),
                                       bad_i.data_ptr(), n, dx.data_ptr(), K, da.data_ptr(), db.data_ptr(),
                                       ws.data_ptr(), wn, s) == 0
        assert pq.stream_status() == pq._lib.SQ_ERR_RANGE
        assert (dx[rows] == 0).all()
        assert torch.equal(dx, want[0]) and torch.equal(da, want[1]) and torch.equal(db, want[2])


@pytest.mark.parametrize("dtype", [BF, F32], ids=str)
@pytest.mark.parametrize("M,lengths", [(700, [300, 400]), (24, [9, 15])], ids=["tiles", "few rows"])
def test_fp32_results_are_as_close_as_elementary_fp32(dtype, M, lengths):
    """Root mean square errors of the fp32 results against 64 bits, beside those of fp32 matrix
    products in torch: sums of the same lengths, and h and u rounded at most once more (or
    cut into parts of 2^-24): at most twice.  (A step of the tensor core cuts up to a unit
    where a rounding is off by half of one, so this asks for short chains.)"""
    x, dy, ad, g = make(M, 2048, 1024, 2, 32, dtype, seed=M)
    bounds, idx = requests(lengths, [1, 0])
    y = torch.randn(M, 1024, generator=g, device="cuda")
    (ref, hid), _ = forward64(y, x, ad, bounds, idx)
    dx = torch.zeros(M, 2048, device="cuda")
    plain_y, plain_h = y.clone(), torch.zeros(M, 32, device="cuda")
    plain_a, plain_b = torch.zeros(2, 32, 2048, device="cuda"), torch.zeros(2, 1024, 32, device="cuda")
    for m, l in rows_of(bounds, idx):
        A, B, s = ad.a[l].float(), ad.b[l].float(), ad.scale[l]
        plain_h[m] = x[m].float() @ A.t()
        plain_y[m] += s * (plain_h[m] @ B.t())
        u = s * (dy[m].float() @ B)
        dx[m] = u @ A
        plain_a[l] = u.t() @ x[m].float()
        plain_b[l] = s * (dy[m].float().t() @ plain_h[m])
    got_y, hidden = pq.adapter_add(y, x, ad, bounds, idx, return_hidden=True)
    want, _ = backward64(dy, x, plain_h, ad, bounds, idx)
    got = pq.adapter_backward(dy, x, plain_h, ad, bounds, idx)
    rms = lambda t, r: (t.double() - r).square().mean().sqrt().item()  # noqa: E731
    pairs = [(hidden, plain_h, hid), (got_y, plain_y, ref), (got[1], plain_a, want[1]), (got[2], plain_b, want[2])]
    if dtype == F32:
        pairs.append((got[0], dx, want[0]))
    for k, (t, p, r) in enumerate(pairs):
        assert rms(t, r) <= 2 * rms(p, r), (k, rms(t, r), rms(p, r))


@pytest.mark.parametrize("R", [16, 128])
def test_long_sums_of_one_sign_have_no_bias(R):
    """16384 positive terms a sum.  A chain of 32 matrix steps cut towards zero loses at most
    one unit of its last place (2^-23) a step, of a partial sum that grows evenly:
    2^-23 * 16.5 < 2^-18.9 of the sum; 32 chains added in fp32 are off by 32 * 2^-24 = 2^-19 at
    most: 2^-18 together.  The second product and the row's gradients run in at most 24 steps,
    2^-23 * 12.5 < 2^-19 more (2^-18 with their own roundings)."""
    g = torch.Generator(device="cuda").manual_seed(R)
    pos = lambda *s: (0.5 + torch.rand(*s, generator=g, device="cuda")).to(BF)  # noqa: E731
    M, D, E = 300, 16384, 32
    bounds, idx = requests([130, 170], [1, 0])
    wide, narrow = pos(2, R, D), pos(2, E, R)
    x = pos(M, D)
    y, ad = torch.zeros(M, E, device="cuda"), pq.Adapters(wide, narrow)
    (ref, hid), _ = forward64(y, x, ad, bounds, idx)
    _, hidden = pq.adapter_add(y, x, ad, bounds, idx, return_hidden=True)
    assert ((hidden.double() / hid - 1).abs() <= 2.0 ** -18).all()
    assert ((y.double() / ref - 1).abs() <= 2.0 ** -17).all()
    # u = dy B over the long axis, then da = u^T x
    ad = pq.Adapters(narrow.transpose(1, 2).contiguous(), wide.transpose(1, 2).contiguous())
    dy, x = x, pos(M, E)
    h = x.float() @ narrow[0].float()
    (_, da, db), _ = backward64(dy, x, h, ad, bounds, idx)
    got = pq.adapter_backward(dy, x, h, ad, bounds, idx)
    assert ((got[1].double() / da - 1).abs() <= 2.0 ** -17).all()
    assert ((got[2].double() / db - 1).abs() <= 2.0 ** -18).all()


def test_empty_batches():
    x, y, ad, _ = make(20, 128, 64, 2, 8)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = y.clone()
    _, h = pq.adapter_add(y, x, ad, start, none, return_hidden=True)
    assert torch.equal(y, before) and (h == 0).all()
    dx, da, db = pq.adapter_backward(y, x, h, ad, start, none)
    assert (dx == 0).all() and (da == 0).all() and (db == 0).all()
    pq.adapter_add(y[:0], x[:0], ad, start, none)
    dx, da, db = pq.adapter_backward(y[:0], x[:0], h[:0], ad, start, none)
    assert dx.shape == (0, 128) and (da == 0).all() and (db == 0).all()


def test_graph_replays_with_new_requests():
    x, y, ad, _ = make(400, 256, 320, 3, 16, seed=12)
    plans = [requests([100, 300], [0, 2]), requests([399, 1], [1, 1]), requests([0, 0], [0, 0])]
    bounds, idx = plans[0][0].clone(), plans[0][1].clone()
    y1, ys = y.clone(), torch.empty_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys.copy_(y1)
        _, h = pq.adapter_add(ys, x, ad, bounds, idx, return_hidden=True)
        gr = pq.adapter_backward(y1, x, h, ad, bounds, idx)
    for b, i in plans:
        bounds.copy_(b)
        idx.copy_(i)
        graph.replay()
        want, h2 = pq.adapter_add(y.clone(), x, ad, b, i, return_hidden=True)
        assert torch.equal(ys, want) and torch.equal(h, h2)
        assert all(torch.equal(a, c) for a, c in zip(gr, pq.adapter_backward(y, x, h2, ad, b, i)))


@pytest.mark.parametrize("B,S,C,N,act", [(2, 256, 1152, 1152, "none"), (3, 33, 256, 400, "silu")])
def test_norm_codes_linear_adapters_run(B, S, C, N, act):
    """The run a block makes: norm to codes and bf16 rows, the quantized linear, adapters.
    Each step equals the separate calls bit for bit; the whole is the 64-bit value of the
    layer on the codes plus the term."""
    g = torch.Generator(device="cuda").manual_seed(B)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, gamma, beta = (2 * rn(B, S, C) + 0.5).to(BF), 1 + 0.1 * rn(C), 0.1 * rn(C)
    M, R = B * S, 16
    qw = pq.quantize_weights(0.02 * rn(N, C), (0, C))
    ad = pq.Adapters((rn(2, R, C) / C ** 0.5).to(BF), (rn(2, N, R) / R ** 0.5).to(BF))
    bounds, idx = requests([S] * B, [i % 2 for i in range(B)])
    y16 = pq.group_norm_act(x, 32, gamma, beta, act=act).view(M, C)
    sp, sn = pq.calibrate(y16, (0, C))
    qp, qn, rows = pq.quantize_activations_norm(x, 32, gamma, beta, (0, C), sp, sn, act=act, return_y=True)
    base = pq.linear_from_codes(qp, qn, qw, sp, sn)
    assert torch.equal(base, pq.linear(y16, qw, sp, sn))
    (want, _), (e, _) = forward64(base, rows, ad, bounds, idx)
    check(pq.adapter_add(base, rows, ad, bounds, idx), want, e)
    # base rounded, the sum rounded: two half steps of the layer's 64-bit value
    q = qp.double() + qn.double()
    full = torch.where(q >= 0, q * sp.double(), q * sn.double()) @ (qw.codes.double() * qw.scales[0].double()[:, None]).t()
    (ref, _), (e2, _) = forward64(full, rows, ad, bounds, idx)
    mag = q.abs() @ (qw.codes.double().abs() * qw.scales[0].double()[:, None]).t() * max(sp.item(), sn.item())
    check(base, ref, e2 + e + half_step(BF) * full.abs() + 1e-6 * mag)


def test_other_output_in_a_graph_on_an_explicit_stream():
    """Captured on a stream that is named in the calls, replayed with new requests: bad ones, an
    empty batch and good ones one after the other leave nothing behind."""
    x, y, ad, _ = make(400, 256, 320, 3, 16, BF, F32, seed=13)
    plans = [requests([100, 300], [0, 2]), requests([399, 1], [1, 7]), requests([0, 0], [0, 0]),
             requests([10, 500], [1, 2]), requests([200, 200], [2, 1])]
    bounds, idx = plans[0][0].clone(), plans[0][1].clone()
    out = torch.full((400, 320), float("nan"), device="cuda", dtype=BF)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        _, h = pq.adapter_add(y, x, ad, bounds, idx, return_hidden=True, stream=s, out=out)
        gr = pq.adapter_backward(y, x, h, ad, bounds, idx, stream=s)
    for b, i in plans:
        bounds.copy_(b)
        idx.copy_(i)
        out.fill_(float("nan"))
        graph.replay()
        want, h2 = pq.adapter_add(y, x, ad, b, i, return_hidden=True, out=torch.empty_like(out))
        assert torch.equal(out, want) and torch.equal(h, h2)
        assert all(torch.equal(a, c) for a, c in zip(gr, pq.adapter_backward(y, x, h2, ad, b, i)))
    assert pq.stream_status() == pq._lib.SQ_ERR_RANGE


@pytest.mark.parametrize("S,C,N", [(256, 1152, 1152), (33, 256, 400)])
def test_norm_codes_linear_adapters_run_rounded_once(S, C, N):
    """The run with an fp32 layer output and an output of its own: within one half step of the
    64-bit value.  A rounding's mean square error goes with the mean square of what is
    rounded, so the bf16 layer output adds E[layer^2] / E[sum^2] of the one rounding's; half
    of that has to be gone."""
    g = torch.Generator(device="cuda").manual_seed(S)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, M, R = (2 * rn(2, S, C) + 0.5).to(BF), 2 * S, 16
    qw = pq.quantize_weights(0.05 * rn(N, C), (0, C))
    ad = pq.Adapters((rn(2, R, C) / C ** 0.5).to(BF), (0.3 * rn(2, N, R) / R ** 0.5).to(BF))
    bounds, idx = requests([S, S], [1, 0])
    sp, sn = pq.calibrate(pq.group_norm_act(x, 32).view(M, C), (0, C))
    qp, qn, rows = pq.quantize_activations_norm(x, 32, None, None, (0, C), sp, sn, return_y=True)
    wide = pq.linear_from_codes(qp, qn, qw, sp, sn, out_dtype=F32)
    once = pq.adapter_add(wide, rows, ad, bounds, idx, out=torch.empty(M, N, device="cuda", dtype=BF))
    twice = pq.adapter_add(pq.linear_from_codes(qp, qn, qw, sp, sn), rows, ad, bounds, idx)
    q = qp.double() + qn.double()
    w = qw.codes.double() * qw.scales[0].double()[:, None]
    full = torch.where(q >= 0, q * sp.double(), q * sn.double()) @ w.t()
    (ref, _), _ = forward64(full, rows, ad, bounds, idx)
    _, (e, _) = forward64(full.to(BF), rows, ad, bounds, idx)
    check(once, ref, e + 1e-6 * q.abs() @ w.abs().t() * max(sp.item(), sn.item()))
    one, two = ((t.double() - ref).square().mean().item() for t in (once, twice))
    assert one * (1 + 0.5 * (full.square().mean() / ref.square().mean()).item()) < two


@pytest.mark.parametrize("R", [16, 64, 128])
def test_results_repeat_under_load(R):
    """The same call over and over, other calls in flight around it, gives the same bits:
    sums have a fixed order, and no step overtakes another in the kernels' rings (a slot
    given back while its last rows were still being read showed here)."""
    x, y, ad, g = make(8192, 1152, 768, 4, R, seed=R)
    dy = torch.randn(8192, 768, generator=g, device="cuda").to(BF)
    bounds, idx = requests([256] * 30 + [100, 412], [i % 4 for i in range(32)])
    other = torch.randn_like(y)
    base = y.clone()
    want, hidden = pq.adapter_add(y.clone(), x, ad, bounds, idx, return_hidden=True)
    grads = pq.adapter_backward(dy, x, hidden, ad, bounds, idx)
    for _ in range(40):
        pq.adapter_add(other, x, ad, bounds, idx)
        y.copy_(base)
        _, h = pq.adapter_add(y, x, ad, bounds, idx, return_hidden=True)
        again = pq.adapter_backward(dy, x, h, ad, bounds, idx)
        assert torch.equal(y, want) and torch.equal(h, hidden)
        assert all(torch.equal(a, b) for a, b in zip(again, grads))
    assert pq.stream_status() == 0
