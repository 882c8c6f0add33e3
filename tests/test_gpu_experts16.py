"""Experts in 16-bit storage on the GPU: grouped products and their weight gradient, the
gated activation and its gradient, and the AdamW step, each against its definition in 64
bits (bounds derived from the roundings of the operation) and, for the gradients, against
differences of the 64-bit forward."""
import numpy as np
import pytest
import torch

from combine_moe_route_03_gb300 import _lib, api

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
# one truncated binary32 addition, relative to the largest partial sum (2^-23), doubled for
# the products of one instruction being aligned to the largest of them
ADD = 2.0 ** -22


def starts_of(counts, align=1, cap=0):
    if cap:
        return [e * cap for e in range(len(counts))]
    out, at = [], 0
    for c in counts:
        out.append(at)
        at += -(-c // align) * align
    return out


def rows_of(counts, align=1, cap=0):
    if cap:
        return len(counts) * cap
    return sum(-(-c // align) * align for c in counts)


def normal(gen, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def i32(counts):
    return torch.tensor(counts, dtype=torch.int32, device="cuda")


def check_close(got, ref, slack, dtype):
    """got is the rounding to dtype of some value within slack of ref: rounding keeps the
    order, so it lies between the roundings of ref - slack and ref + slack."""
    low, high = (ref - slack).float().to(dtype), (ref + slack).float().to(dtype)
    assert got.dtype == dtype
    ok = (got >= low) & (got <= high)
    assert bool(ok.all()), f"{int((~ok).sum())} values off, largest error {float((got.double() - ref).abs().max()):.3g}"


COUNTS = {
    "one_row": [1],
    "one_expert": [300],
    "no_rows": [0, 0, 0],
    "empty_between": [0, 5, 0, 0, 130, 1, 0],
    "tile_edges": [127, 128, 129, 255, 256, 257, 0, 512, 513],
    "steps_of_16": [15, 16, 17, 31, 32, 33, 63, 64, 65],
    "one_popular": [3, 1, 1400, 0, 2, 7],
}
SHAPES = [(8, 8), (64, 72), (264, 520), (520, 136), (1032, 264)]


def gemm_reference(x, w, counts, starts, trans):
    """{expert: (rows, product, product of magnitudes)} in 64 bits."""
    for e, (c, s) in enumerate(zip(counts, starts)):
        if c:
            wd = w[e].double() if trans else w[e].double().t()
            xd = x[s:s + c].double()
            yield s, c, xd @ wd, xd.abs() @ wd.abs()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("pattern", sorted(COUNTS))
@pytest.mark.parametrize("n,k", SHAPES)
def test_grouped_gemm_matches_its_definition(dev, pattern, n, k, trans):
    counts = COUNTS[pattern]
    gen = torch.Generator("cuda").manual_seed(len(pattern) + n + k)
    for align, dtype in ((1, BF16), (128, F16)):
        rows, starts = max(1, rows_of(counts, align)) + 3, starts_of(counts, align)
        red, cols = (n, k) if trans else (k, n)
        x = torch.full((rows, red), float("nan"), dtype=dtype, device=dev)  # padding: NaN
        for c, s in zip(counts, starts):
            x[s:s + c] = normal(gen, c, red, dtype=dtype)
        w = normal(gen, len(counts), n, k, dtype=dtype, scale=red ** -0.5)
        out = torch.full((rows, cols), -7.0, dtype=dtype, device=dev)
        status = api.new_status()
        got = api.grouped_gemm(x, w, i32(counts), trans=trans, align=align, out=out, status=status)
        assert got is out and api.read_status(status) == 0
        keep = torch.ones(rows, dtype=torch.bool, device=dev)
        for s, c, ref, mag in gemm_reference(x, w, counts, starts, trans):
            check_close(out[s:s + c], ref, (red + 8) * ADD * mag, dtype)
            keep[s:s + c] = False
        assert bool((out[keep] == -7.0).all())               # rows of no segment
        again = api.grouped_gemm(x, w, i32(counts), trans=trans, align=align)
        assert torch.equal(again[~keep], out[~keep])         # the same bits


@pytest.mark.parametrize("trans", [False, True])
def test_grouped_gemm_masked_layout_and_device_found_errors(dev, trans):
    """Slots of `cap` rows; a count above cap, a negative one, and a segment that passes the
    buffer are cut and reported, and nothing outside is written."""
    gen = torch.Generator("cuda").manual_seed(5)
    n, k, cap = 136, 264, 70
    red, cols = (n, k) if trans else (k, n)
    w = normal(gen, 4, n, k, scale=0.1)
    x = normal(gen, 4 * cap, red)
    for counts, cut, bits in (([70, 0, 3, 69], [70, 0, 3, 69], 0),
                              ([71, 5, 1000, 1], [70, 5, 70, 1], _lib.STATUS_CAPACITY),
                              ([7, -5, 1, 1], [7, 0, 1, 1], _lib.STATUS_BAD_INDEX)):
        out = torch.full((4 * cap, cols), -7.0, dtype=BF16, device=dev)
        status = api.new_status()
        api.grouped_gemm(x, w, i32(counts), trans=trans, cap=cap, out=out, status=status)
        assert api.read_status(status) == bits
        for e in range(4):
            lo, hi = e * cap, e * cap + cut[e]
            if cut[e]:
                wd = w[e].double() if trans else w[e].double().t()
                xd = x[lo:hi].double()
                check_close(out[lo:hi], xd @ wd, (red + 8) * ADD * (xd.abs() @ wd.abs()), BF16)
            assert bool((out[hi:(e + 1) * cap] == -7.0).all())
    # packed rows that pass the buffer, and sums that pass 31 bits
    for counts, cut in (([100, 150, 100], [100, 150, 30]),
                        ([100, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], [100, 180, 0, 0])):
        out = torch.full((280, cols), -7.0, dtype=BF16, device=dev)
        status = api.new_status()
        api.grouped_gemm(x[:280], w[:len(counts)].contiguous(), i32(counts), trans=trans, out=out, status=status)
        assert api.read_status(status) == _lib.STATUS_CAPACITY
        for s, c, ref, mag in gemm_reference(x, w, cut, starts_of(cut), trans):
            check_close(out[s:s + c], ref, (red + 8) * ADD * mag, BF16)
        assert not bool((out == -7.0).all(dim=1).any())


@pytest.mark.parametrize("trans", [False, True])
def test_grouped_gemm_keeps_infinities_and_nan_to_their_rows(dev, trans):
    counts, n, k = [40, 37, 90], 72, 200
    gen = torch.Generator("cuda").manual_seed(9)
    red = n if trans else k
    x = normal(gen, sum(counts), red)
    w = normal(gen, 3, n, k)
    clean = api.grouped_gemm(x, w, i32(counts), trans=trans)
    bad = x.clone()
    bad[39, 3], bad[40, 0], bad[77, red - 1] = float("inf"), float("nan"), -float("inf")
    out = api.grouped_gemm(bad, w, i32(counts), trans=trans)
    same = torch.ones(sum(counts), dtype=torch.bool, device=dev)
    same[[39, 40, 77]] = False
    assert torch.equal(out[same], clean[same])
    assert not bool(torch.isfinite(out[[39, 40, 77]]).any())
    w[1] = float("nan")                                  # an expert's weights: its rows alone
    out = api.grouped_gemm(x, w, i32(counts), trans=trans)
    assert bool(torch.isnan(out[40:77]).all())
    assert torch.equal(out[:40], clean[:40]) and torch.equal(out[77:], clean[77:])


@pytest.mark.parametrize("out_dtype", [None, F32, "accumulate"])
@pytest.mark.parametrize("pattern", sorted(COUNTS))
@pytest.mark.parametrize("n,k", SHAPES)
def test_grouped_wgrad_matches_its_definition(dev, pattern, n, k, out_dtype):
    counts = COUNTS[pattern]
    gen = torch.Generator("cuda").manual_seed(len(pattern) + n + 3 * k)
    E = len(counts)
    for align, dtype in ((1, F16), (128, BF16)):
        rows, starts = max(1, rows_of(counts, align)), starts_of(counts, align)
        dy = torch.full((rows, n), float("nan"), dtype=dtype, device=dev)   # padding: NaN
        x = torch.full((rows, k), float("inf"), dtype=dtype, device=dev)    # and infinities
        for c, s in zip(counts, starts):
            dy[s:s + c] = normal(gen, c, n, dtype=dtype, scale=0.1)
            x[s:s + c] = normal(gen, c, k, dtype=dtype)
        base = torch.randn(E, n, k, generator=gen, device=dev)
        status = api.new_status()
        if out_dtype == "accumulate":
            got = api.grouped_wgrad(dy, x, i32(counts), align=align, out=base.clone(), accumulate=True, status=status)
            again = api.grouped_wgrad(dy, x, i32(counts), align=align, out=base.clone(), accumulate=True)
        else:
            got = api.grouped_wgrad(dy, x, i32(counts), align=align, out_dtype=out_dtype, status=status)
            again = api.grouped_wgrad(dy, x, i32(counts), align=align, out_dtype=out_dtype)
        assert api.read_status(status) == 0 and torch.equal(got, again)
        assert got.dtype == (dtype if out_dtype is None else F32)
        for e, (c, s) in enumerate(zip(counts, starts)):
            a, b = dy[s:s + c].double(), x[s:s + c].double()
            ref, mag = a.t() @ b, a.abs().t() @ b.abs()
            if out_dtype == "accumulate":
                ref = ref + base[e].double()
                mag = mag + base[e].double().abs()
                if c == 0:
                    assert torch.equal(got[e], base[e])
            adds = c + 8 if out_dtype is None else min(c, 512) + c // 512 + 10
            check_close(got[e], ref, adds * ADD * mag, got.dtype)


def test_wgrad_in_binary32_stays_exact_over_long_segments(dev):
    """20 000 rows of one expert: the relative error of the binary32 gradient stays near
    one addition's (partial sums of 512 rows), not 20 000 truncations of one sign."""
    gen = torch.Generator("cuda").manual_seed(1)
    dy, x = normal(gen, 20000, 128).abs(), normal(gen, 20000, 136).abs()
    got = api.grouped_wgrad(dy, x, i32([20000]), out_dtype=F32)[0].double()
    ref = dy.double().t() @ x.double()
    assert float((got - ref).norm() / ref.norm()) <= (512 / 16 + 20000 / 512) * 2.0 ** -24


@pytest.mark.parametrize("dtype,t", [(F16, 2 ** 21), (BF16, 2 ** 23)])
def test_long_sums_round_once(dev, dtype, t):
    """Sums of one sign over millions of terms: partial sums of 4096 (256 truncating
    instructions) and one addition for each keep the error below the 16-bit rounding, which
    truncation throughout would pass several times."""
    gen = torch.Generator("cuda").manual_seed(24)
    a = normal(gen, t, 8, dtype=dtype, scale=2.0 ** -6).abs()
    b = normal(gen, t, 16, dtype=dtype, scale=2.0 ** -8).abs()
    ref = torch.zeros(8, 16, dtype=torch.float64, device=dev)
    for at in range(0, t, 2 ** 20):
        ref += a[at:at + 2 ** 20].double().t() @ b[at:at + 2 ** 20].double()
    slack = (4096 / 16 + t / 4096 + 8) * ADD * ref
    check_close(api.grouped_wgrad(a, b, i32([t]))[0], ref, slack, dtype)
    at, bt = a.t().contiguous(), b.t().contiguous()          # [8][t], [16][t]
    check_close(api.grouped_gemm(at, bt[None], i32([8])), ref, slack, dtype)
    check_close(api.grouped_gemm(bt, a[None], i32([16]), trans=True), ref.t(), slack.t(), dtype)


@pytest.mark.parametrize("sms", [0, 4])
def test_long_sums_beside_short_ones(dev, sms):
    """Segments (gradient) and contractions (forward, trans) on both sides of the longest sum
    that is not joined, several units a pair, NaN in the padding.  Whole numbers whose sums
    binary32 holds: equality."""
    gen = torch.Generator("cuda").manual_seed(25)

    def whole(*shape):
        return torch.randint(-2, 3, shape, generator=gen, device="cuda").to(F16)
    counts, n, k = [16385, 0, 37, 16384, 20011, 400, 4096, 33000], 520, 328
    starts, rows = starts_of(counts, 64), rows_of(counts, 64)
    dy = torch.full((rows, n), float("nan"), dtype=F16, device=dev)
    x = torch.full((rows, k), float("nan"), dtype=F16, device=dev)
    want = torch.zeros(len(counts), n, k, device=dev)
    for e, (m, s) in enumerate(zip(counts, starts)):
        dy[s:s + m], x[s:s + m] = whole(m, n), whole(m, k)
        want[e] = (dy[s:s + m].double().t() @ x[s:s + m].double()).float()
    for _ in range(3):
        assert torch.equal(api.grouped_wgrad(dy, x, i32(counts), align=64, num_sms_=sms), want.to(F16))
        assert torch.equal(api.grouped_wgrad(dy, x, i32(counts), align=64, out_dtype=F32, num_sms_=sms), want)
    counts = [3, 300, 0, 513, 256, 257]
    for t in (16384, 16392, 20520):
        w, x = whole(len(counts), 264, t), whole(sum(counts), t)
        w2 = w.transpose(1, 2).contiguous()
        want = torch.cat([x[s:s + m].double() @ w[e].double().t()
                          for e, (m, s) in enumerate(zip(counts, starts_of(counts)))]).float().to(F16)
        for _ in range(3):
            assert torch.equal(api.grouped_gemm(x, w, i32(counts), num_sms_=sms), want)
            assert torch.equal(api.grouped_gemm(x, w2, i32(counts), trans=True, num_sms_=sms), want)


def test_wgrad_is_the_gradient_of_the_product(dev):
    """Central differences of L = sum(c * y), y the 64-bit forward, at random weights and
    inputs against grouped_wgrad and grouped_gemm(trans)."""
    counts, n, k = [5, 0, 19], 24, 40
    gen = torch.Generator("cuda").manual_seed(3)
    x, w = normal(gen, 24, k), normal(gen, 3, n, k)
    c = normal(gen, 24, n)
    dw = api.grouped_wgrad(c, x, i32(counts), out_dtype=F32)
    dx = api.grouped_gemm(c, w, i32(counts), trans=True)
    xd, wd, cd = x.double(), w.double(), c.double()

    def loss(xv, wv):
        y = torch.cat([xv[:5] @ wv[0].t(), xv[5:] @ wv[2].t()])
        return float((cd * y).sum())
    rng = np.random.default_rng(0)
    h = 2.0 ** -10                   # the loss is linear in each: no truncation error
    for _ in range(12):
        e, j, i, r = rng.choice([0, 1, 2]), rng.integers(n), rng.integers(k), rng.integers(24)
        wp, wm, xp, xm = wd.clone(), wd.clone(), xd.clone(), xd.clone()
        wp[e, j, i] += h
        wm[e, j, i] -= h
        xp[r, i] += h
        xm[r, i] -= h
        d = (loss(xd, wp) - loss(xd, wm)) / (2 * h)
        assert abs(float(dw[e, j, i]) - d) <= 1e-5 * 24 + 1e-6 * abs(d)
        d = (loss(xp, wd) - loss(xm, wd)) / (2 * h)
        assert abs(float(dx[r, i]) - d) <= 2.0 ** -8 * abs(d) + 1e-4


def test_offsets_past_31_bits(dev):
    """Weights, rows and gradients whose element offsets pass 2^31."""
    gen = torch.Generator("cuda").manual_seed(4)
    E, n, k = 36, 8192, 8192                                  # 2.4e9 weights
    w = torch.zeros(E, n, k, dtype=BF16, device=dev)
    w[E - 1] = normal(gen, n, k, scale=0.01)
    x = normal(gen, 3, k)
    counts = [0] * (E - 1) + [3]
    xd, wd = x.double(), w[E - 1].double()
    y = api.grouped_gemm(x, w, i32(counts))
    check_close(y, xd @ wd.t(), (k + 8) * ADD * (xd.abs() @ wd.abs().t()), BF16)
    y = api.grouped_gemm(x, w, i32(counts), trans=True)
    check_close(y, xd @ wd, (k + 8) * ADD * (xd.abs() @ wd.abs()), BF16)
    dw = api.grouped_wgrad(x, x, i32(counts), out=w)[E - 1]
    check_close(dw, xd.t() @ xd, 11 * ADD * (xd.abs().t() @ xd.abs()), BF16)
    assert not bool(w[:E - 1].any())
    del w, wd, dw, y
    rows, k = 300_000, 8192                                   # 2.5e9 elements of x
    x = torch.zeros(rows, k, dtype=BF16, device=dev)
    x[-5:] = normal(gen, 5, k)
    w = normal(gen, 2, 8, k, scale=0.01)
    counts = [rows - 5, 5]
    xd, wd = x[-5:].double(), w[1].double()
    y = api.grouped_gemm(x, w, i32(counts))
    check_close(y[-5:], xd @ wd.t(), (k + 8) * ADD * (xd.abs() @ wd.abs().t()), BF16)
    assert not bool(y[:-5].any())
    dy = normal(gen, rows, 8)
    dw = api.grouped_wgrad(dy, x, i32(counts), out_dtype=F32)
    dd = dy[-5:].double()
    check_close(dw[1], dd.t() @ xd, 15 * ADD * (dd.abs().t() @ xd.abs()), F32)
    assert not bool(dw[0].any())
    h = api.swiglu(x)
    a = x[-5:].float()
    g, u = a[:, :k // 2].double(), a[:, k // 2:].double()
    check_close(h[-5:], g * torch.sigmoid(g) * u, 64 * ADD * (g * u).abs(), BF16)
    assert not bool(h[:-5].any())


@pytest.mark.parametrize("trans", [False, True])
def test_grouped_gemm_of_the_largest_number_of_rows(dev, trans):
    """One segment with every row of the range, and one behind a few others: whole numbers,
    equality."""
    rows, ends, part = 2 ** 31 - 1 - 1024, 5000, 2 ** 27
    gen = torch.Generator("cuda").manual_seed(23)
    x, out = (torch.empty(rows, 8, dtype=BF16, device=dev) for _ in range(2))
    x.fill_(1.0)
    for s in (slice(0, ends), slice(rows - ends, rows)):
        x[s] = torch.randint(-3, 4, (ends, 8), generator=gen, device=dev).to(BF16)
    w = torch.randint(-3, 4, (3, 8, 8), generator=gen, device=dev).to(BF16)
    for counts in ([rows], [7, 0, rows - 7]):
        status = api.new_status()
        api.grouped_gemm(x, w[:len(counts)], i32(counts), trans=trans, out=out.fill_(-99.0), status=status)
        assert api.read_status(status) == 0
        m = w[len(counts) - 1].float() if trans else w[len(counts) - 1].float().t()
        assert torch.equal(out[7:ends], (x[7:ends].float() @ m).to(BF16))
        assert torch.equal(out[rows - ends:], (x[rows - ends:].float() @ m).to(BF16))
        want = m.sum(0).to(BF16)
        for at in range(ends, rows - ends, part):
            assert bool((out[at:min(at + part, rows - ends)] == want).all())


def test_swiglu_of_the_largest_number_of_rows(dev):
    """The last rows of the range: the step past them does not fit 31 bits."""
    rows, ends = 2 ** 31 - 1 - 1024, 40_000
    gen = torch.Generator("cuda").manual_seed(22)
    gu = torch.zeros(rows, 2, dtype=BF16, device=dev)
    dh = torch.zeros(rows, 1, dtype=BF16, device=dev)
    for part in (slice(0, ends), slice(rows - ends, rows)):
        gu[part], dh[part] = normal(gen, ends, 2), normal(gen, ends, 1)
    for counts in (None, i32([5, rows - 70_000, 0, 69_995])):
        h = api.swiglu(gu, counts=counts)
        for part in (slice(0, ends), slice(rows - ends, rows)):
            ref, slack = swiglu_reference(gu[part], None, None)
            check_close(h[part], ref, slack, BF16)
        assert not bool(h[ends:rows - ends].any())
        del h
        dgu, _ = api.swiglu_backward(gu, dh, counts=counts)
        for part in (slice(0, ends), slice(rows - ends, rows)):
            ref, slack, _, _ = swiglu_reference(gu[part], dh[part], None)
            check_close(dgu[part], ref, slack, BF16)
        assert not bool(dgu[ends:rows - ends].any())
        del dgu


def test_largest_number_of_experts(dev):
    gen = torch.Generator("cuda").manual_seed(6)
    E, n, k = 1024, 16, 24
    counts = torch.randint(0, 6, (E,), generator=torch.Generator().manual_seed(2)).tolist()
    rows = sum(counts)
    x, w, dy = normal(gen, rows, k), normal(gen, E, n, k), normal(gen, rows, n)
    which = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).to(dev)
    wd = w.double()[which]
    y = api.grouped_gemm(x, w, i32(counts))
    check_close(y, torch.einsum("rk,rnk->rn", x.double(), wd), (k + 8) * ADD * torch.einsum("rk,rnk->rn", x.double().abs(), wd.abs()), BF16)
    dw = api.grouped_wgrad(dy, x, i32(counts), out_dtype=F32)
    ref = torch.zeros(E, n, k, dtype=torch.float64, device=dev)
    ref.index_add_(0, which, dy.double()[:, :, None] * x.double()[:, None, :])
    mag = torch.zeros_like(ref).index_add_(0, which, (dy.double()[:, :, None] * x.double()[:, None, :]).abs())
    check_close(dw, ref, 16 * ADD * mag, F32)


@pytest.mark.parametrize("sms", [1, 2, 3, 7])
def test_grouped_products_on_few_sms(dev, sms):
    """The grid's size changes nothing in the result."""
    gen = torch.Generator("cuda").manual_seed(8)
    counts, n, k = [300, 0, 17, 600], 264, 520
    x, w, dy = normal(gen, 917, k), normal(gen, 4, n, k), normal(gen, 917, n)
    assert torch.equal(api.grouped_gemm(x, w, i32(counts), num_sms_=sms), api.grouped_gemm(x, w, i32(counts)))
    assert torch.equal(api.grouped_wgrad(dy, x, i32(counts), num_sms_=sms), api.grouped_wgrad(dy, x, i32(counts)))


# ------------------------------------------------------------- gated activation
def swiglu_reference(gu, dh, w):
    I = gu.shape[1] // 2
    g, u = gu[:, :I].double(), gu[:, I:].double()
    w = torch.ones(gu.shape[0], dtype=torch.float64, device=gu.device) if w is None else w.double()
    w = w[:, None]
    s = torch.sigmoid(g)
    a = g * s
    h = w * a * u
    if dh is None:
        return h, (g.abs() + 16) * ADD * h.abs()
    d = dh.double()
    dgu = torch.cat((w * d * u * (s + a * torch.sigmoid(-g)), w * d * a), dim=1)
    slack = torch.cat(((w * d * u).abs() * (g.abs() + 16) * ADD * (s + a.abs()),
                       (w * d * a).abs() * (g.abs() + 16) * ADD), dim=1)
    terms = d * a * u
    return dgu, slack, terms.sum(1), ((g.abs() + 16) * ADD * terms.abs()).sum(1) + (I + 64) * ADD / 2 * terms.abs().sum(1)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,I", [(1, 1), (1, 8), (3, 7), (5, 257), (300, 264), (129, 2048), (7000, 520), (2500, 33)])
def test_swiglu_and_its_gradient_match_their_definition(dev, rows, I, dtype):
    gen = torch.Generator("cuda").manual_seed(rows + I)
    gu = normal(gen, rows, 2 * I, dtype=dtype, scale=3.0)
    dh = normal(gen, rows, I, dtype=dtype)
    w = torch.rand(rows, generator=gen, device=dev) * 3
    for row_w in (None, w):
        h, slack = swiglu_reference(gu, None, row_w)
        check_close(api.swiglu(gu, row_w=row_w), h, slack, dtype)
        ref, slack, rw, rw_slack = swiglu_reference(gu, dh, row_w)
        drow = torch.empty(rows, device=dev)
        dgu, got = api.swiglu_backward(gu, dh, row_w=row_w, drow_w=drow)
        assert got is drow
        check_close(dgu, ref, slack, dtype)
        check_close(drow, rw, rw_slack, F32)
        dgu2, drow2 = api.swiglu_backward(gu, dh, row_w=row_w, drow_w=torch.empty(rows, device=dev))
        assert torch.equal(dgu, dgu2) and torch.equal(drow, drow2)
        inplace = gu.clone()
        api.swiglu_backward(inplace, dh, row_w=row_w, dgu=inplace)
        assert torch.equal(inplace, dgu)
    assert api.swiglu_backward(gu, dh)[1] is None


@pytest.mark.parametrize("align,cap", [(1, 0), (128, 0), (1, 40)])
@pytest.mark.parametrize("I", [40, 37])
def test_swiglu_over_segments_leaves_padding_alone(dev, align, cap, I):
    counts = [0, 5, 33, 0, 1, 40, 0]
    rows, starts = rows_of(counts, align, cap) + 2, starts_of(counts, align, cap)
    gen = torch.Generator("cuda").manual_seed(I)
    live = torch.zeros(rows, dtype=torch.bool, device=dev)
    for c, s in zip(counts, starts):
        live[s:s + c] = True
    gu, dh = normal(gen, rows, 2 * I), normal(gen, rows, I)
    w = torch.rand(rows, generator=gen, device=dev)
    gu[~live], dh[~live], w[~live] = float("nan"), float("nan"), float("nan")
    h = torch.full((rows, I), -7.0, dtype=BF16, device=dev)
    dgu, drow = torch.full((rows, 2 * I), -7.0, dtype=BF16, device=dev), torch.full((rows,), -7.0, device=dev)
    st = api.new_status()
    kw = dict(row_w=w, counts=i32(counts), align=align, cap=cap, status=st)
    api.swiglu(gu, out=h, **kw)
    api.swiglu_backward(gu, dh, dgu=dgu, drow_w=drow, **kw)
    assert api.read_status(st) == 0
    for t in (h, dgu, drow):
        assert bool((t[~live] == -7.0).all())
    ref, slack = swiglu_reference(gu[live], None, w[live])
    check_close(h[live], ref, slack, BF16)
    ref, slack, rw, rw_slack = swiglu_reference(gu[live], dh[live], w[live])
    check_close(dgu[live], ref, slack, BF16)
    check_close(drow[live], rw, rw_slack, F32)


def test_swiglu_of_unaligned_tensors_and_extreme_gates(dev):
    """Storage one element off a 16-byte boundary takes the plain path; gates from -inf to
    inf and largest values give what the formula gives in binary32."""
    gen = torch.Generator("cuda").manual_seed(2)
    rows, I = 9, 64
    flat = normal(gen, rows * 2 * I + 1, scale=2.0)
    off = flat[1:].view(rows, 2 * I)
    assert torch.equal(api.swiglu(off), api.swiglu(off.clone()))
    dh = normal(gen, rows * I + 1)[1:].view(rows, I)
    a, b = api.swiglu_backward(off, dh), api.swiglu_backward(off.clone(), dh.clone())
    assert torch.equal(a[0], b[0])
    g = torch.tensor([-1e30, -200.0, -100.0, -88.0, -0.0, 0.0, 88.0, 100.0, 200.0, 1e30], device=dev)
    gu = torch.stack((g, torch.ones_like(g)), 1).to(BF16)      # I = 1
    h = api.swiglu(gu).float()[:, 0]
    want = torch.where(g < -80, torch.zeros_like(g), g.to(BF16).float())
    assert bool(((h - want).abs() <= 1e-30).all())
    d, _ = api.swiglu_backward(gu, torch.ones(10, 1, dtype=BF16, device=dev))
    assert torch.equal(d[:, 0].float(), torch.where(g > 80, 1.0, torch.where(g < -80, 0.0, 0.5)))
    odd = torch.tensor([[float("nan"), 1.0], [1.0, float("nan")], [float("inf"), 1.0], [1.0, -float("inf")]], dtype=BF16, device=dev)
    h = api.swiglu(odd).float()[:, 0]
    assert torch.isnan(h[:2]).all() and h[2] == float("inf") and h[3] == -float("inf")


@pytest.mark.parametrize("I", [1, 64])
def test_swiglu_of_very_negative_gates(dev, I):
    """Gates whose sigmoid is near binary32's smallest values, times an up value and a row
    weight that bring the product back: down to -87 the sigmoid is a normal number, with e^g's
    relative error of about |g| roundings; below, the subnormal's own rounding (2^-150) adds.
    What stays below 2^-100 for such a gate counts as zero."""
    g = -torch.arange(80.0, 100.0, 0.5, device=dev).to(BF16)
    gu = torch.stack((g, torch.full_like(g, 1e30)), 1).repeat_interleave(I, dim=1)
    w = torch.full((len(g),), 3.0, device=dev)
    dh = torch.ones(len(g), I, dtype=BF16, device=dev)
    gd, u = gu[:, :I].double(), gu[:, I:].double()
    s = torch.sigmoid(gd)
    rel = (gd.abs() + 16) * ADD + 2.0 ** -149 / s
    h = 3 * gd * s * u
    check_close(api.swiglu(gu, row_w=w), h, rel * h.abs(), BF16)
    dgu, dw = api.swiglu_backward(gu, dh, row_w=w)
    dg = 3 * u * s * (1 + gd * torch.sigmoid(-gd))
    check_close(dgu[:, :I], dg, rel * 3 * u * s * (1 + gd.abs()), BF16)
    check_close(dgu[:, I:], 3 * gd * s, rel * (3 * gd * s).abs() + 2.0 ** -100, BF16)
    check_close(dw, (gd * s * u).sum(1), ((rel + (I + 64) * ADD / 2) * (gd * s * u).abs()).sum(1), F32)
    h16 = api.swiglu(torch.stack((g, torch.ones_like(g)), 1).to(F16))     # under fp16's range: zero
    assert not bool(h16.any())


def test_errors_of_calls_without_a_status_word_are_kept(dev):
    """Each operator, on the current and on another stream, and inside a graph; sticky until
    cleared."""
    gen = torch.Generator("cuda").manual_seed(27)
    x, w = normal(gen, 12, 16), normal(gen, 2, 24, 16)
    gu, dh, dy = normal(gen, 12, 32), normal(gen, 12, 16), normal(gen, 12, 24)
    torch.cuda.synchronize()
    api.default_status(clear=True)
    side = torch.cuda.Stream()
    for call in (lambda c, **kw: api.grouped_gemm(x, w, c, **kw),
                 lambda c, **kw: api.grouped_wgrad(dy, x, c, **kw),
                 lambda c, **kw: api.swiglu(gu, counts=c, **kw),
                 lambda c, **kw: api.swiglu_backward(gu, dh, counts=c, **kw)):
        for counts, bits in (([5, 7], 0), ([-1, 3], _lib.STATUS_BAD_INDEX), ([9, 9], _lib.STATUS_CAPACITY)):
            for kw in ({}, dict(stream=side)):
                call(i32(counts), **kw)
                torch.cuda.synchronize()
                assert api.default_status() == bits and api.default_status(clear=True) == bits
                assert api.default_status() == 0
        own = api.new_status()
        call(i32([-1, 3]), status=own)
        assert api.read_status(own) == _lib.STATUS_BAD_INDEX and api.default_status() == 0
        c, g = i32([5, 7]), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call(c)
        c.copy_(i32([13, -9]))
        g.replay()
        torch.cuda.synchronize()
        assert api.default_status(clear=True) == _lib.STATUS_CAPACITY | _lib.STATUS_BAD_INDEX


def test_swiglu_gradient_is_the_difference_of_the_forward(dev):
    gen = torch.Generator("cuda").manual_seed(12)
    rows, I = 4, 16
    gu, dh = normal(gen, rows, 2 * I, dtype=F16), normal(gen, rows, I, dtype=F16)
    w = torch.rand(rows, generator=gen, device=dev) + 0.5
    dgu, dw = api.swiglu_backward(gu, dh, row_w=w)
    loss = lambda z, v: float((swiglu_reference(z, None, v)[0] * dh.double()).sum())  # noqa: E731
    z, v, h = gu.double(), w.double(), 1e-5
    for r in range(rows):
        for j in range(0, 2 * I, 5):
            a, b = z.clone(), z.clone()
            a[r, j] += h
            b[r, j] -= h
            d = (loss(a, v) - loss(b, v)) / (2 * h)
            assert abs(float(dgu[r, j]) - d) <= 2.0 ** -11 * abs(d) + 1e-6
        a, b = v.clone(), v.clone()
        a[r] += h
        b[r] -= h
        d = (loss(z, a) - loss(z, b)) / (2 * h)
        assert abs(float(dw[r]) - d) <= 1e-5 * (1 + abs(d))


# ------------------------------------------------------------------------ AdamW
F = np.float32


def np_decode(code, scale, levels):
    q = code.astype(F) * F(1.0 / levels)
    s = np.repeat(scale, 256)[:len(code)]
    return (q * np.abs(q)) * s


def np_encode(x, levels, floor_one=False):
    """Codes by comparison with every bound, and scales, of magnitudes x (finite)."""
    n, sq = len(x), F(levels) * F(levels)
    pad = np.zeros(-(-n // 256) * 256, F)
    pad[:n] = x
    b = pad.reshape(-1, 256)
    s = b.max(1)
    with np.errstate(divide="ignore"):
        inv = np.where(s >= F(2.0 ** -126), F(1) / s, F(0)).astype(F)
    z = (b * inv[:, None]) * sq
    bounds = ((np.arange(1, levels + 1) - 0.5) ** 2).astype(F)
    c = np.searchsorted(bounds, z.reshape(-1), side="right").reshape(b.shape)
    if floor_one:
        c = np.where(b > 0, np.maximum(c, 1), c)
    return c.reshape(-1)[:n], s


class NumpyAdamW:
    """The definition of include/moe.h in binary32 NumPy (moments) and float64 (p)."""

    def __init__(self, p, bits, lr, betas, eps, decay):
        self.p, self.bits, self.h, self.t = p.astype(np.float64), bits, (lr, betas, eps, decay), 0
        n, nb = len(p), -(-len(p) // 256)
        self.m, self.v = np.zeros(n, F), np.zeros(n, F)
        self.codes = [np.zeros(n, np.int64), np.zeros(nb, F), np.zeros(n, np.int64), np.zeros(nb, F)]

    def step(self, g):
        lr, (b1, b2), eps, decay = self.h
        self.t += 1
        if self.bits == 8:
            mc, ms, rc, rs = self.codes
            self.m = np_decode(mc, ms, 127)
            r = np_decode(rc, rs, 255)
            self.v = r * r
        self.m = self.m * F(b1) + g * F(1 - b1)
        self.v = self.v * F(b2) + (g * g) * F(1 - b2)
        m, v = self.m.astype(np.float64), self.v.astype(np.float64)
        self.p *= 1 - lr * decay
        self.p -= lr / (1 - b1 ** self.t) * m / (np.sqrt(v) / np.sqrt(1 - b2 ** self.t) + eps)
        if self.bits == 8:
            c, ms = np_encode(np.abs(self.m), 127)
            rc, rs = np_encode(np.sqrt(self.v), 255, floor_one=True)
            self.codes = [np.where(self.m < 0, -c, c), ms, rc, rs]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("g_dtype,copy_dtype", [(BF16, BF16), (F32, None), (F16, F16), (BF16, F32)])
def test_adamw_matches_its_definition(dev, bits, g_dtype, copy_dtype):
    rng = np.random.default_rng(bits)
    sizes = [1, 255, 256, 257, 5000, 70_001, 0, 512]
    lr, betas, eps, decay = 3e-3, (0.9, 0.98), 1e-8, 0.05
    p0 = [rng.standard_normal(n).astype(F) for n in sizes]
    params = [torch.from_numpy(p.copy()).to(dev) for p in p0]
    copies = None if copy_dtype is None else [torch.empty_like(p, dtype=copy_dtype) for p in params]
    opt = api.AdamW(params, lr=lr, betas=betas, eps=eps, weight_decay=decay, state_bits=bits, copies=copies)
    ref = [NumpyAdamW(p, bits, lr, betas, eps, decay) for p in p0]
    for t in range(4):
        grads = []
        for n, r in zip(sizes, ref):
            g = (rng.standard_normal(n) * 10.0 ** rng.uniform(-6, 0, n)).astype(F)
            if t == 2:
                g[n // 2:] = 0
            gd = torch.from_numpy(g).to(dev).to(g_dtype)
            grads.append(gd)
            r.step(gd.float().cpu().numpy())
        opt.step(grads)
    assert opt.steps == 4
    m, v = (t.cpu().numpy() for t in opt.state())
    for i, (n, o, r) in enumerate(zip(sizes, opt.offsets, ref)):
        if bits == 32:
            assert np.array_equal(m[o:o + n], r.m) and np.array_equal(v[o:o + n], r.v)
        else:
            b, nb = o // 256, -(-n // 256)
            assert np.array_equal(opt.m_code.cpu().numpy()[o:o + n], r.codes[0])
            assert np.array_equal(opt.r_code.cpu().numpy()[o:o + n], r.codes[2])
            assert np.array_equal(opt.m_scale.cpu().numpy()[b:b + nb], r.codes[1])
            assert np.array_equal(opt.r_scale.cpu().numpy()[b:b + nb], r.codes[3])
            assert np.array_equal(m[o:o + n], np_decode(r.codes[0], r.codes[1], 127))
            rr = np_decode(r.codes[2], r.codes[3], 255)
            assert np.array_equal(v[o:o + n], rr * rr)
        # four steps, each with a few roundings of p and of an update of at most
        # lr (1 / (1 - beta1) + decay |p|)
        got = params[i].cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - r.p) <= 4 * 2.0 ** -22 * (np.abs(r.p) + 10 * lr))
        if copies is not None:
            assert torch.equal(copies[i], params[i].to(copy_dtype))
    gap = torch.ones(opt.numel, dtype=torch.bool)              # between the pieces: untouched
    for n, o in zip(sizes, opt.offsets):
        gap[o:o + n] = False
    assert not np.any(m[gap.numpy()]) and not np.any(v[gap.numpy()])


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_unaligned_tensors_equals_aligned(dev, bits):
    """Views at odd offsets of a flat buffer give the bits of aligned tensors, and their
    neighbours in the buffer are not touched."""
    gen = torch.Generator("cuda").manual_seed(1)
    sizes, flat = [700, 1, 3000], torch.randn(4000, generator=gen, device=dev)
    g, cp = normal(gen, 4000), torch.zeros(4000, dtype=BF16, device=dev)
    keep, at, views = flat.clone(), 1, []
    for n in sizes:
        views.append(slice(at, at + n))
        at += n + 2
    aligned = [flat[v].clone() for v in views]
    gal, cal = [g[v].clone() for v in views], [torch.zeros(n, dtype=BF16, device=dev) for n in sizes]
    a = api.AdamW([flat[v] for v in views], state_bits=bits, copies=[cp[v] for v in views])
    b = api.AdamW(aligned, state_bits=bits, copies=cal)
    scale = torch.tensor(0.25, device=dev)
    for _ in range(3):
        a.step([g[v] for v in views], grad_scale=scale)
        b.step([x.clone() for x in gal], grad_scale=scale)
    live = torch.zeros(4000, dtype=torch.bool, device=dev)
    for v, x, c in zip(views, aligned, cal):
        live[v] = True
        assert torch.equal(flat[v], x) and torch.equal(cp[v], c) and torch.equal(c, x.to(BF16))
    assert torch.equal(flat[~live], keep[~live]) and not bool(cp[~live].any())
    for s, t in zip(a.state(), b.state()):
        assert torch.equal(s, t)


def test_adamw_more_tensors_than_one_table(dev):
    """600 tensors: two tables of 256 and one of 88; grad_scale multiplies the gradient."""
    gen = torch.Generator("cuda").manual_seed(7)
    sizes = [1 + 37 * (i % 23) for i in range(600)]
    ps = [torch.randn(n, generator=gen, device=dev) for n in sizes]
    gs = [torch.randn(n, generator=gen, device=dev) for n in sizes]
    one = [p.clone() for p in ps]
    opt = api.AdamW(ps, lr=0.1, weight_decay=0.0, betas=(0.0, 0.0), eps=0.0)
    opt.step(gs, grad_scale=torch.full((1,), -2.0, device=dev))
    for p, q, g in zip(ps, one, gs):
        assert bool(((p - (q + 0.1 * torch.sign(g))).abs() <= 1e-6 * (1 + q.abs())).all())


def test_adamw_8bit_codes_at_the_extremes(dev):
    """Zeros, subnormal blocks, one huge value among small ones, infinities and NaN: the
    codes of include/moe.h, and a second moment above zero never becomes zero."""
    n = 256 * 6
    m, v = np.zeros(n, F), np.zeros(n, F)
    rng = np.random.default_rng(0)
    m[256:512] = rng.standard_normal(256) * 1e-39            # subnormal: held as zeros
    v[256:512] = 1e-44
    m[512:768], v[512:768] = 1e-12, 1e-30
    m[512], v[512] = 1.0, 1.0                                # the others are below half a step
    m[768:1024] = np.concatenate([[3.0], -np.logspace(-6, 0, 255)])
    v[768:1024] = np.logspace(-12, 3, 256)
    m[1024:1280], v[1024:1280] = 1.0, 1.0
    m[1030], v[1031] = np.nan, np.inf
    m[1280:], v[1280:] = rng.standard_normal(256), rng.random(256) * 3e38
    opt = api.AdamW([torch.zeros(n, device=dev)], state_bits=8)
    opt.load_state(torch.from_numpy(m).to(dev), torch.from_numpy(v).to(dev), 5)
    assert opt.steps == 5
    gm, gv = (t.cpu().numpy() for t in opt.state())
    mc, rc = opt.m_code.cpu().numpy(), opt.r_code.cpu().numpy()
    fine = np.r_[0:1024, 1280:n]
    c, s = np_encode(np.abs(m[fine]), 127)
    assert np.array_equal(mc[fine], np.where(m[fine] < 0, -c, c))
    c, s = np_encode(np.sqrt(v[fine]), 255, floor_one=True)
    assert np.array_equal(rc[fine], c)
    assert not gm[:512].any() and not gv[:256].any()
    assert np.all(gv[512:1024] > 0) and np.all(rc[512:768][1:] == 1)
    assert np.isnan(gm[1024:1280]).all() and not np.isfinite(gv[1024:1280]).any()
    # within half a square-law step of the value: |dx| <= (2 q + 1/L) / (2 L) s
    for x, y, lv in ((np.abs(m), np.abs(gm), 127), (np.sqrt(v), np.sqrt(gv), 255)):
        for b in (768, 1280):
            blk, s = slice(b, b + 256), x[b:b + 256].max()
            q = np.sqrt(x[blk].astype(np.float64) / s)
            assert np.all(np.abs(x[blk] - y[blk].astype(np.float64)) <= ((q + 0.5 / lv) / lv + 1.5 / lv ** 2 + 1e-6) * s)


def test_adamw_state_round_trip(dev):
    gen = torch.Generator("cuda").manual_seed(3)
    ps = [torch.randn(1000, generator=gen, device=dev), torch.randn(300, generator=gen, device=dev)]
    for bits in (8, 32):
        a = api.AdamW([p.clone() for p in ps], state_bits=bits)
        for _ in range(3):
            a.step([torch.randn(p.shape, generator=gen, device=dev) for p in ps])
        m, v = a.state()
        b = api.AdamW([p.clone() for p in a.params], state_bits=bits)
        b.load_state(m, v, a.steps)
        for s, t in zip(a.state(), b.state()):
            assert torch.equal(s, t)
        g = [torch.randn(p.shape, generator=gen, device=dev) for p in ps]
        a.step(g)
        b.step(g)
        for s, t in zip(a.params, b.params):
            assert torch.equal(s, t)


# ---------------------------------------------------------------------- streams
def test_operators_on_another_stream(dev):
    """Inputs made on the current stream just before the call, the call on another, the
    inputs dropped right after it."""
    gen = torch.Generator("cuda").manual_seed(11)
    side = torch.cuda.Stream()
    counts, n, k = [700, 0, 1300], 512, 1024
    w = normal(gen, 3, n, k)
    want = got = None
    for where in (None, side):
        torch.cuda.synchronize()
        g2 = torch.Generator("cuda").manual_seed(13)
        x, dh = normal(g2, 2000, k), normal(g2, 2000, n // 2)
        p = torch.randn(100_000, generator=g2, device=dev)
        opt = api.AdamW([p], state_bits=8)
        gu = api.grouped_gemm(x, w, i32(counts), stream=where)
        h = api.swiglu(gu, counts=i32(counts), stream=where)
        dgu, _ = api.swiglu_backward(gu, dh, counts=i32(counts), stream=where)
        dw = api.grouped_wgrad(dgu, x, i32(counts), out_dtype=F32, stream=where)
        opt.step([torch.randn(100_000, generator=g2, device=dev)], stream=where)
        del x, dh
        torch.empty(2000, k, dtype=BF16, device=dev).fill_(float("nan"))
        torch.cuda.synchronize()
        want, got = got, (gu, h, dgu, dw, p, opt.m_code)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_on_another_stream_keeps_what_it_holds(dev, bits):
    """The object and its copy dropped right after a step and a read-out on a stream that is
    still busy: their memory is not handed out before those are done."""
    side, n = torch.cuda.Stream(), 1 << 20
    gen = torch.Generator("cuda").manual_seed(26)
    p0, g = torch.randn(n, generator=gen, device=dev), torch.randn(n, generator=gen, device=dev)
    m0, v0 = torch.randn(n, generator=gen, device=dev), torch.rand(n, generator=gen, device=dev)

    def make(p):
        opt = api.AdamW([p], state_bits=bits, copies=[torch.empty(n, dtype=BF16, device=dev)])
        opt.load_state(m0, v0, 3)
        return opt
    want = p0.clone()
    opt = make(want)
    opt.step([g])
    moments = [t.clone() for t in opt.state()]
    del opt
    sizes = sorted({n, n * 2, n * 4, n // 64})
    torch.cuda.synchronize()
    got, opt = p0.clone(), None
    opt = make(got)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)                       # about 0.1 s
    opt.step([g], stream=side)
    state = opt.state(stream=side)
    held = state if bits == 8 else None
    del opt, state
    used = [torch.full((s,), 0xFF, dtype=torch.uint8, device=dev) for s in sizes for _ in range(4)]
    torch.cuda.synchronize()
    del used
    assert torch.equal(got, want)
    if held is not None:
        for a, b in zip(held, moments):
            assert torch.equal(a, b)


def test_operators_in_a_captured_graph(dev):
    gen = torch.Generator("cuda").manual_seed(17)
    counts, n, k = i32([100, 0, 44]), 128, 256
    x, w = normal(gen, 144, k), normal(gen, 3, n, k)
    out, h, st = torch.empty(144, n, dtype=BF16, device=dev), torch.empty(144, n // 2, dtype=BF16, device=dev), api.new_status()
    api.grouped_gemm(x, w, counts, out=out, status=st)
    api.swiglu(out, counts=counts, out=h, status=st)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        api.grouped_gemm(x, w, counts, out=out, status=st)
        api.swiglu(out, counts=counts, out=h, status=st)
    x.copy_(normal(gen, 144, k))
    counts.copy_(i32([20, 124, 0]))
    g.replay()
    torch.cuda.synchronize()
    want = api.grouped_gemm(x, w, counts)
    assert torch.equal(out, want) and torch.equal(h, api.swiglu(want, counts=counts))


@pytest.mark.parametrize("counts", [[45, 274, 115, 60, 50, 35], [9, 0, 900, 1300],
                                    [319, 320, 321, 384, 385, 448, 449, 513, 0, 769]])
@pytest.mark.parametrize("n,k", [(5792, 1984), (1232, 672), (4288, 376)])
def test_many_units_a_pair_with_partial_tiles_between(dev, counts, n, k):
    """Each CTA pair works through several tiles, whole ones and ones that pass the extents
    by turns, back to back.  Whole numbers whose sums binary32 holds: equality, whatever the
    order of the additions."""
    gen = torch.Generator("cuda").manual_seed(11)
    rows = sum(counts)

    def whole(*shape):
        return torch.randint(-3, 4, shape, generator=gen, device="cuda").to(BF16)

    x, dy, w, c = whole(rows, k), whole(rows, n), whole(len(counts), n, k), i32(counts)
    base = torch.randint(-9, 10, w.shape, generator=gen, device="cuda").to(F32)
    y, dx, dw = [], [], []
    for e, (start, m) in enumerate(zip(starts_of(counts), counts)):
        xe, dye = x[start:start + m].double(), dy[start:start + m].double()
        y.append(xe @ w[e].double().t())
        dx.append(dye @ w[e].double())
        dw.append((dye.t() @ xe).to(F32))
    y, dx, dw = torch.cat(y).to(F32).to(BF16), torch.cat(dx).to(F32).to(BF16), torch.stack(dw)
    acc = base.clone()
    for turn in range(3):
        assert torch.equal(api.grouped_gemm(x, w, c), y)
        assert torch.equal(api.grouped_gemm(dy, w, c, trans=True), dx)
        assert torch.equal(api.grouped_wgrad(dy, x, c), dw.to(BF16))
        assert torch.equal(api.grouped_wgrad(dy, x, c, out_dtype=F32), dw)
        api.grouped_wgrad(dy, x, c, out=acc, accumulate=True)
        assert torch.equal(acc, base + (turn + 1) * dw)


@pytest.mark.parametrize("align", [1, 64])
@pytest.mark.parametrize("n,k", [(1232, 672), (4288, 2056)])
def test_wgrad_keeps_what_follows_a_segment_out(dev, n, k, align):
    """Every number of rows past a segment's last multiple of 16, with the next segment's rows
    (align 1) or NaN (align 64) behind it, tile after tile on every pair.  Whole numbers:
    equality."""
    gen = torch.Generator("cuda").manual_seed(21)
    counts = [i + 16 * (i % 5) for i in range(1, 16)] + [64, 79, 127, 0, 400, 513]
    rows, starts, c = rows_of(counts, align), starts_of(counts, align), i32(counts)
    dy = torch.full((rows, n), float("nan"), dtype=BF16, device=dev)
    x = torch.full((rows, k), float("nan"), dtype=BF16, device=dev)
    want = torch.zeros(len(counts), n, k, device=dev)
    for e, (m, s) in enumerate(zip(counts, starts)):
        dy[s:s + m] = torch.randint(-3, 4, (m, n), generator=gen, device=dev).to(BF16)
        x[s:s + m] = torch.randint(-3, 4, (m, k), generator=gen, device=dev).to(BF16)
        want[e] = (dy[s:s + m].double().t() @ x[s:s + m].double()).float()
    for _ in range(10):
        assert torch.equal(api.grouped_wgrad(dy, x, c, align=align), want.to(BF16))
        assert torch.equal(api.grouped_wgrad(dy, x, c, align=align, out_dtype=F32), want)


@pytest.mark.parametrize("n,k", [(1232, 672), (1096, 264), (264, 1032)])
def test_wgrad_of_several_tiles_a_unit(dev, n, k):
    """One pair, so that a unit takes several Q tiles over the P tiles that it holds: segments of
    one block to six, longer ones in chunks with two accumulators, tails of every kind, a partial
    last Q tile.  Whole numbers: equality."""
    gen = torch.Generator("cuda").manual_seed(28)
    for counts, align in (([65, 319, 320, 321, 384, 385, 449, 513, 769, 1300], 1),
                          ([1300, 1, 0, 383, 400, 64, 63, 7, 777, 128, 129, 192, 255, 256, 0, 5000], 64),
                          ([16, 15, 17, 48, 31, 33, 97, 80, 200, 79, 1, 2, 3, 4, 5, 6], 64)):
        rows, starts = rows_of(counts, align), starts_of(counts, align)
        dy = torch.full((rows, n), float("nan"), dtype=BF16, device=dev)
        x = torch.full((rows, k), float("nan"), dtype=BF16, device=dev)
        want = torch.zeros(len(counts), n, k, device=dev)
        for e, (m, s) in enumerate(zip(counts, starts)):
            dy[s:s + m] = torch.randint(-3, 4, (m, n), generator=gen, device=dev).to(BF16)
            x[s:s + m] = torch.randint(-3, 4, (m, k), generator=gen, device=dev).to(BF16)
            want[e] = (dy[s:s + m].double().t() @ x[s:s + m].double()).float()
        tiles = len(counts) * -(-k // 256) * -(-n // 256)
        for sms in (2, 4, 0):
            assert sms == 0 or tiles // (16 * (sms // 2)) >= (2 if sms == 2 else 1)
            for dtype in (BF16, F16):
                out = torch.full((len(counts), n, k), -7.0, dtype=dtype, device=dev)
                for _ in range(3):
                    got = api.grouped_wgrad(dy.to(dtype), x.to(dtype), i32(counts), align=align, out=out, num_sms_=sms)
                    assert torch.equal(got, want.to(dtype))
            assert torch.equal(api.grouped_wgrad(dy, x, i32(counts), align=align, out_dtype=F32, num_sms_=sms), want)
