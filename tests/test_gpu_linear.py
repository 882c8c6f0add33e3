"""Dense products with their epilogue on the GPU against their definition in 64 bits, and
their gradients against the formula and differences."""
import math

import pytest
import torch

from combine_moe_route_03_gb300 import api

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
# one truncated binary32 addition, relative to the largest partial sum (2^-23), doubled for
# the products of one instruction being aligned to the largest of them
ADD = 2.0 ** -22
ROWS = [1, 31, 128, 257, 700]
SHAPES = [(8, 8), (64, 72), (264, 520), (520, 136), (1032, 264), (256, 7168), (2304, 512)]


def normal(gen, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def check_close(got, ref, slack, dtype):
    """got lies between the roundings of ref - slack and ref + slack."""
    low, high = (ref - slack).float().to(dtype), (ref + slack).float().to(dtype)
    assert got.dtype == dtype and got.shape == ref.shape
    ok = (got >= low) & (got <= high)
    assert bool(ok.all()), f"{int((~ok).sum())} values off, largest error {float((got.double() - ref).abs().max()):.3g}"


def activate(z, act):
    return {None: lambda: z, "relu": lambda: torch.relu(z), "silu": lambda: z * torch.special.expit(z),
            "gelu": lambda: z * torch.special.ndtr(z)}[act]()


def slope(z, act):
    s = torch.special.expit(z)
    return {None: lambda: torch.ones_like(z), "relu": lambda: (z > 0).double(),
            "silu": lambda: s * (1 + z * torch.special.expit(-z)),
            "gelu": lambda: torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)}[act]()


def terms(red, out):
    """Truncating additions of one sum: all, or of binary32 outputs a part of 512 and the parts'."""
    return red + 8 if out != F32 else min(red, 512) + 8 + red // 512


def reference(x, w, bias, trans, out):
    wd = w.double() if trans else w.double().t()
    z, mag = x.double() @ wd, x.double().abs() @ wd.abs()
    if bias is not None:
        z = z + bias.double()
    return z, terms(x.shape[1], out) * ADD * mag + 2.0 ** -23 * (z.abs() + mag)


def through(z, slack, act, res):
    """The epilogue: a slope of at most 1.13, a few binary32 roundings of z (their exponential
    and error function are within 2^-21 of 1, the largest value of what multiplies z)."""
    y = activate(z, act)
    if act is not None:
        slack = 1.13 * slack + 2.0 ** -20 * z.abs() + 2.0 ** -120
    if res is not None:
        y = y + res.double()
        slack = slack + 2.0 ** -23 * (y.abs() + res.double().abs())
    return y, slack


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("n,k", SHAPES)
def test_linear_matches_its_definition(dev, rows, n, k, trans):
    gen = torch.Generator("cuda").manual_seed(rows + n + k)
    red, cols = (n, k) if trans else (k, n)
    for dtype, out, act, some in ((BF16, BF16, None, 0), (F16, F32, "gelu", 1), (BF16, F32, None, 0), (F16, F16, "silu", 1),
                                  (BF16, BF16, "relu", 1), (BF16, F32, "silu", 1)):
        x, w = normal(gen, rows, red, dtype=dtype), normal(gen, n, k, dtype=dtype, scale=red ** -0.5)
        bias = normal(gen, cols, dtype=F32) if some else None
        z, slack = reference(x, w, bias, trans, out)
        res = normal(gen, rows, cols, dtype=out) if some else None
        whole = torch.full((rows + 3, cols), -7.0, dtype=out, device=dev)
        pre = torch.full((rows + 3, cols), -7.0, dtype=dtype, device=dev) if some else None
        status = api.new_status()
        got = api.linear(x, w, bias=bias, act=act, residual=res, trans=trans, out=whole[:rows],
                         pre=None if pre is None else pre[:rows], status=status)
        assert api.read_status(status) == 0
        y, y_slack = through(z, slack, act, res)
        check_close(got, y, y_slack, out)
        assert bool((whole[rows:] == -7).all())                   # rows behind the last
        if some:
            check_close(pre[:rows], z, slack, dtype)
            assert bool((pre[rows:] == -7).all())
            mine = res.clone()                                     # in place, and the same bits
            assert torch.equal(api.linear(x, w, bias=bias, act=act, residual=mine, trans=trans, out=mine), got)
        else:
            assert torch.equal(api.linear(x, w, act=act, trans=trans, out_dtype=out), got)


@pytest.mark.parametrize("rows,n,k,sms", [(3000, 1544, 200, 0), (3000, 1544, 200, 6), (1100, 520, 72, 2), (8200, 256, 1024, 0),
                                          (200, 6000, 1024, 0), (130, 256, 2048, 40)])
def test_many_tiles_a_pair_and_few_sms(dev, rows, n, k, sms):
    gen = torch.Generator("cuda").manual_seed(rows)
    x, w, res = normal(gen, rows, k), normal(gen, n, k, scale=k ** -0.5), normal(gen, rows, n)
    for out in (BF16, F32):
        z, slack = reference(x, w, None, False, out)
        y, slack = through(z, slack, "silu", res.to(out))
        check_close(api.linear(x, w, act="silu", residual=res.to(out), num_sms_=sms, out_dtype=out), y, slack, out)


@pytest.mark.parametrize("dtype,red", [(F16, 16384 + 72), (BF16, 131072 + 8)])
@pytest.mark.parametrize("rows", [3, 300])
def test_long_sums(dev, dtype, red, rows):
    """Sums that are joined from parts of 4096 terms: positive terms, whose truncations add up."""
    gen = torch.Generator("cuda").manual_seed(rows)
    x, w = normal(gen, rows, red, dtype=dtype).abs(), (normal(gen, 40, red, dtype=dtype).abs() * red ** -0.5).to(dtype)
    z, mag = x.double() @ w.double().t(), x.double() @ w.double().t()
    for out in (dtype, F32):
        part = 512 if out == F32 else 4096
        check_close(api.linear(x, w, out_dtype=out), z, mag * ((part + 8) * ADD + (red // part + 8) * 2.0 ** -24), out)


def test_infinities_and_nan_stay_in_their_rows_and_columns(dev):
    gen = torch.Generator("cuda").manual_seed(1)
    x, w = normal(gen, 300, 520), normal(gen, 264, 520)
    x[5, 7], x[299, 519], w[17, 3] = float("nan"), float("inf"), float("nan")
    for rows in (300, 40):
        y = api.linear(x[-rows:], w)
        bad = torch.isnan(x[-rows:]).any(1)
        inf = torch.isinf(x[-rows:]).any(1)
        assert bool(torch.isnan(y[bad]).all()) and bool(torch.isnan(y[:, 17]).all())
        others = y[~bad & ~inf][:, [i for i in range(264) if i != 17]]
        assert bool(torch.isfinite(others).all()) and not bool(torch.isfinite(y[inf]).any())


def test_activations_at_their_ends(dev):
    """z from the bias alone: what is far out, next to zero, infinite or NaN."""
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3.0, -3.0, 30.0, -30.0, -86.0, -88.0, -100.0, 1e4, -1e4, 3e38, -3e38,
                      float("nan")], device=dev)
    x, w = torch.zeros(2, 8, dtype=BF16, device=dev), torch.zeros(16, 8, dtype=BF16, device=dev)
    for act in ("relu", "silu", "gelu"):
        got = api.linear(x, w, bias=z, act=act, out_dtype=F32)[1].double()
        want = activate(z.double(), act)
        assert bool(torch.isnan(got[-1]))
        err = (got[:-1] - want[:-1]).abs()
        # silu's product with a quick exponential (its argument's rounding, 100 2^-24, besides);
        # gelu's 1 + erf, a difference on the left
        assert bool((err <= want[:-1].abs() * 2.0 ** -16 + (z[:-1].double().abs().clamp(max=6) * 2.0 ** -23 if act == "gelu" else 2.0 ** -120)).all())


@pytest.mark.parametrize("act", [None, "relu", "gelu", "silu"])
@pytest.mark.parametrize("rows,n,k,dtype", [(1, 8, 8, BF16), (33, 264, 136, F16), (300, 520, 264, BF16), (77, 1000, 1544, F16)])
def test_gradients_match_the_formula(dev, rows, n, k, dtype, act):
    gen = torch.Generator("cuda").manual_seed(rows + n)
    x, w, dy = normal(gen, rows, k, dtype=dtype), normal(gen, n, k, dtype=dtype, scale=n ** -0.5), normal(gen, rows, n, dtype=dtype)
    pre, add = normal(gen, rows, n, dtype=dtype, scale=2.0), normal(gen, rows, k, dtype=dtype)
    pre[0, 0] = 0
    dz = dy.double() * slope(pre.double(), act)
    # binary32 of slopes up to 1.13 whose parts are within 2^-20; then rounded to the type
    z_slack = dy.double().abs() * 2.0 ** -20
    got = api.linear_backward(dy, x, w, act=act, z=None if act is None else pre, add=add, bias=True)
    rounded = z_slack + (0 if act is None else HALF[dtype] * dz.abs() * (1 + 2.0 ** -9) + 2.0 ** -25)
    dx = dz @ w.double() + add.double()
    check_close(got["dx"], dx, rounded @ w.double().abs() + (n + 8) * ADD * (dz.abs() @ w.double().abs()) + 2.0 ** -22 * dx.abs(), dtype)
    dw = dz.t() @ x.double()
    w_slack = rounded.t() @ x.double().abs() + (rows + 8) * ADD * (dz.abs().t() @ x.double().abs())
    check_close(got["dw"], dw, w_slack, dtype)
    b_slack = (z_slack + dz.abs() * rows * 2.0 ** -24).sum(0) + 2.0 ** -30
    assert got["dbias"].dtype == F32 and bool(((got["dbias"].double() - dz.sum(0)).abs() <= b_slack).all())
    # added to binary32 gradients of an earlier micro-batch; nothing asked for the bias
    first = normal(gen, n, k, dtype=F32)
    acc, db = first.clone(), torch.ones(n, device=dev)
    more = api.linear_backward(dy, x, w, act=act, z=pre, bias=True, dw=acc, dbias=db, accumulate=True)
    assert more["dw"] is acc
    assert bool(((acc.double() - first.double() - dw).abs() <= w_slack + 2.0 ** -22 * (first.abs() + dw.abs())).all())
    assert bool(((db.double() - 1 - dz.sum(0)).abs() <= b_slack + 2.0 ** -23 * (1 + dz.sum(0).abs())).all())
    assert api.linear_backward(dy, x, w, act=act, z=pre)["dbias"] is None
    odd = torch.empty(rows * n + 1, dtype=dtype, device=dev)[1:].view(rows, n).copy_(dy)   # off 16 bytes
    z1, b1 = api.act_backward(odd, pre, act)
    if act is not None:
        z2, b2 = api.act_backward(dy, pre, act)
        assert torch.equal(z1, z2)
        mine = dy.clone()
        assert api.act_backward(mine, pre, act, dz=mine, dbias=False)[1] is None and torch.equal(mine, z2)
    assert bool(((b1.double() - dz.sum(0)).abs() <= b_slack).all())


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_gradients_match_differences(dev, act):
    gen = torch.Generator("cuda").manual_seed(2)
    x, w, dy, bias = normal(gen, 40, 72), normal(gen, 64, 72, scale=0.1), normal(gen, 40, 64), normal(gen, 64, dtype=F32)
    pre = torch.empty(40, 64, dtype=BF16, device=dev)
    api.linear(x, w, bias=bias, act=act, pre=pre)
    got = api.linear_backward(dy, x, w, act=act, z=pre, bias=True)
    f = lambda x, w, b: (activate(x @ w.t() + b, act) * dy.double()).sum()  # noqa: E731
    xd, wd, bd, t = x.double(), w.double(), bias.double(), 1e-5
    for i, (name, at) in enumerate((("dx", xd), ("dw", wd), ("dbias", bd))):
        v = torch.randn(at.shape, generator=gen, device=dev, dtype=torch.float64)
        args = [[xd, wd, bd], [xd, wd, bd]]
        args[0][i], args[1][i] = at + t * v, at - t * v
        want = (f(*args[0]) - f(*args[1])) / (2 * t)
        # the kept z, dz and the result are each rounded to bf16 (2^-8): z by 2^-8 |z| < 2^-6
        # changes a slope by as much, against slopes of 1; all of them one way
        size = {"dx": dy.double().abs() @ wd.abs(), "dw": dy.double().abs().t() @ xd.abs(), "dbias": dy.double().abs().sum(0)}[name]
        assert abs(float((got[name].double() * v).sum() - want)) <= float((size * v.abs()).sum()) * (2.0 ** -6 + 2 * 2.0 ** -8)


def test_empty_batches(dev):
    x, w = torch.empty(0, 64, dtype=BF16, device=dev), torch.ones(32, 64, dtype=BF16, device=dev)
    assert api.linear(x, w, out_dtype=F32).shape == (0, 32)
    dy = torch.empty(0, 32, dtype=BF16, device=dev)
    got = api.linear_backward(dy, x, w, act="relu", z=dy, bias=True)
    assert got["dx"].shape == (0, 64) and not bool(got["dw"].any()) and not bool(got["dbias"].any())
    db = torch.ones(32, device=dev)
    api.act_backward(dy, dy, "silu", dbias=db, accumulate=True)
    assert bool((db == 1).all())


def test_rows_far_into_memory(dev):
    """Offsets past 2^31 values, of the operand and of the output."""
    rows, n, k = 300_000, 7680, 512
    x = torch.zeros(rows, k, dtype=BF16, device=dev)
    gen = torch.Generator("cuda").manual_seed(1)
    x[-5:] = normal(gen, 5, k)
    w = normal(gen, n, k, scale=k ** -0.5)
    z, slack = reference(x[-5:], w, None, False, BF16)
    y = api.linear(x, w)
    check_close(y[-5:], z, slack, BF16)
    assert not bool(y[:-5].any())
    z, slack = reference(y[-5:], w, None, True, BF16)
    check_close(api.linear(y, w, trans=True)[-5:], z, slack, BF16)
    dz, db = api.act_backward(y, y, "relu")
    assert torch.equal(dz[-5:], torch.relu(y[-5:])) and bool(((db - torch.relu(y[-5:].float()).sum(0)).abs() <= 2e-5 * db.abs()).all())


def test_two_streams_and_graphs(dev):
    gen = torch.Generator("cuda").manual_seed(2)
    x, w, dy, bias = normal(gen, 128, 2048), normal(gen, 512, 2048, scale=0.02), normal(gen, 128, 512), normal(gen, 512, dtype=F32)
    pre = torch.empty(128, 512, dtype=BF16, device=dev)
    want = api.linear(x, w, bias=bias, act="gelu", pre=pre)
    grads = api.linear_backward(dy, x, w, act="gelu", z=pre, bias=True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:                                          # two calls at once
            got.append((api.linear(x, w, bias=bias, act="gelu", stream=s),
                        api.linear_backward(dy, x, w, act="gelu", z=pre, bias=True, stream=s)))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for y, g in got:
        assert torch.equal(y, want) and all(torch.equal(g[n], grads[n]) for n in g)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = api.linear(x, w, bias=bias, act="gelu", pre=pre)
            outs.append((y, api.linear_backward(dy, x, w, act="gelu", z=pre, bias=True)))
        graphs.append(g)
    x.copy_(normal(gen, 128, 2048))
    for g in graphs:
        g.replay()
    want = api.linear(x, w, bias=bias, act="gelu", pre=pre)
    grads = api.linear_backward(dy, x, w, act="gelu", z=pre, bias=True)
    for y, g in outs:
        assert torch.equal(y, want) and all(torch.equal(g[n], grads[n]) for n in g)


def phi(z):
    """The normal distribution function by erfc, which keeps its digits on the left."""
    return torch.special.erfc(z * -math.sqrt(0.5)) / 2


def normal_distribution_bound(z):
    """The distribution function's error relative to its value: a quotient and an exponential
    within 2^-22 (of the quotient's error up to twice arrives), the exponential's argument z^2 / 2
    in binary32 (2^-23 of 0.6 z^2), 5 roundings, and the fit's 2^-26."""
    return 1.15 * 2.0 ** -20 * (1 + z * z / 8)


def test_gelu_and_its_slope_against_64_bits(dev):
    """z from the bias alone, so exact in binary32: on the left, where the distribution function is
    next to nothing, as near to it as elsewhere."""
    z = torch.cat([torch.linspace(-13, 13, 1 << 17, device=dev), torch.linspace(-0.01, 0.01, 1 << 12, device=dev)])
    x, w = torch.zeros(1, 8, dtype=BF16, device=dev), torch.zeros(z.numel(), 8, dtype=BF16, device=dev)
    got = api.linear(x, w, bias=z, act="gelu", out_dtype=F32)[0].double()
    zd = z.double()
    want = zd * phi(zd)
    assert bool(((got - want).abs() <= want.abs() * (normal_distribution_bound(zd) + 2.0 ** -24) + 2.0 ** -118).all())
    for dtype in (BF16, F16):
        pre = z.to(dtype)[None]
        _, slope = api.act_backward(torch.ones_like(pre), pre, "gelu")
        zd = pre[0].double()
        cdf, along = phi(zd), zd * torch.exp(-zd * zd / 2) / math.sqrt(2 * math.pi)
        assert bool(((slope.double() - cdf - along).abs() <= (cdf + along.abs()) * normal_distribution_bound(zd) + 2.0 ** -118).all())


def test_more_sms_asked_for_than_there_are(dev):
    """The grid and the units' order go by what the device has, also for millions of columns."""
    gen = torch.Generator("cuda").manual_seed(8)
    x, w = normal(gen, 40, 8), normal(gen, 6_100_000, 8)
    want = api.linear(x, w)
    assert torch.equal(api.linear(x, w, num_sms_=2 ** 31 - 1), want)
    z, slack = reference(x, w[-300:], None, False, BF16)
    check_close(want[:, -300:].contiguous(), z, slack, BF16)


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,n,k,trans", [(128, 256, 7168, False), (1, 4096, 7168, False), (2500, 264, 7168, False),
                                            (8192, 256, 7168, False), (128, 7168, 256, True), (1500, 7168, 520, True)])
def test_binary32_outputs_hold_more_than_16_bits(dev, rows, n, k, trans, dtype):
    """Relative 2-norm of the error of sums of 7168 random terms, split over a cluster or not.  An
    instruction adds 16 products and drops what is below the last of the sum's 24 bits, 0.36 2^-23 of the
    sum on average, towards zero.  For terms of size 1 the 32 drops of a partial sum of 512 add up to at
    most 0.36 2^-23 sum_j 4 sqrt(j) = 2.1e-5, those of 14 partial sums, of either sign, to 7.8e-5 of
    84.7, 9.2e-7; the roundings of 14 additions to less than 1e-7 of it in squares.  One sum of all 448
    instructions would lose 11 times as much, an output rounded to 16 bits 200 times."""
    gen = torch.Generator("cuda").manual_seed(rows)
    red = n if trans else k
    x, w = normal(gen, rows, red, dtype=dtype), normal(gen, n, k, dtype=dtype, scale=red ** -0.5)
    got = api.linear(x, w, trans=trans, out_dtype=F32)
    assert off(got, x.double() @ (w.double() if trans else w.double().t())) <= 1e-6


@pytest.mark.parametrize("dtype,red", [(F16, 16384 + 72), (BF16, 131072 + 8)])
@pytest.mark.parametrize("rows", [3, 300])
def test_long_sums_of_positive_terms(dev, dtype, red, rows):
    """Truncations of positive terms all add up.  Binary32 outputs: in a part of 512 terms 32
    truncations of at most 2^-22 of a sum that grows evenly, and a rounding (2^-24) a joined
    part of a sum that does: below what one sum of all terms loses, 0.18 2^-23 of it an
    instruction.  16-bit outputs, four times as long: parts of 4096 terms, seen in the mean over many
    outputs, whose own roundings cancel there."""
    gen = torch.Generator("cuda").manual_seed(rows)
    make = lambda r: (normal(gen, rows, r, dtype=dtype).abs(), (normal(gen, 40, r, dtype=dtype).abs() * r ** -0.5).to(dtype))  # noqa: E731
    x, w = make(red)
    z = x.double() @ w.double().t()
    bound = 17 * 2.0 ** -22 + (red // 512 + 2) / 2 * 2.0 ** -24
    assert bound < 0.18 * 2.0 ** -23 * red / 16
    assert bool(((api.linear(x, w, out_dtype=F32).double() - z).abs() <= z * bound).all())
    x, w = make(4 * red)
    z = x.double() @ w.double().t()
    half = 2.0 ** -11 if dtype == F16 else 2.0 ** -8
    bound = 129 * 2.0 ** -22 + 5 * half / (3 * z.numel()) ** 0.5 + (red // 1024 + 2) / 2 * 2.0 ** -24
    if rows == 300:
        assert bound < 0.18 * 2.0 ** -23 * red / 4
    assert abs(float((api.linear(x, w).double() / z - 1).mean())) <= bound
