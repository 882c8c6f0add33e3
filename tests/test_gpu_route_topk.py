"""Routing from given logits on the GPU against its definition in 64 bits: the choice
exactly, the weights and gradients within their roundings."""
import math

import pytest
import torch

from combine_moe_route_03_gb300 import api, configs

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SOFT, SIG = configs.SOFTMAX, configs.SIGMOID


def config(B, N, K, **kw):
    return configs.MoEConfig("routing", B=B, H=128, N=N, K=K, I=128, **kw)


def choose(cfg, z, bias):
    """One token at a time, Python floats."""
    out = []
    for row in z.double().cpu().tolist():
        fine = [not math.isnan(v) and v != -math.inf for v in row]
        b = [0.0] * cfg.N if bias is None else bias.double().cpu().tolist()
        sig = lambda v: 1 / (1 + math.exp(-v)) if v >= 0 else math.exp(v) / (1 + math.exp(v))  # noqa: E731
        score = [(v if cfg.score_fn == SOFT else sig(v) + d) if f else -math.inf for v, d, f in zip(row, b, fine)]
        order = [(v if f else -math.inf) if bias is None else c for v, c, f in zip(row, score, fine)]
        live = set(range(cfg.N))
        if cfg.n_group > 1:
            size = cfg.N // cfg.n_group
            best = [sum(sorted(score[g * size:(g + 1) * size])[-2:]) for g in range(cfg.n_group)]
            kept = sorted(range(cfg.n_group), key=lambda g: (-best[g], g))[:cfg.topk_group]
            live = {e for g in kept for e in range(g * size, (g + 1) * size)}
        pick = sorted((e for e in live if order[e] != -math.inf), key=lambda e: (-order[e], e))[:cfg.K]
        out.append(pick + [-1] * (cfg.K - len(pick)))
    return torch.tensor(out, dtype=torch.int32, device=z.device).view(-1, cfg.K)


def weights(cfg, z, idx):
    none = idx < 0
    zk = z.gather(1, idx.clamp(min=0).long()).masked_fill(none, -math.inf)
    if cfg.score_fn == SIG:
        s = torch.sigmoid(zk)
        w = s / s.sum(1, keepdim=True) if cfg.renorm else s
    elif cfg.renorm:
        w = torch.softmax(zk, 1)
    else:
        w = torch.exp(zk - torch.logsumexp(z.masked_fill(torch.isnan(z), -math.inf), 1, keepdim=True))
    return (w * cfg.route_scale).masked_fill(none, 0)


# expf and a quotient are within 2^-22 of theirs; a softmax sums up to 512 / 32 of them a lane
# and five times across; renormalising adds another such sum and quotient.
W_REL = 64 * 2.0 ** -24
CONFIGS = [
    dict(N=8, K=2), dict(N=1, K=1), dict(N=33, K=5, renorm=1), dict(N=60, K=4, score_fn=SIG), dict(N=512, K=16, renorm=1),
    dict(N=256, K=8, n_group=8, topk_group=4, score_fn=SIG, renorm=1, route_scale=2.5),
    dict(N=64, K=6, n_group=4, topk_group=2, renorm=1), dict(N=60, K=3, n_group=5, topk_group=1, score_fn=SIG),
    dict(N=64, K=16, n_group=32, topk_group=8), dict(N=510, K=9, n_group=3, topk_group=2, score_fn=SIG, renorm=1),
    dict(N=4, K=4, n_group=2, topk_group=2, score_fn=SIG), dict(N=100, K=7, n_group=10, topk_group=3, renorm=1),
]


def logits(gen, B, N, dtype, masked):
    z = torch.randn(B, N, generator=gen, device="cuda") * 1.5
    if masked:
        z[torch.rand(B, N, generator=gen, device="cuda") < 0.3] = -math.inf
        z[torch.rand(B, N, generator=gen, device="cuda") < 0.1] = math.nan
        z[::7] = -math.inf
        z[3::11, 1:] = -math.inf
    return z.to(dtype)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("kw", CONFIGS, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_choice_weights_and_counts(dev, kw, dtype, masked):
    gen = torch.Generator("cuda").manual_seed(kw["N"])
    for B in (1, 77):
        cfg = config(B, **kw)
        z = logits(gen, B, cfg.N, dtype, masked)
        for bias in [None] + ([torch.randn(cfg.N, generator=gen, device=dev) * 0.1, torch.zeros(cfg.N, device=dev)]
                              if cfg.score_fn == SIG else []):
            got = api.route_topk(cfg, z, bias)
            want = choose(cfg, z, bias)
            assert torch.equal(got["topk_idx"], want)
            ref = weights(cfg, z.double(), want)
            ref = torch.where(want < 0, 0.0, ref)
            assert bool(((got["topk_w"].double() - ref).abs() <= W_REL * ref + 2.0 ** -140).all())
            counts = torch.bincount(want[want >= 0].long(), minlength=cfg.N)
            assert torch.equal(got["counts"].long(), counts)
        other = api.route_topk(cfg, torch.cat([z.view(-1)[:1], z.view(-1)])[1:].view(B, cfg.N), counts=False)
        assert other["counts"] is None and torch.equal(other["topk_idx"], api.route_topk(cfg, z)["topk_idx"])


def test_scores_that_binary32_cannot_tell_apart(dev):
    """Biases that lift many experts to one score, but for what their rounding leaves: gaps
    below 2^-24 decide, among experts and among groups."""
    gen = torch.Generator("cuda").manual_seed(9)
    closest = 1.0
    for kw in (dict(N=64, K=8), dict(N=64, K=8, n_group=8, topk_group=3), dict(N=256, K=8, n_group=8, topk_group=4)):
        z = torch.randn(1, kw["N"], generator=gen, device=dev)
        level = torch.full_like(z, 1.0).double()
        bias = (level - torch.sigmoid(z.double())).float().view(-1)
        cfg = config(40, score_fn=SIG, renorm=1, **kw)
        rows = z.repeat(40, 1)
        rows[1:] += torch.randn(39, kw["N"], generator=gen, device=dev) * 1e-7   # a few bits of the logits
        c = torch.sort(torch.sigmoid(rows.double()) + bias.double(), 1).values
        closest = min(closest, float((c[:, 1:] - c[:, :-1]).min()))
        got = api.route_topk(cfg, rows, bias)
        assert torch.equal(got["topk_idx"], choose(cfg, rows, bias))
    assert closest < 2.0 ** -26


@pytest.mark.parametrize("B", [64, 8300])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("many", [2, 12, 30])
def test_a_few_scores_that_binary32_cannot_tell_apart(dev, many, dtype, B):
    """Some experts at one score, but for the last bits of their biases' rounding, at the border
    of the K best; and groups whose two best are at one score."""
    gen = torch.Generator("cuda").manual_seed(many)
    z = torch.randn(1, 256, generator=gen, device=dev).to(dtype)
    s = torch.sigmoid(z.double()).view(-1)
    level = torch.full((256,), 0.4, dtype=torch.float64, device=dev) - torch.rand(256, generator=gen, device=dev) * 0.3
    level[torch.randperm(256, generator=gen, device=dev)[:many]] = 0.6
    level[7:9], level[250:252] = 0.9, 0.8                     # above them
    bias = (level - s).float()
    rows = z.repeat(B, 1)
    if dtype == F32:
        rows[1:] += torch.randn(B - 1, 256, generator=gen, device=dev) * 1e-7
    for kw in (dict(), dict(n_group=8, topk_group=4)):
        cfg = config(B, N=256, K=8, score_fn=SIG, renorm=1, **kw)
        pick = torch.arange(0, B, max(1, B // 64), device=dev)
        assert torch.equal(api.route_topk(cfg, rows, bias)["topk_idx"][pick], choose(cfg, rows[pick], bias))
    # groups: the two best of each at one score, the rest lower
    level = torch.full((8, 32), 0.3, dtype=torch.float64, device=dev)
    level[:, 3], level[:, 20] = 0.9, 0.7
    level[2, 3], level[5, 20] = 0.95, 0.75
    bias = (level.view(-1) - s).float()
    cfg = config(B, N=256, K=8, n_group=8, topk_group=4, score_fn=SIG, renorm=1)
    assert torch.equal(api.route_topk(cfg, rows, bias)["topk_idx"][pick], choose(cfg, rows[pick], bias))


@pytest.mark.parametrize("kw", [CONFIGS[i] for i in (4, 5, 6, 11)] + [dict(N=64, K=6), dict(N=128, K=12, score_fn=SIG)],
                         ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_many_tokens(dev, kw):
    """The kernels for many tokens: every type, masked experts, ties of 16-bit logits, no bias,
    one of zeros and one that steers."""
    gen = torch.Generator("cuda").manual_seed(kw["N"] + 2)
    for dtype, masked in ((F32, True), (BF16, False), (F16, True)):
        cfg = config(8205, **kw)
        z = logits(gen, cfg.B, cfg.N, dtype, masked)
        pick = torch.cat([torch.arange(0, cfg.B, 61, device=dev), torch.arange(cfg.B - 9, cfg.B, device=dev)])
        for bias in [None] + ([torch.randn(cfg.N, generator=gen, device=dev) * 0.1, torch.zeros(cfg.N, device=dev)]
                              if cfg.score_fn == SIG else []):
            got = api.route_topk(cfg, z, bias)
            want = choose(cfg, z[pick], bias)
            assert torch.equal(got["topk_idx"][pick], want)
            ref = torch.where(want < 0, 0.0, weights(cfg, z[pick].double(), want))
            assert bool(((got["topk_w"][pick].double() - ref).abs() <= W_REL * ref + 2.0 ** -140).all())
            idx = got["topk_idx"]
            assert torch.equal(got["counts"].long(), torch.bincount(idx[idx >= 0].long(), minlength=cfg.N))


@pytest.mark.parametrize("B", [1, 8, 9, 20, 30, 33, 41, 50, 65, 128, 256, 257, 1000])
def test_counts_of_any_batch(dev, B):
    """Over memory that held something else."""
    gen = torch.Generator("cuda").manual_seed(B)
    cfg = config(B, N=200, K=5, renorm=1)
    for _ in range(3):
        junk = torch.full((200,), 12345, dtype=torch.int32, device=dev)
        del junk
        got = api.route_topk(cfg, logits(gen, B, 200, F32, True))
        idx = got["topk_idx"]
        assert torch.equal(got["counts"].long(), torch.bincount(idx[idx >= 0].long(), minlength=200))


def test_equal_scores_go_to_the_lower_index(dev):
    for score in (SOFT, SIG):
        cfg = config(3, N=96, K=5, score_fn=score, renorm=1)
        z = torch.zeros(3, 96, device=dev)
        z[1, 40:60], z[2, ::2] = 1.0, 0.5
        for bias in (None, torch.zeros(96, device=dev)) if score == SIG else (None,):
            got = api.route_topk(cfg, z, bias)["topk_idx"].tolist()
            assert got == [[0, 1, 2, 3, 4], [40, 41, 42, 43, 44], [0, 2, 4, 6, 8]]
        both = api.route_topk(config(3, N=96, K=5, n_group=8, topk_group=2, score_fn=score), z)["topk_idx"].tolist()
        assert both == [[0, 1, 2, 3, 4], [40, 41, 42, 43, 44], [0, 2, 4, 6, 8]]


def test_extreme_logits(dev):
    inf, big = math.inf, 3e38
    z = torch.tensor([[inf, 1.0, inf, -inf], [big, -big, 0.0, big], [-200.0, -100.0, -300.0, -inf], [100.0, 200.0, -inf, 300.0]],
                     device=dev)
    for score, renorm in ((SOFT, 1), (SOFT, 0), (SIG, 1), (SIG, 0)):
        got = api.route_topk(config(4, N=4, K=2, score_fn=score, renorm=renorm), z)
        assert got["topk_idx"].tolist() == [[0, 2], [0, 3], [1, 0], [3, 1]]
        assert bool(torch.isfinite(got["topk_w"]).all())
        grad = api.route_topk_backward(config(4, N=4, K=2, score_fn=score, renorm=renorm), z, got["topk_idx"],
                                       torch.ones(4, 2, device=dev))
        assert bool(torch.isfinite(grad).all())
    assert api.route_topk(config(4, N=4, K=2, renorm=1), z)["topk_w"][0].tolist() == [0.5, 0.5]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (F16, F32), (F32, BF16)])
@pytest.mark.parametrize("kw", CONFIGS, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_gradient_matches_autograd(dev, kw, dtype, out, masked):
    gen = torch.Generator("cuda").manual_seed(kw["N"] + 1)
    cfg = config(77, **kw)
    z = logits(gen, 77, cfg.N, dtype, masked)
    idx = api.route_topk(cfg, z)["topk_idx"]
    dw = torch.randn(77, cfg.K, generator=gen, device=dev)
    zd = z.double().masked_fill(torch.isnan(z), -math.inf).requires_grad_()
    weights(cfg, zd, idx).backward(dw.double().masked_fill(idx < 0, 0.0))
    want = torch.nan_to_num(zd.grad, nan=0.0)
    got = api.route_topk_backward(cfg, z, idx, dw.masked_fill(idx < 0, math.nan), out_dtype=out)
    # relative to the terms that make a value: scale max|dw| (1 + K) of its score, at most 1
    size = cfg.route_scale * dw.abs().amax(1, keepdim=True).double() * (1 + cfg.K)
    half = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}[out]
    assert got.dtype == out
    assert bool(((got.double() - want).abs() <= want.abs() * half + size * W_REL + 2.0 ** -25).all())


def test_gradient_of_repeated_and_foreign_indices(dev):
    """The same expert twice adds both; an index outside the experts adds nothing."""
    gen = torch.Generator("cuda").manual_seed(4)
    for score, renorm in ((SIG, 0), (SOFT, 0)):
        cfg = config(2, N=40, K=4, score_fn=score, renorm=renorm)
        z = torch.randn(2, 40, generator=gen, device=dev)
        idx = torch.tensor([[3, 7, 3, 3], [5, -1, 40, 2 ** 31 - 1]], dtype=torch.int32, device=dev)
        dw = torch.randn(2, 4, generator=gen, device=dev)
        zd = z.double().requires_grad_()
        valid = (idx >= 0) & (idx < 40)
        w = weights(cfg, zd, torch.where(valid, idx, 0)) * valid
        w.backward(dw.double())
        got = api.route_topk_backward(cfg, z, idx, dw)
        assert bool(((got.double() - zd.grad).abs() <= 1e-5).all())


def test_empty_batch_long_batch_other_stream_and_graph(dev):
    cfg = config(0, N=256, K=8, n_group=8, topk_group=4, score_fn=SIG, renorm=1)
    got = api.route_topk(cfg, torch.empty(0, 256, device=dev))
    assert got["topk_idx"].shape == (0, 8) and not bool(got["counts"].any())
    assert api.route_topk_backward(cfg, torch.empty(0, 256, device=dev), got["topk_idx"], got["topk_w"]).shape == (0, 256)
    gen = torch.Generator("cuda").manual_seed(6)
    z, bias = torch.randn(50_001, 256, generator=gen, device=dev), torch.randn(256, generator=gen, device=dev) * 0.1
    whole = api.route_topk(cfg, z, bias)
    part = api.route_topk(cfg, z[-300:], bias)
    assert torch.equal(whole["topk_idx"][-300:], part["topk_idx"]) and torch.equal(whole["topk_w"][-300:], part["topk_w"])
    assert int(whole["counts"].sum()) == 50_001 * 8
    s = torch.cuda.Stream()
    there = api.route_topk(cfg, z, bias, stream=s)
    back = api.route_topk_backward(cfg, z, there["topk_idx"], there["topk_w"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(there["topk_idx"], whole["topk_idx"])
    assert torch.equal(back, api.route_topk_backward(cfg, z, whole["topk_idx"], whole["topk_w"]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = api.route_topk(cfg, z, bias)
        d = api.route_topk_backward(cfg, z, r["topk_idx"], r["topk_w"])
    for _ in range(2):
        z.copy_(torch.randn(50_001, 256, generator=gen, device=dev))
        g.replay()
        want = api.route_topk(cfg, z, bias)
        assert torch.equal(r["topk_idx"], want["topk_idx"]) and torch.equal(r["counts"], want["counts"])
        assert torch.equal(d, api.route_topk_backward(cfg, z, want["topk_idx"], want["topk_w"]))


def test_tokens_far_into_memory(dev):
    """Offsets past 2^31 logits."""
    cfg = config(0, N=512, K=4, renorm=1)
    B = (1 << 31) // 512 + 9
    z = torch.zeros(B, 512, dtype=BF16, device=dev)
    z[-9:] = torch.randn(9, 512, generator=torch.Generator("cuda").manual_seed(1), device=dev).to(BF16)
    got = api.route_topk(cfg, z)
    few = api.route_topk(cfg, z[-9:])
    assert torch.equal(got["topk_idx"][-9:], few["topk_idx"]) and torch.equal(got["topk_w"][-9:], few["topk_w"])
    dw = torch.ones(B, 4, device=dev)
    dw[:, 0] = 2
    grad = api.route_topk_backward(cfg, z, got["topk_idx"], dw)
    assert torch.equal(grad[-9:], api.route_topk_backward(cfg, z[-9:], few["topk_idx"], dw[-9:]))


def test_groups_with_many_equal_or_few_experts(dev):
    """Groups whose experts score alike (more than a lane's list holds), and groups with one
    expert or none left, beside ordinary ones."""
    gen = torch.Generator("cuda").manual_seed(12)
    for dtype, score in ((F32, SIG), (BF16, SIG), (F32, SOFT)):
        for N, G, tg, K in ((256, 8, 4, 8), (512, 8, 2, 4), (128, 4, 4, 3), (256, 2, 1, 2)):
            cfg = config(8200, N=N, K=K, n_group=G, topk_group=tg, score_fn=score, renorm=1)
            z = torch.randn(cfg.B, N, generator=gen, device=dev)
            z[::5] = z[::5].round()                                  # steps of 1: many alike
            z[1::5] = 0.25
            z.view(cfg.B, G, -1)[2::5, :2, 1:] = -math.inf            # one expert left, ...
            z.view(cfg.B, G, -1)[3::5, 1:] = -math.inf                # ... or one group
            z = z.to(dtype)
            bias = torch.randn(N, generator=gen, device=dev) * 0.05 if score == SIG else None
            pick = torch.arange(0, cfg.B, 53, device=dev)
            for b in {id(bias): bias, id(None): None}.values():
                got = api.route_topk(cfg, z, b)
                assert torch.equal(got["topk_idx"][pick], choose(cfg, z[pick], b))
                idx = got["topk_idx"]
                assert torch.equal(got["counts"].long(), torch.bincount(idx[idx >= 0].long(), minlength=N))


@pytest.mark.parametrize("B", [64, 8200])
@pytest.mark.parametrize("K", [1, 2, 3, 5, 9])
def test_logits_that_differ_in_their_last_bits(dev, K, B):
    """A few experts far above the others whose binary32 logits differ in the last bits alone,
    the best of them anywhere; more and fewer than are chosen."""
    gen = torch.Generator("cuda").manual_seed(K)
    for many in (4, 7, 9, 12):
        cfg = config(B, N=64, K=K, renorm=1)
        z = torch.randn(B, 64, generator=gen, device=dev) * 0.1 - 3
        at = torch.rand(B, 64, generator=gen, device=dev).argsort(1)[:, :many].sort(1).values
        z.scatter_(1, at, 1 + torch.rand(B, many, generator=gen, device=dev).argsort(1) * 2.0 ** -23)
        z[1].scatter_(0, at[1], 1 + torch.arange(many, device=dev) * 2.0 ** -23)      # the best one last
        pick = torch.arange(0, B, max(1, B // 64), device=dev)
        pick[1] = 1
        assert torch.equal(api.route_topk(cfg, z)["topk_idx"][pick], choose(cfg, z[pick], None))


@pytest.mark.parametrize("B", [64, 8200])
@pytest.mark.parametrize("K", [1, 2, 3, 8, 9])
def test_close_scores_beside_equal_ones(dev, K, B):
    """A few experts above the others at one score, but for what binary32 cannot tell; some of them
    twice, with one logit and one bias; more and fewer than are chosen."""
    gen = torch.Generator("cuda").manual_seed(K + 20)
    for many in (3, 6, 8, 12):
        cfg = config(B, N=64, K=K, score_fn=SIG, renorm=1)
        z = torch.randn(B, 64, generator=gen, device=dev)
        at = torch.randperm(64, generator=gen, device=dev)[:many].sort().values
        z[:] = z[0]
        level = 0.4 - torch.rand(64, generator=gen, device=dev).double() * 0.3
        level[at] = 0.9
        bias = (level - torch.sigmoid(z[0].double())).float()
        for i in range(0, many - 2, 3):                           # experts like an earlier one
            z[:, at[i + 2]], bias[at[i + 2]] = z[:, at[i]], bias[at[i]]
        z[1::2, at[1]] += torch.randn(B // 2, generator=gen, device=dev) * 1e-7
        pick = torch.arange(0, B, max(1, B // 64), device=dev)
        assert torch.equal(api.route_topk(cfg, z, bias)["topk_idx"][pick], choose(cfg, z[pick], bias))


@pytest.mark.parametrize("B", [5, 8200])
def test_sums_and_biases_past_binary32(dev, B):
    """Groups whose two best logits add up past binary32's range, either way; biases without end."""
    inf = math.inf
    cfg = config(B, N=128, K=3, n_group=4, topk_group=2, renorm=1)
    z = torch.zeros(B, 128, device=dev)
    z[0::5, 5:7], z[0::5, 40:42], z[0::5, 70:72] = 2e38, 3e38, 2.5e38
    z[1::5, :64], z[1::5, 64:96], z[1::5, 96:] = -3e38, -2e38, -inf
    z[2::5, :32], z[2::5, 32:64], z[2::5, 64:] = -inf, -2e38, -3e38
    z[3::5, 7], z[3::5, 100], z[3::5, 101] = 3e38, 2e38, 2e38
    got = api.route_topk(cfg, z)["topk_idx"]
    assert torch.equal(got[:5], choose(cfg, z[:5], None)) and torch.equal(got, got[:5].repeat((B + 4) // 5, 1)[:B])
    z = torch.randn(5, 128, generator=torch.Generator("cuda").manual_seed(2), device=dev).repeat((B + 4) // 5, 1)[:B]
    z[1, 1:32] = -inf
    cfg = config(B, N=128, K=3, n_group=4, topk_group=2, score_fn=SIG, renorm=1)
    for places in ({0: inf}, {0: inf, 40: inf, 41: 3e38, 90: inf, 91: -3e38}, {i: -3e38 for i in range(64)},
                   {i: -inf if i % 3 else math.nan for i in range(32, 96)}):
        bias = torch.zeros(128, device=dev)
        for e, v in places.items():
            bias[e] = v
        counts_as = bias.nan_to_num(nan=-inf, posinf=inf, neginf=-inf)
        counts_as = torch.where(counts_as == -inf, counts_as, counts_as.clamp(-2.0 ** 100, 2.0 ** 100))
        got = api.route_topk(cfg, z, bias)["topk_idx"]
        assert torch.equal(got[:5], choose(cfg, z[:5], counts_as))


@pytest.mark.parametrize("B", [50, 8200])
def test_groups_a_few_last_bits_of_64_apart(dev, B):
    """1 - sigmoid(34) is 1.7e-15 and of 36 2.3e-16: six and one last places of the sums here."""
    cfg = config(B, N=64, K=2, n_group=2, topk_group=1, score_fn=SIG, renorm=1)
    z = torch.full((B, 64), -50.0, device=dev)
    z[:, 3], z[:, 40] = 34.0, 36.0
    z[:, 9] = z[:, 33] = torch.randn(B, generator=torch.Generator("cuda").manual_seed(3), device=dev)
    assert api.route_topk(cfg, z)["topk_idx"].unique(dim=0).tolist() == [[40, 33]]


@pytest.mark.parametrize("B", [64, 8200])
@pytest.mark.parametrize("most", [1e2, 1e4, 1e5, 1e7])
def test_groups_whose_two_best_scores_cancel(dev, most, B):
    """One expert of each group lifted as far as the others are lowered: the sum of a group's two
    best scores is near 1, but carries the rounding of numbers as large as the biases."""
    gen = torch.Generator("cuda").manual_seed(int(most))
    for K, topk in ((8, 4), (2, 1), (5, 7)):
        cfg = config(B, N=256, K=K, n_group=8, topk_group=topk, score_fn=SIG, renorm=1)
        bias = torch.full((8, 32), -most, device=dev)
        bias.scatter_(1, torch.randint(32, (8, 1), generator=gen, device=dev), most)
        z = torch.randn(B, 256, generator=gen, device=dev) * 0.02          # sums within 0.04 of one another
        z[1::2] *= 50
        pick = torch.arange(0, B, max(1, B // 64), device=dev)
        for zs in (z, z.to(BF16)):
            got = api.route_topk(cfg, zs, bias.view(-1))["topk_idx"]
            assert torch.equal(got[pick], choose(cfg, zs[pick], bias.view(-1)))


@pytest.mark.parametrize("B", [64, 8200])
def test_groups_with_biases_of_every_size(dev, B):
    """Some groups with large scores of both signs beside others with small ones: how far apart
    binary32 can tell two sums depends on the groups compared."""
    gen = torch.Generator("cuda").manual_seed(31)
    for size in (8, 32):
        cfg = config(B, N=8 * size, K=4, n_group=8, topk_group=3, score_fn=SIG, renorm=1)
        for _ in range(6):
            bias = torch.randn(8, size, generator=gen, device=dev) * 0.01
            most = 10.0 ** (torch.rand(8, generator=gen, device=dev) * 7)
            wide = torch.rand(8, generator=gen, device=dev) < 0.5
            bias[wide] -= most[wide, None]
            bias[wide, 3] += 2 * most[wide]                               # near 1 again, with one of -most
            z = torch.randn(B, 8 * size, generator=gen, device=dev) * 0.02
            pick = torch.arange(0, B, max(1, B // 64), device=dev)
            got = api.route_topk(cfg, z, bias.view(-1))["topk_idx"]
            assert torch.equal(got[pick], choose(cfg, z[pick], bias.view(-1)))
