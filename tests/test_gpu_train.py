"""ExpertTrainer against the same layer by automatic differentiation in 64 bits, and its
use over several micro-batches and steps."""
import pytest
import torch

from combine_moe_route_03_gb300 import _lib, api, configs, train

pytestmark = pytest.mark.gpu

SMALL = configs.SMALL_CONTIG.with_(B=77, N=8, K=3, H=512, I=256, n_group=1, topk_group=1, shared=False)
# Relative 2-norm bounds.  A rounding to bf16 is at most 2^-8 of a value.  The output passes
# four (gu, whose error the activation at most doubles, h, the rows, their sum), a gradient
# at most six more (dy is exact, dh, dgu, and those of h and gu in them).
OUT, GRAD = 5 * 2.0 ** -8, 10 * 2.0 ** -8


def make(cfg, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s, scale=1.0: torch.randn(*s, generator=gen, device="cuda") * scale  # noqa: E731
    W13 = r(cfg.N, 2 * cfg.I, cfg.H, scale=cfg.H ** -0.5).bfloat16().float()
    W2 = r(cfg.N, cfg.H, cfg.I, scale=cfg.I ** -0.5).bfloat16().float()
    x, dout = r(cfg.B, cfg.H).bfloat16(), r(cfg.B, cfg.H).bfloat16()
    route = api.route(cfg, x, r(cfg.N, cfg.H, scale=cfg.H ** -0.5), None)
    return W13, W2, x, dout, route["topk_idx"], route["topk_w"]


def reference(cfg, W13, W2, x, dout, idx, w):
    W13, W2, x, w = (t.double().requires_grad_() for t in (W13, W2, x, w))
    out = torch.zeros_like(x)
    for e in range(cfg.N):
        t, k = (idx == e).nonzero(as_tuple=True)
        if len(t):
            gu = x[t] @ W13[e].t()
            g, u = gu[:, :cfg.I], gu[:, cfg.I:]
            out = out.index_add(0, t, w[t, k][:, None] * ((g * torch.sigmoid(g) * u) @ W2[e].t()))
    out.backward(dout.double())
    return out.detach(), x.grad, w.grad, W13.grad, W2.grad


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_forward_and_gradients_match_autograd(dev):
    W13, W2, x, dout, idx, w = make(SMALL)
    t = train.ExpertTrainer(SMALL, W13, W2)
    out = t.forward(x, idx, w)
    dx, dw = t.backward(dout)
    want = reference(SMALL, W13, W2, x, dout, idx, w)
    assert api.read_status(t.status) == 0
    assert off(out, want[0]) <= OUT
    for got, ref in zip((dx, dw, t.grads[0], t.grads[1]), want[1:]):
        assert off(got, ref) <= GRAD


def test_pairs_left_out_have_no_gradient(dev):
    """Expert indices outside [0, N), one token's all of them, over memory that held NaN."""
    W13, W2, x, dout, idx, w = make(SMALL, 2)
    idx = idx.clone()
    idx[3, 1], idx[10, 0], idx[76, 2] = -1, SMALL.N, -7
    idx[20] = -1
    out_of = (idx < 0) | (idx >= SMALL.N)
    t = train.ExpertTrainer(SMALL, W13, W2)
    used = [torch.full((2 ** n,), 0xFF, dtype=torch.uint8, device=dev) for n in range(10, 24) for _ in range(4)]
    del used
    out = t.forward(x, idx, w)
    dx, dw = t.backward(dout)
    want = reference(SMALL, W13, W2, x, dout, idx, w)
    assert api.read_status(t.status) == _lib.STATUS_BAD_INDEX
    assert not bool(dw[out_of].any()) and not bool(out[20].any()) and not bool(dx[20].any())
    assert off(out, want[0]) <= OUT
    for got, ref in zip((dx, dw, t.grads[0], t.grads[1]), want[1:]):
        assert off(got, ref) <= GRAD


def test_micro_batches_add_up_and_a_step_clears_them(dev):
    W13, W2, x, dout, idx, w = make(SMALL, 1)
    a, b = (train.ExpertTrainer(SMALL, W13, W2, state_bits=8, weight_decay=0.0) for _ in range(2))
    a.forward(x, idx, w)
    a.backward(dout)
    one = [g.clone() for g in a.grads]
    a.forward(x, idx, w)
    a.backward(dout)
    for g, h in zip(a.grads, one):
        assert torch.equal(g, 2 * h)               # doubling is exact
    b.forward(x, idx, w)
    b.backward(dout)
    a.step(grad_scale=torch.tensor(0.5, device=dev))
    b.step()
    for p, q, c in zip(a.master, b.master, a.weights):
        assert torch.equal(p, q) and torch.equal(c, p.bfloat16())
        assert not torch.equal(p, W13 if p.shape == W13.shape else W2)
    with pytest.raises(ValueError, match="backward before"):
        a.step()
    with pytest.raises(ValueError, match="forward before"):
        a.backward(dout)
    a.forward(x, idx, w)
    a.backward(dout)
    b.forward(x, idx, w)
    b.backward(dout)
    for g, h in zip(a.grads, b.grads):
        assert torch.equal(g, h)                   # nothing of the last step is left in them


def test_what_the_device_found_wrong_is_raised(dev):
    W13, W2, x, dout, idx, w = make(SMALL, 3)
    t = train.ExpertTrainer(SMALL, W13, W2)
    t.forward(x, idx, w)
    t.backward(dout)
    t.check_status()
    bad = idx.clone()
    bad[0, 0] = -1
    t.forward(x, bad, w)
    t.backward(dout)
    with pytest.raises(RuntimeError, match="BAD_INDEX"):
        t.check_status()
    t.check_status()


@pytest.mark.parametrize("bits", ["8", "32"])
def test_the_example_learns(dev, bits, capsys):
    losses = train.main(["--steps", "12", "--state-bits", bits])
    assert losses[-1] < 0.7 * losses[0]


def test_refuses_other_layouts(dev):
    W13, W2, *_ = make(SMALL)
    for cfg in (SMALL.with_(layout=configs.MASKED, cap=128), SMALL.with_(n_phys=10)):
        with pytest.raises(ValueError, match="expected"):
            train.ExpertTrainer(cfg, W13, W2)
    with pytest.raises(ValueError, match="expected"):
        train.ExpertTrainer(SMALL, W2, W13)


def test_masked_rows_through_the_chain(dev):
    """The decode layout: dispatch into slots of `cap` rows, both products and the activation over
    them, combine; against the layer's definition.  Slots past a count hold NaN."""
    cfg = SMALL.with_(layout=configs.MASKED, cap=128)
    W13, W2, x, dout, idx, w = make(cfg, 4)
    status = api.new_status()
    d = api.dispatch(cfg, x, idx, fmt=api.FMT_BF16, status=status)
    rows_x, row_of = d["A"].view(torch.bfloat16), d["row_of"]
    live = torch.zeros(d["rows"], dtype=torch.bool, device=dev)
    live[row_of.long().reshape(-1)] = True
    rows_x[~live] = float("nan")
    row_w = torch.full((d["rows"],), float("nan"), device=dev)
    row_w[row_of.long().reshape(-1)] = w.reshape(-1)
    seg = dict(counts=d["counts"], cap=cfg.cap, status=status)
    gu = api.grouped_gemm(rows_x, W13.bfloat16(), **seg)
    y = api.grouped_gemm(api.swiglu(gu, row_w=row_w, **seg), W2.bfloat16(), **seg)
    out = api.combine(y, row_of, torch.ones_like(w), status=status)
    assert api.read_status(status) == 0
    assert off(out, reference(cfg, W13, W2, x, dout, idx, w)[0]) <= OUT
