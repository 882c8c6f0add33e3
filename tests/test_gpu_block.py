"""The operators around the experts as they are used together: a block in training against
automatic differentiation in 64 bits, the norm in front of the serving layer, and a dense
layer in 8 bits on the norm's output."""
import numpy as np
import pytest
import torch

import oracle
from combine_moe_route_03_gb300 import api, configs, inputs, train
from oracle.ffn import expert_ffn, layer_tokens
from support import within_tol

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
SMALL = configs.SMALL_CONTIG.with_(B=77, N=16, K=3, H=512, I=256, n_group=4, topk_group=2, shared=True)
EPS = 1e-6
# Relative 2-norm bounds; a rounding to bf16 is at most 2^-8 of a value.  The output passes y,
# gu (whose error the activation at most doubles), h, the rows, their sum and that with the
# shared expert; a gradient at most seven more (dout is exact: dh, dgu, dx of each product, their
# sums, and those of what the forward kept).
OUT, GRAD = 7 * 2.0 ** -8, 14 * 2.0 ** -8


def parameters(cfg, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s, scale=1.0: torch.randn(*s, generator=gen, device="cuda") * scale  # noqa: E731
    q = lambda t: t.bfloat16().float()  # noqa: E731
    p = [1 + r(cfg.H, scale=0.2), q(r(cfg.N, cfg.H, scale=cfg.H ** -0.5)), q(r(cfg.N, 2 * cfg.I, cfg.H, scale=cfg.H ** -0.5)),
         q(r(cfg.N, cfg.H, cfg.I, scale=cfg.I ** -0.5))]
    if cfg.shared:
        p += [q(r(2 * cfg.I, cfg.H, scale=cfg.H ** -0.5)), q(r(cfg.H, cfg.I, scale=cfg.I ** -0.5))]
    return p, r


def reference(cfg, params, x, residual, idx, dout, dh):
    """Output, and gradients of h and the parameters, for the choice that was made."""
    g, wr, w13, w2, *shared = params = [p.double().requires_grad_() for p in params]
    h = (x.double() + (0 if residual is None else residual.double())).requires_grad_()
    y = h * g / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
    z = (y @ wr.t()).gather(1, idx.long())
    if cfg.score_fn == configs.SIGMOID:
        w = torch.sigmoid(z)
        w = w / w.sum(1, keepdim=True)
    else:
        w = torch.exp(z - torch.logsumexp(y @ wr.t(), 1, keepdim=True))
    w = w * cfg.route_scale
    ffn = lambda t, a, b: (lambda gu: (torch.nn.functional.silu(gu[:, :cfg.I]) * gu[:, cfg.I:]) @ b.t())(t @ a.t())  # noqa: E731
    out = torch.zeros_like(h)
    for e in range(cfg.N):
        t, k = (idx == e).nonzero(as_tuple=True)
        if len(t):
            out = out.index_add(0, t, w[t, k][:, None] * ffn(y[t], w13[e], w2[e]))
    if shared:
        out = out + ffn(y, *shared)
    (out * dout.double()).sum().backward()
    return out.detach(), h.grad + (0 if dh is None else dh.double()), [p.grad for p in params]


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("stream_type", [None, BF16, F32])
@pytest.mark.parametrize("kw", [dict(), dict(shared=False, n_group=1, topk_group=1, score_fn=configs.SOFTMAX, renorm=0, route_scale=1.0)],
                         ids=["sigmoid_shared", "softmax"])
def test_block_matches_autograd(dev, kw, stream_type):
    cfg = SMALL.with_(**kw)
    params, r = parameters(cfg)
    x, dout = r(cfg.B, cfg.H).bfloat16(), r(cfg.B, cfg.H).bfloat16()
    residual = None if stream_type is None else r(cfg.B, cfg.H, scale=2.0).to(stream_type)
    dh = None if stream_type is None else r(cfg.B, cfg.H).to(stream_type)
    bias = r(cfg.N, scale=0.1) if cfg.score_fn == configs.SIGMOID else None
    t = train.LayerTrainer(cfg, *params, bias=bias, eps=EPS)
    out, h = t.forward(x, residual)
    idx = t._saved[3]
    dx = t.backward(dout, dh)
    t.check_status()
    want, want_h, want_p = reference(cfg, params, x, residual, idx, dout, dh)
    assert h is x if residual is None else h.dtype == stream_type
    assert int(t.counts.sum()) == cfg.B * cfg.K
    assert off(out, want) <= OUT
    assert dx.dtype == h.dtype and off(dx, want_h) <= GRAD
    grads = [t.grads[0], t.grads[1], *t.experts.grads, *t.grads[2:]]
    for got, ref in zip(grads, want_p):
        assert off(got, ref) <= GRAD


def test_micro_batches_add_up_and_a_step_moves_the_weights(dev):
    params, r = parameters(SMALL, 1)
    a, b = (train.LayerTrainer(SMALL, *params, weight_decay=0.0) for _ in range(2))
    batches = [(r(SMALL.B, SMALL.H).bfloat16(), r(SMALL.B, SMALL.H), r(SMALL.B, SMALL.H).bfloat16()) for _ in range(2)]
    sums = None
    for x, res, dout in batches:
        a.forward(x, res)
        a.backward(dout)
        b.forward(x, res)
        b.backward(dout)
        part = [g.clone() for g in (*b.grads, *b.experts.grads)]
        b.experts._fresh = True                      # start anew
        sums = part if sums is None else [s + p for s, p in zip(sums, part)]
    for got, ref in zip((*a.grads, *a.experts.grads), sums):
        # binary32 sums of at most 512 rows and few additions of them, in another order
        assert bool(((got - ref).abs() <= 2.0 ** -21 * sum(g.abs().max() for g in (got, ref))).all())
    before = [w.clone() for w in (*a.master, *a.experts.master)]
    a.step()
    for w, old in zip((*a.master, *a.experts.master), before):
        assert not torch.equal(w, old)
    for w, copy in zip(a.master[1:], a.weights):
        assert torch.equal(w.bfloat16(), copy)
    with pytest.raises(ValueError, match="backward"):
        a.step()
    with pytest.raises(ValueError, match="forward"):
        a.backward(batches[0][2])


def test_gradients_of_a_captured_block(dev):
    """Forward and backward in one graph, replayed over new inputs, with an eager block's
    buffers alive beside it."""
    params, r = parameters(SMALL, 2)
    t, eager = (train.LayerTrainer(SMALL, *params) for _ in range(2))
    x, res, dout = r(SMALL.B, SMALL.H).bfloat16(), r(SMALL.B, SMALL.H), r(SMALL.B, SMALL.H).bfloat16()
    eager.forward(x, res)
    t.forward(x, res)
    t.backward(dout)
    t.experts._fresh = True
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, h = t.forward(x, res)
        dx = t.backward(dout)
    for _ in range(2):
        for b in (x, res, dout):
            b.copy_(r(SMALL.B, SMALL.H))
        g.replay()
        want, wh = eager.forward(x, res)
        wdx = eager.backward(dout)
        eager.experts._fresh = True
        for got, ref in ((out, want), (h, wh), (dx, wdx), *zip(t.grads, eager.grads), *zip(t.experts.grads, eager.experts.grads)):
            assert torch.equal(got, ref)


def test_the_command_runs(dev, capsys):
    assert len(train.main(["--layer", "--steps", "2", "--state-bits", "32"])) == 2
    assert "step 1" in capsys.readouterr().out


def test_trainer_refusals(dev):
    params, _ = parameters(SMALL)
    with pytest.raises(ValueError, match="shared"):
        train.LayerTrainer(SMALL, *params[:4])
    with pytest.raises(ValueError, match="multiple of 8"):
        train.LayerTrainer(SMALL.with_(N=12), *params)
    with pytest.raises(ValueError, match="gain"):
        train.LayerTrainer(SMALL, params[0][:-1], *params[1:])


def layer_weights(cfg, dev):
    ex = inputs.make_all_experts(cfg)
    return ex, {k: torch.from_numpy(np.ascontiguousarray(v)).to(dev) for k, v in ex.items()}


@pytest.mark.parametrize("residual_type", [None, BF16, F32])
def test_layer_behind_a_norm(dev, residual_type):
    """MoELayer with a norm: the layer of the normed input, and the residual holds the sum."""
    cfg = configs.TINY.with_(B=70)
    W, _ = inputs.make_router(cfg)
    ex, wdev = layer_weights(cfg, dev)
    gen = torch.Generator("cuda").manual_seed(5)
    gain = 1 + torch.randn(cfg.H, generator=gen, device=dev) * 0.2
    x = torch.randn(cfg.B, cfg.H, generator=gen, device=dev).bfloat16()
    res = None if residual_type is None else torch.randn(cfg.B, cfg.H, generator=gen, device=dev).to(residual_type)
    args = (cfg, torch.from_numpy(W).to(dev), None, wdev)
    lay, plain = api.MoELayer(*args, device=dev, norm_w=gain), api.MoELayer(*args, device=dev)
    normed = api.rms_norm(x, gain, residual=res)
    want = plain.forward(normed["y"]).clone()
    for stream in (None, torch.cuda.Stream()):
        mine = None if res is None else res.clone()
        out = lay.forward(x, residual=mine, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        if res is not None:
            assert torch.equal(mine, normed["residual"])
    assert api.read_status(lay.status) == 0
    xb = normed["y"].view(torch.int16).cpu().numpy().view(np.uint16)
    get = lambda e: (ex["W13"][e], ex["W13_sf"][e], ex["W2"][e], ex["W2_sf"][e])  # noqa: E731
    ref = layer_tokens(cfg, xb, W, None, get)["out"]
    assert within_tol(oracle.bf16_to_f32(out.view(torch.int16).cpu().numpy().view(np.uint16)), oracle.bf16_to_f32(ref))[0]
    with pytest.raises(ValueError, match="input"):
        lay.forward()
    with pytest.raises(ValueError, match="norm"):
        plain.forward(x, residual=x)


@pytest.mark.parametrize("B", [1, 100, 128, 129, 300, 513])
def test_dense_tiles_are_those_of_a_shared_expert(dev, B):
    cfg = configs.TINY.with_(B=B)
    x = torch.zeros(B, cfg.H, dtype=BF16, device=dev)
    idx = torch.zeros(B, cfg.K, dtype=torch.int32, device=dev)
    want = api.dispatch(cfg, x, idx, shared=True)["shared_tiles"]
    tiles = (B + 127) // 128
    used = 8 + 8 * tiles + 8 * (tiles // 2 + tiles % 2)              # what follows is room
    assert torch.equal(api.dense_tiles(B)[:used], want[:used]) and api.dense_tiles(B).numel() == want.numel()


@pytest.mark.parametrize("fmt", [api.FMT_FP8, api.FMT_FP8_F32])
@pytest.mark.parametrize("rows", [5, 300])
def test_dense_layer_in_8_bits_on_the_norms_output(dev, rows, fmt):
    """rms_norm's codes and scales through gate/up, activation and down with one expert,
    against the oracle's FFN on the same codes."""
    cfg = configs.TINY.with_(N=1, K=1, H=512, I=256)
    ex, wdev = layer_weights(cfg, dev)
    gen = torch.Generator("cuda").manual_seed(rows)
    x, gain = torch.randn(rows, cfg.H, generator=gen, device=dev).bfloat16(), 1 + torch.randn(cfg.H, generator=gen, device=dev) * 0.2
    o = api.rms_norm(x, gain, y16=False, fmt=fmt)
    f32 = fmt == api.FMT_FP8_F32
    scales = api.weight_scales_f32 if f32 else api.pack_weight_scales
    tiles, most, st = api.dense_tiles(rows), (rows + 127) // 128, api.new_status()
    more = dict(max_tiles=most, status=st, scale_fmt=api.SCALE_F32 if f32 else api.SCALE_UE8M0)
    h, h_sf = api.grouped_gemm_fp8(api.GEMM_GATEUP_SWIGLU, o["A"], o["A_sf"], wdev["W13"], scales(wdev["W13_sf"]), tiles, **more)
    y = api.grouped_gemm_fp8(api.GEMM_DOWN, h, h_sf, wdev["W2"], scales(wdev["W2_sf"]), tiles, **more)[:rows]
    assert api.read_status(st) == 0
    blocks = cfg.H // 128
    if f32:
        s = o["A_sf"].view(F32).view(-1, blocks)[:rows]
    else:
        s = o["A_sf"].view(-1, 1, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, 4)[:rows, :blocks].contiguous()
    want = expert_ffn(o["A"][:rows].cpu().numpy(), s.cpu().numpy(), *[ex[k][0] for k in ("W13", "W13_sf", "W2", "W2_sf")],
                      scale_fmt=int(f32))
    assert within_tol(y.float().cpu().numpy(), oracle.bf16_to_f32(want))[0]


def test_calls_on_several_streams_at_once(dev):
    """Everything together and in any order gives the bits that each gives alone: products split over
    clusters beside others that fill the GPU, workspaces of calls in flight."""
    gen = torch.Generator("cuda").manual_seed(21)
    rand = lambda *s, dtype=torch.bfloat16: (torch.randn(*s, generator=gen, device=dev) * 0.5).to(dtype)  # noqa: E731
    jobs = []
    for m, n, k in ((1, 4096, 2048), (128, 256, 7168), (300, 1000, 1544), (2048, 1024, 2048)):
        x, w, dy = rand(m, k), rand(n, k), rand(m, n)
        jobs.append(lambda x=x, w=w, dy=dy: [api.linear(x, w, residual=dy), api.linear(x, w, out_dtype=torch.float32)])
        jobs.append(lambda x=x, w=w, dy=dy: [*api.linear_backward(dy, x, w, act="gelu", z=dy, bias=True).values()])
    h, dy, gain = rand(1024, 7168), rand(1024, 7168), torch.ones(7168, device=dev)
    jobs.append(lambda: [*api.rms_norm_backward(h, gain, dy), *api.rms_norm(h, gain, residual=dy, fmt=api.FMT_FP8).values()])
    cfg = configs.MoEConfig("routing", B=128, H=128, N=256, K=8, I=128, n_group=8, topk_group=4,
                            score_fn=configs.SIGMOID, renorm=1)
    z, bias = rand(128, 256, dtype=torch.float32), rand(256, dtype=torch.float32) * 0.1
    jobs.append(lambda: [*api.route_topk(cfg, z, bias).values()])
    want = [job() for job in jobs]
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for turn in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got += [(j, jobs[j]()) for j in range((turn + i) % 3, len(jobs), 3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for j, out in got for a, b in zip(out, want[j]))
    assert api.default_status() == 0


def test_the_norm_is_left_out_by_no_call(dev):
    """What cannot run the norm refuses the layer; forward in a captured graph runs it."""
    cfg = configs.TINY.with_(B=70)
    W, _ = inputs.make_router(cfg)
    gen = torch.Generator("cuda").manual_seed(6)
    gain = 1 + torch.randn(cfg.H, generator=gen, device=dev) * 0.2
    lay = api.MoELayer(cfg, torch.from_numpy(W).to(dev), None, layer_weights(cfg, dev)[1], device=dev, norm_w=gain)
    host = torch.zeros(cfg.B, cfg.H, dtype=BF16).pin_memory()
    for call in (lambda: lay.forward_host(host, host), lambda: lay.forward_host_pipelined([host], [host]),
                 lambda: api.LayerGraph(lay, torch.cuda.Stream()), lambda: api.LayerGraph(lay, torch.cuda.Stream(), host, host)):
        with pytest.raises(ValueError, match="norm"):
            call()
    x, res = torch.randn(cfg.B, cfg.H, generator=gen, device=dev).bfloat16(), torch.randn(cfg.B, cfg.H, generator=gen, device=dev)
    lay.forward(x, residual=res.clone())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = lay.forward(x, residual=res)
    for _ in range(2):
        x.copy_(torch.randn(cfg.B, cfg.H, generator=gen, device=dev))
        mine = res.clone()
        g.replay()
        got = out.clone()
        assert torch.equal(lay.forward(x, residual=mine), got) and torch.equal(mine, res)


FIRST_CALLS = """
import threading, torch
from combine_moe_route_03_gb300 import api, configs
gen = torch.Generator("cuda").manual_seed(0)
rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
x, w, dy, h, gain = rand(700, 512), rand(264, 512), rand(700, 264), rand(700, 2048), torch.ones(2048, device="cuda")
z = torch.randn(100, 64, generator=gen, device="cuda")
cfg = configs.MoEConfig("routing", B=100, H=128, N=64, K=4, I=128)
def calls():
    b = api.linear_backward(dy, x, w, act="silu", z=dy)
    return [api.linear(x, w), api.linear(x[:8], w, out_dtype=torch.float32), b["dx"], b["dw"], api.rms_norm(h, gain)["y"],
            *api.rms_norm_backward(h, gain, h), *api.route_topk(cfg, z).values()]
torch.cuda.synchronize()
gate, got = threading.Barrier(8), [None] * 8
def go(i):
    gate.wait()
    got[i] = calls()
threads = [threading.Thread(target=go, args=(i,)) for i in range(8)]
for t in threads: t.start()
for t in threads: t.join()
want = calls()
assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
print("the same")
"""


def test_first_calls_of_several_threads_at_once(dev):
    """What a process asks of a device once is asked by all of them."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "the same" in run.stdout, run.stderr[-2000:]


def test_a_refused_backward_leaves_the_gradients_alone(dev):
    """What backward cannot take is refused before anything is added up: the right call after it
    gives what it gives alone."""
    params, r = parameters(SMALL, 3)
    t, fresh = (train.LayerTrainer(SMALL, *params) for _ in range(2))
    x, res = r(SMALL.B, SMALL.H).bfloat16(), r(SMALL.B, SMALL.H)
    dout, dh = r(SMALL.B, SMALL.H).bfloat16(), r(SMALL.B, SMALL.H)
    for u in (t, fresh):
        u.forward(x, res)
    for bad in (dict(dh=dh.bfloat16()), dict(dh=dh[:-1]), dict(dh=dh.t().contiguous().t()), dict(dh=dh.cpu()), dict(dout=dout.float()),
                dict(dout=dout[1:]), dict(dout=dout.cpu())):
        with pytest.raises(ValueError):
            t.backward(**{**dict(dout=dout, dh=dh), **bad})
        assert not any(bool(g.any()) for g in (*t.grads, *t.experts.grads))
    assert torch.equal(t.backward(dout, dh), fresh.backward(dout, dh))
    for got, want in zip((*t.grads, *t.experts.grads), (*fresh.grads, *fresh.experts.grads)):
        assert torch.equal(got, want)
