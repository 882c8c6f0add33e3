"""Training of the routed experts in 16-bit storage, on the library's kernels.

One layer forward and backward:

    route -> dispatch (bf16 rows) -> grouped product W13 -> swiglu x routing weight
          -> grouped product W2 -> combine

The routing weight enters at the activation (h = w silu(g) u), which the second product
then carries through: the combine only sums a token's rows.  So the backward needs no
permutation of its own: the rows' gradient is the dispatch of the output's gradient, and
the input's gradient the combine of the rows' (both with unit weights).  The gradients of
the routing weights come out of the activation's backward.  Of ExpertTrainer the router
(its choice of experts and its weights) and a shared expert are no part: outputs and gradients
are the routed experts' alone.

LayerTrainer is the whole block around them: root-mean-square norm of the residual stream,
router, routed experts and shared expert, with the gradients of all of it.

    python -m combine_moe_route_03_gb300.train [--layer] [--steps N] [--state-bits 8|32]

fits a small layer's experts (--layer: a whole block) to another's outputs and prints the loss.
"""
from __future__ import annotations

import argparse

import torch

from . import _lib, api
from .configs import CONTIG, SMALL_CONTIG, MoEConfig

ALIGN = 128     # rows a contiguous dispatch rounds a segment up to


class ExpertTrainer:
    """The experts of one MoE layer (W13 [N][2I][H], W2 [N][H][I]; gate rows, then up rows,
    as moe_grouped_gemm_fp8 has them) as bf16 weights with binary32 masters, their
    gradients, and an AdamW over both.

    ``forward`` keeps what ``backward`` needs; ``backward`` returns the gradients of the
    input and of the routing weights, and adds to the weights' gradients (binary32) until
    ``step`` applies and clears them, so several forward/backward pairs make one step.  What
    the device finds wrong meanwhile is kept: ``check_status`` raises it."""

    def __init__(self, cfg: MoEConfig, W13: torch.Tensor, W2: torch.Tensor, state_bits: int = 32,
                 **adamw):
        if cfg.layout != CONTIG or cfg.N_phys != cfg.N:
            raise ValueError("training: a contiguous layout without replicas expected")
        self.cfg = cfg
        shapes = (cfg.N, 2 * cfg.I, cfg.H), (cfg.N, cfg.H, cfg.I)
        self.master = [w.to(torch.float32, copy=True).contiguous() for w in (W13, W2)]
        for w, s, what in zip(self.master, shapes, ("W13", "W2")):
            api._expect(w, what, (torch.float32,), s)
        self.W13, self.W2 = self.weights = [w.to(torch.bfloat16) for w in self.master]
        self.grads = [torch.zeros_like(w) for w in self.master]
        self.opt = api.AdamW(self.master, state_bits=state_bits, copies=self.weights, **adamw)
        self.status = api.new_status(W13.device)
        self._fresh = True          # the gradients hold nothing yet
        self._saved = None

    def _dispatch(self, x, topk_idx):
        d = api.dispatch(self.cfg, x, topk_idx, fmt=api.FMT_BF16, status=self.status)
        return d["A"].view(torch.bfloat16), d

    def forward(self, x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor) -> torch.Tensor:
        """x bf16 [B][H], topk_idx and topk_w [B][K] (as api.route gives them) -> bf16 [B][H].
        A pair whose expert index lies outside [0, N) is left out, as dispatch and combine do:
        it adds nothing, the gradient of its weight is 0, and check_status raises."""
        rows_x, d = self._dispatch(x, topk_idx)
        seg = dict(counts=d["counts"], align=ALIGN, status=self.status)
        row_of, rows = d["row_of"], d["rows"]
        # pairs left out (row -1) share one entry behind the rows
        at = torch.where(row_of < 0, rows, row_of).reshape(-1).long()
        row_w = torch.zeros(rows + 1, dtype=torch.float32, device=x.device)
        row_w[at] = topk_w.reshape(-1)
        row_w = row_w[:rows]
        gu = api.grouped_gemm(rows_x, self.W13, **seg)
        h = api.swiglu(gu, row_w=row_w, **seg)
        y = api.grouped_gemm(h, self.W2, **seg)
        ones = torch.ones_like(topk_w)
        self._saved = (topk_idx, rows_x, gu, h, row_w, row_of, at, ones, seg)
        return api.combine(y, row_of, ones, status=self.status)

    def backward(self, dout: torch.Tensor):
        """dout bf16 [B][H], the gradient of forward's output -> (dx bf16 [B][H], the
        gradient of topk_w fp32 [B][K])."""
        if self._saved is None:
            raise ValueError("backward: a forward before it expected")
        topk_idx, rows_x, gu, h, row_w, row_of, at, ones, seg = self._saved
        self._saved = None
        dy, _ = self._dispatch(dout, topk_idx)
        more = dict(accumulate=not self._fresh, **seg)
        self._fresh = False
        api.grouped_wgrad(dy, h, out=self.grads[1], **more)
        dh = api.grouped_gemm(dy, self.W2, trans=True, **seg)
        drow_w = torch.zeros(row_w.numel() + 1, dtype=torch.float32, device=dy.device)
        dgu, _ = api.swiglu_backward(gu, dh, row_w=row_w, dgu=gu, drow_w=drow_w[:-1], **seg)
        api.grouped_wgrad(dgu, rows_x, out=self.grads[0], **more)
        dx = api.grouped_gemm(dgu, self.W13, trans=True, **seg)
        return api.combine(dx, row_of, ones, status=self.status), drow_w[at].view(ones.shape)

    def check_status(self) -> None:
        """Raises if a call so far found something wrong on the device: pairs left out, a cut
        segment, or a wait that gave up, whose results are incomplete.  Waits for the current
        stream; call it as often as a result is relied on.  The word is cleared."""
        torch.cuda.current_stream(self.status.device).synchronize()
        bits = api.read_status(self.status)
        if bits:
            self.status.zero_()
            names = [n for n in ("CAPACITY", "TIMEOUT", "BAD_INDEX") if bits & getattr(_lib, "STATUS_" + n)]
            raise RuntimeError("device status " + (", ".join(names) or str(bits)))

    def step(self, grad_scale: torch.Tensor | None = None) -> None:
        """Applies the gradients added up since the last step."""
        if self._fresh:
            raise ValueError("step: a backward before it expected")
        self.opt.step(self.grads, grad_scale=grad_scale)
        self._fresh = True


class LayerTrainer:
    """One MoE block in training, with its residual stream (bf16 or fp32):

        h = x + residual -> norm -> y;  router logits y W_router^T (binary32) -> route_topk
        out = routed experts of y (+ shared expert of y)

    ``forward`` returns (out, h): the next block's norm adds out to h.  Parameters: the norm's
    gains [H], W_router [N][H], the routed experts (an ExpertTrainer) and with a shared expert
    W13s [2I][H], W2s [H][I]; matrices as bf16 weights with binary32 masters, one AdamW for what
    is not the experts'.  ``bias`` (sigmoid scores) steers the choice of experts and has no
    gradient; it is the caller's to change between steps, as are the last routing's
    ``counts``.  Micro-batches add up and steps apply as ExpertTrainer's do."""

    def __init__(self, cfg: MoEConfig, gain: torch.Tensor, W_router: torch.Tensor, W13: torch.Tensor,
                 W2: torch.Tensor, W13s: torch.Tensor | None = None, W2s: torch.Tensor | None = None,
                 bias: torch.Tensor | None = None, eps: float = 1e-6, state_bits: int = 32, **adamw):
        if cfg.shared != (W13s is not None) or cfg.shared != (W2s is not None):
            raise ValueError("shared expert: weights where the configuration has one, else none")
        if cfg.N % 8:
            raise ValueError("training the router: a multiple of 8 experts expected")
        self.cfg, self.bias, self.eps = cfg, bias, eps
        self.experts = ExpertTrainer(cfg, W13, W2, state_bits, **adamw)
        given = [gain, W_router] + ([W13s, W2s] if cfg.shared else [])
        shapes = [(cfg.H,), (cfg.N, cfg.H), (2 * cfg.I, cfg.H), (cfg.H, cfg.I)]
        self.master = [w.to(torch.float32, copy=True).contiguous() for w in given]
        for w, s, what in zip(self.master, shapes, ("gain", "W_router", "W13s", "W2s")):
            api._expect(w, what, (torch.float32,), s)
        self.gain = self.master[0]
        self.weights = [w.to(torch.bfloat16) for w in self.master[1:]]
        self.grads = [torch.zeros_like(w) for w in self.master]
        self.opt = api.AdamW(self.master, state_bits=state_bits, copies=[None, *self.weights], **adamw)
        self.counts = None
        self._saved = None

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        """x bf16 [B][H], residual bf16 or fp32 [B][H] (None: 0, the stream then is x itself) ->
        (out bf16 [B][H], h)."""
        status = dict(status=self.experts.status)
        n = api.rms_norm(x, self.gain, residual=residual, eps=self.eps)
        y, h = n["y"], n.get("residual", x)
        logits = api.linear(y, self.weights[0], out_dtype=torch.float32, **status)
        r = api.route_topk(self.cfg, logits, self.bias)
        self.counts = r["counts"]
        out = self.experts.forward(y, r["topk_idx"], r["topk_w"])
        shared = None
        if self.cfg.shared:
            gu = api.linear(y, self.weights[1], **status)
            a = api.swiglu(gu)
            out = api.linear(a, self.weights[2], residual=out, out=out, **status)
            shared = gu, a
        self._saved = y, h, logits, r["topk_idx"], shared
        return out, h

    def backward(self, dout: torch.Tensor, dh: torch.Tensor | None = None) -> torch.Tensor:
        """dout bf16 [B][H], the gradient of forward's output, and dh, of h's type, what flows
        into h from later blocks -> the gradient of h's terms (x and the residual), of h's type."""
        if self._saved is None:
            raise ValueError("backward: a forward before it expected")
        y, h, logits, topk_idx, shared = self._saved
        # before anything is added to a gradient
        api._is(dout, "dout", torch.bfloat16, h.shape)
        if dh is not None:
            api._is(dh, "dh", h.dtype, h.shape)
        _lib.ptrs(dout, dh)
        self._saved = None
        more = dict(accumulate=not self.experts._fresh)
        dy, dw = self.experts.backward(dout)
        more["status"] = self.experts.status
        dlogits = api.route_topk_backward(self.cfg, logits, topk_idx, dw, out_dtype=torch.bfloat16)
        dy = api.linear_backward(dlogits, y, self.weights[0], add=dy, dw=self.grads[1], **more)["dx"]
        if shared is not None:
            gu, a = shared
            da = api.linear_backward(dout, a, self.weights[2], dw=self.grads[3], **more)["dx"]
            dgu, _ = api.swiglu_backward(gu, da, dgu=gu)
            dy = api.linear_backward(dgu, y, self.weights[1], add=dy, dw=self.grads[2], **more)["dx"]
        return api.rms_norm_backward(h, self.gain, dy, eps=self.eps, dres=dh, dw=self.grads[0],
                                     accumulate=more["accumulate"])[0]

    def check_status(self) -> None:
        """As ExpertTrainer's, for all calls of the block."""
        self.experts.check_status()

    def step(self, grad_scale: torch.Tensor | None = None) -> None:
        """Applies the gradients added up since the last step."""
        self.experts.step(grad_scale)
        self.opt.step(self.grads, grad_scale=grad_scale)


def _fit_layer(args) -> list[float]:
    cfg, gen = SMALL_CONTIG, torch.Generator("cuda").manual_seed(0)
    rand = lambda *s, scale=1.0: torch.randn(*s, generator=gen, device="cuda") * scale  # noqa: E731
    new = lambda: [1 + rand(cfg.H, scale=0.1), rand(cfg.N, cfg.H, scale=cfg.H ** -0.5),  # noqa: E731
                   rand(cfg.N, 2 * cfg.I, cfg.H, scale=cfg.H ** -0.5), rand(cfg.N, cfg.H, cfg.I, scale=cfg.I ** -0.5),
                   rand(2 * cfg.I, cfg.H, scale=cfg.H ** -0.5), rand(cfg.H, cfg.I, scale=cfg.I ** -0.5)]
    goal, start = new(), new()
    teacher = LayerTrainer(cfg, *goal)
    student = LayerTrainer(cfg, *[0.5 * s + 0.5 * t for s, t in zip(start, goal)], state_bits=args.state_bits,
                           lr=1e-3, betas=(0.9, 0.95), weight_decay=0.0)
    x, residual = rand(cfg.B, cfg.H).to(torch.bfloat16), rand(cfg.B, cfg.H)
    want = teacher.forward(x, residual)[0].float()
    losses = []
    for i in range(args.steps):
        diff = student.forward(x, residual)[0].float() - want
        losses.append(float(diff.square().mean()))
        student.backward((diff * (2.0 / diff.shape[0])).to(torch.bfloat16))
        student.step()
        print(f"step {i}: loss {losses[-1]:.5f}")
    teacher.check_status()
    student.check_status()
    return losses


def main(argv=None) -> list[float]:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=8)
    ap.add_argument("--layer", action="store_true", help="a whole block: norm, router, experts, shared expert")
    args = ap.parse_args(argv)
    if args.layer:
        return _fit_layer(args)
    cfg, gen = SMALL_CONTIG, torch.Generator("cuda").manual_seed(0)
    rand = lambda *s, scale=1.0: torch.randn(*s, generator=gen, device="cuda") * scale  # noqa: E731
    new = lambda: (rand(cfg.N, 2 * cfg.I, cfg.H, scale=cfg.H ** -0.5),  # noqa: E731
                   rand(cfg.N, cfg.H, cfg.I, scale=cfg.I ** -0.5))
    W_router = rand(cfg.N, cfg.H, scale=cfg.H ** -0.5)
    teacher = ExpertTrainer(cfg, *new())
    start = new()
    student = ExpertTrainer(cfg, *[0.5 * s + 0.5 * t for s, t in zip(start, teacher.master)],
                            state_bits=args.state_bits, lr=1e-3, betas=(0.9, 0.95), weight_decay=0.0)
    x = rand(cfg.B, cfg.H).to(torch.bfloat16)
    r = api.route(cfg, x, W_router, None)
    want = teacher.forward(x, r["topk_idx"], r["topk_w"]).float()
    losses = []
    for i in range(args.steps):
        diff = student.forward(x, r["topk_idx"], r["topk_w"]).float() - want
        losses.append(float(diff.square().mean()))
        student.backward((diff * (2.0 / diff.shape[0])).to(torch.bfloat16))
        student.step()
        print(f"step {i}: loss {losses[-1]:.5f}")
    teacher.check_status()
    student.check_status()
    return losses


if __name__ == "__main__":
    main()
