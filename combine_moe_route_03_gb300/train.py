"""Training of the routed experts in 16-bit storage, on the library's kernels.

One layer forward and backward:

    route -> dispatch (bf16 rows) -> grouped product W13 -> swiglu x routing weight
          -> grouped product W2 -> combine

The routing weight enters at the activation (h = w silu(g) u), which the second product
then carries through: the combine only sums a token's rows.  So the backward needs no
permutation of its own: the rows' gradient is the dispatch of the output's gradient, and
the input's gradient the combine of the rows' (both with unit weights).  The gradients of
the routing weights come out of the activation's backward; the router itself (its choice of
experts and its weights) is the caller's to train.  A shared expert of the configuration is
no part of this: outputs and gradients are the routed experts' alone.

    python -m combine_moe_route_03_gb300.train [--steps N] [--state-bits 8|32]

fits a small layer to another's outputs and prints the loss.
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


def main(argv=None) -> list[float]:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=8)
    args = ap.parse_args(argv)
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
