"""Operators that train the experts of the MoE layer in 16-bit storage: cases and plain forms.

* grouped products over ragged segments of rows, one expert's weights per segment, in
  three directions: y = x W_e^T ("fwd"), dx = dy W_e ("dgrad"), dW_e = dy^T x ("wgrad",
  stored in 16 bits or added to binary32 gradients);
* the gated activation h = w silu(g) u between the two products of an expert, and its
  gradients with respect to g, u and the row weight w;
* one AdamW step over many tensors at once, moments in binary32 or in 8-bit codes.

Every case is a dict of plain values.  Segments: expert e's rows start at the sum over
q < e of counts[q] rounded up to ``align`` rows; rows past a segment's count are padding
that nothing reads or writes.  The 8-bit moments are square-law codes per block of 256
consecutive values: m = s q|q| with q = code / 127, and r = sqrt(v) = s q^2 with
q = code / 255, s the block's largest magnitude.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 256            # values of one 8-bit block
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.95, 1e-8, 0.1


# ----------------------------------------------------------------------- cases
def listed():
    return [
        # the router's smallest layer (64 tokens, 2 of 8 experts): launch latency
        dict(name="fwd_tiny", op="fwd", E=8, rows=128, n=256, k=256, skew=0.0, align=1, type="bf16"),
        # serving without quantisation: 128 tokens, 8 of 64 experts, ~16 rows each; the
        # product reads 3.8 GB of weights
        dict(name="fwd_decode", op="fwd", E=64, rows=1024, n=4096, k=7168, skew=0.0, align=1, type="bf16"),
        # a training or prefill batch of 2048 tokens, gate and up projections
        dict(name="fwd_prefill", op="fwd", E=64, rows=16384, n=4096, k=7168, skew=0.0, align=128, type="bf16"),
        # the same batch, gradient of the down projection's input
        dict(name="dgrad_prefill", op="dgrad", E=64, rows=16384, n=7168, k=2048, skew=0.0, align=128, type="bf16"),
        # a popular expert beside empty ones, widths that fill no tile, half precision
        dict(name="dgrad_ragged_f16", op="dgrad", E=37, rows=4099, n=1000, k=1544, skew=1.2, align=1, type="f16"),
        # the same batch, weight gradients of gate and up in 16 bits
        dict(name="wgrad_prefill", op="wgrad", E=64, rows=16384, n=4096, k=7168, skew=0.0, align=128, type="bf16", out="bf16"),
        # gradient accumulation over micro-batches into binary32, skewed routing
        dict(name="wgrad_acc_f32", op="wgrad", E=32, rows=6144, n=2048, k=2048, skew=1.2, align=1, type="bf16", out="f32"),
        # the activation of a decode-sized batch, backward with row weights
        dict(name="swiglu_bwd_small", op="swiglu_bwd", E=64, rows=1024, I=2048, align=1, weights=True, type="bf16"),
        # the activation of 8192 tokens with 8 experts each
        dict(name="swiglu_fwd", op="swiglu", E=256, rows=65536, I=2048, align=128, weights=True, type="bf16"),
        dict(name="swiglu_bwd", op="swiglu_bwd", E=256, rows=65536, I=2048, align=128, weights=True, type="bf16"),
        # the parameters of four layers (32 experts, hidden size 1024): 20 tensors from
        # a 32-value bias to 34 M values, moments in binary32, a bf16 copy for the model
        dict(name="adamw_f32", op="adamw", layers=4, E=32, H=1024, I=512, bits=32, type="bf16"),
        # the same parameters with moments in 8 bits
        dict(name="adamw_8bit", op="adamw", layers=4, E=32, H=1024, I=512, bits=8, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "dgrad", "wgrad", "fwd", "dgrad", "wgrad", "swiglu", "swiglu_bwd", "adamw"])
    type_ = rng.choice(["bf16", "bf16", "f16"])
    if op == "adamw":
        E, H = _log(rng, 1, 32), 8 * _log(rng, 8, 128)
        return dict(op=op, layers=_log(rng, 1, 8) if E < 16 else rng.randint(1, 4), E=E, H=H,
                    I=_log(rng, 32, 512), bits=rng.choice([32, 8]), type=type_)
    align = rng.choice([1, 1, 128])
    E = _log(rng, 1, 64)
    if op.startswith("swiglu"):
        return dict(op=op, E=E, rows=_log(rng, 1, 65536), I=rng.choice([_log(rng, 16, 2048), 8 * _log(rng, 4, 256)]),
                    align=align, weights=rng.random() < 0.7, type=type_)
    skew = rng.choice([0.0, 0.0, 1.2])
    rows = _log(rng, 1, 16384)
    n, k = 8 * _log(rng, 8, 896), 8 * _log(rng, 8, 896)
    most = 5e10 if skew else 4e11        # rows x n x k: the plain form pads to the longest segment
    while rows * n * k > most or E * n * k > 1.8e9:
        rows, n, k = max(1, rows * 2 // 3), max(64, n * 3 // 4 // 8 * 8), max(64, k * 3 // 4 // 8 * 8)
    n, k = (v + 8 if v == 3072 else v for v in (n, k))
    c = dict(op=op, E=E, rows=rows, n=n, k=k, skew=skew, align=align, type=type_)
    if op == "wgrad":
        c["out"] = rng.choice([type_, "f32"])
    return c


# ---------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(gen, *shape, scale=1.0, dtype=torch.float32):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat, step = out.view(-1), 1 << 28
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV) * scale)
    return out


def _counts(case, seed):
    """Rows of each expert: a multinomial draw, Zipf(skew) popularity over a permutation."""
    g = torch.Generator().manual_seed(seed)
    E = case["E"]
    p = (torch.randperm(E, generator=g) + 1).double().pow(-case.get("skew", 0.0))
    c = torch.bincount(torch.multinomial(p, case["rows"], replacement=True, generator=g), minlength=E)
    return c.to(torch.int32)


def _rows_alloc(case):
    """Rows that hold any counts: every segment may end in align - 1 rows of padding."""
    return case["rows"] + min(case["E"], case["rows"]) * (case["align"] - 1)


def _pad(t, live):
    """Rows of padding hold what was in memory: here NaN."""
    t[~live] = float("nan")
    return t


def _sizes(case):
    """Parameter tensors of `layers` MoE layers: experts, router, its bias, two norms."""
    E, H, I = case["E"], case["H"], case["I"]
    return [E * 2 * I * H, E * H * I, E * H, E, H + 7] * case["layers"]


def _offsets(sizes):
    at, total = [], 0
    for n in sizes:
        at.append(total)
        total += (n + BLOCK - 1) // BLOCK * BLOCK
    return at, total


def prepare(case, seed):
    op, gen = case["op"], _gen(seed)
    dt = TYPES[case["type"]]
    if op == "adamw":
        return _prepare_adamw(case, gen)
    counts = _counts(case, seed)
    rows = _rows_alloc(case)
    s = dict(case=case, counts=counts.to(DEV), rows=rows, longest=int(counts.max()))
    live = _live(s)[0]
    if op in ("fwd", "dgrad"):
        E, n, k = case["E"], case["n"], case["k"]
        red, cols = (k, n) if op == "fwd" else (n, k)
        s["x"] = _pad(_normal(gen, rows, red, dtype=dt), live)
        s["w"] = _normal(gen, E, n, k, scale=k ** -0.5, dtype=dt)
        s["out"] = torch.zeros(rows, cols, dtype=dt, device=DEV)
    elif op == "wgrad":
        E, n, k = case["E"], case["n"], case["k"]
        s["dy"] = _pad(_normal(gen, rows, n, scale=0.1, dtype=dt), live)
        s["x"] = _pad(_normal(gen, rows, k, dtype=dt), live)
        if case["out"] == "f32":           # gradients that earlier micro-batches left
            s["acc"] = _normal(gen, E, n, k)
        else:
            s["out"] = torch.zeros(E, n, k, dtype=dt, device=DEV)
    else:
        I = case["I"]
        s["gu"] = _pad(_normal(gen, rows, 2 * I, scale=1.5, dtype=dt), live)
        s["row_w"] = None
        if case["weights"]:
            s["row_w"] = _pad(torch.rand(rows, generator=gen, device=DEV) * 2.5 + 1e-3, live)
        if op == "swiglu":
            s["h"] = torch.zeros(rows, I, dtype=dt, device=DEV)
        else:
            s["dh"] = _pad(_normal(gen, rows, I, scale=0.1, dtype=dt), live)
            s["dgu"] = torch.zeros(rows, 2 * I, dtype=dt, device=DEV)
            s["drow_w"] = torch.zeros(rows, device=DEV) if case["weights"] else None
    return s


def _prepare_adamw(case, gen):
    sizes = _sizes(case)
    at, total = _offsets(sizes)
    live = torch.zeros(total, dtype=torch.bool, device=DEV)
    for o, n in zip(at, sizes):
        live[o:o + n] = True
    dt = TYPES[case["type"]]
    s = dict(case=case, t=0)
    s["p"] = _normal(gen, total, scale=0.02) * live
    s["g"] = (_normal(gen, total, scale=1e-3) * live).to(dt)
    s["copy"] = s["p"].to(dt)
    nb = total // BLOCK
    if case["bits"] == 32:
        s["m"] = _normal(gen, total, scale=3e-4) * live
        s["v"] = (_normal(gen, total, scale=1e-3) * live).square()
    else:
        s["m_code"] = (torch.randint(-127, 128, (total,), generator=gen, device=DEV) * live).to(torch.int8)
        s["r_code"] = (torch.randint(1, 256, (total,), generator=gen, device=DEV) * live).to(torch.uint8)
        s["m_scale"] = torch.rand(nb, generator=gen, device=DEV) * 1e-3 + 1e-4
        s["r_scale"] = torch.rand(nb, generator=gen, device=DEV) * 2e-3 + 1e-4
    if own:
        from combine_moe_route_03_gb300 import api
        piece = lambda flat: [flat[o:o + n] for o, n in zip(at, sizes)]  # noqa: E731
        opt = api.AdamW(piece(s["p"]), lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY,
                        state_bits=case["bits"], copies=piece(s["copy"]))
        for name in ("m", "v") if case["bits"] == 32 else ("m_code", "r_code", "m_scale", "r_scale"):
            getattr(opt, name).copy_(s.pop(name))
        s["opt"], s["grads"] = opt, piece(s["g"])
    return s


# ------------------------------------------------------------------------- run
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from combine_moe_route_03_gb300 import api
    case = s["case"]
    op = case["op"]
    if op == "adamw":
        s["opt"].step(s["grads"])
        m, v = s["opt"].state()
        return dict(p=s["p"], copy=s["copy"], m=m, v=v)
    seg = dict(counts=s["counts"], align=case["align"])
    if op == "fwd":
        return api.grouped_gemm(s["x"], s["w"], out=s["out"], **seg)
    if op == "dgrad":
        return api.grouped_gemm(s["x"], s["w"], trans=True, out=s["out"], **seg)
    if op == "wgrad":
        if "acc" in s:
            return api.grouped_wgrad(s["dy"], s["x"], out=s["acc"], accumulate=True, **seg)
        return api.grouped_wgrad(s["dy"], s["x"], out=s["out"], **seg)
    if op == "swiglu":
        return api.swiglu(s["gu"], row_w=s["row_w"], out=s["h"], **seg)
    dgu, drow_w = api.swiglu_backward(s["gu"], s["dh"], row_w=s["row_w"], dgu=s["dgu"], drow_w=s["drow_w"], **seg)
    return dict(dgu=dgu, drow_w=drow_w)


def _live(s):
    """Which rows hold data, and for each (expert, place in its segment) the row and
    whether there is one."""
    counts, align = s["counts"].long(), s["case"]["align"]
    size = (counts + align - 1) // align * align
    place = torch.arange(s["longest"], device=DEV)
    has = place[None] < counts[:, None]
    at = (torch.cumsum(size, 0) - size)[:, None] + place[None]
    live = torch.zeros(s["rows"], dtype=torch.bool, device=DEV)
    live[at[has]] = True
    return live, at.clamp(max=s["rows"] - 1), has


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "adamw":
        return _adamw_plain(s)
    live, at, has = _live(s)
    part = lambda t: torch.where(has[..., None], t.float()[at], 0.0)  # noqa: E731  [E][longest][cols]
    if op in ("fwd", "dgrad"):
        w = s["w"].float()
        y = torch.bmm(part(s["x"]), w.transpose(1, 2) if op == "fwd" else w)
        s["out"][at[has]] = y[has].to(s["out"].dtype)
        return s["out"]
    if op == "wgrad":
        dw = torch.bmm(part(s["dy"]).transpose(1, 2), part(s["x"]))
        if "acc" in s:
            return s["acc"].add_(dw)
        return s["out"].copy_(dw)
    I = case["I"]
    g, u = s["gu"].float().split(I, dim=1)
    sig = 1.0 / (1.0 + torch.exp(-g))
    a = g * sig
    w = 1.0 if s["row_w"] is None else s["row_w"][:, None]
    if op == "swiglu":
        s["h"][live] = (w * a * u)[live].to(s["h"].dtype)
        return s["h"]
    dh = s["dh"].float()
    d = torch.cat((w * dh * u * (sig + a * (1.0 - sig)), w * dh * a), dim=1)
    s["dgu"][live] = d[live].to(s["dgu"].dtype)
    if s["row_w"] is not None:
        s["drow_w"][live] = (dh * a * u).sum(1)[live]
    return dict(dgu=s["dgu"], drow_w=s["drow_w"])


def _decode(s):
    q = (s["m_code"].float() * (1.0 / 127)).view(-1, BLOCK)
    m = q * q.abs() * s["m_scale"][:, None]
    t = (s["r_code"].float() * (1.0 / 255)).view(-1, BLOCK)
    r = t * t * s["r_scale"][:, None]
    return m.view(-1), (r * r).view(-1)


def _encode(x, levels):
    """Square-law codes of the blocks of x >= 0: the whole number c whose interval
    [(c - 1/2)^2, (c + 1/2)^2) holds levels^2 x / s."""
    b = x.view(-1, BLOCK)
    scale = b.amax(1)
    inv = torch.where(scale >= 2.0 ** -126, 1.0 / scale, torch.zeros_like(scale))
    z = b * inv[:, None] * float(levels * levels)
    c = torch.round(torch.sqrt(z))
    low, high = (c - 0.5) * (c - 0.5), (c + 0.5) * (c + 0.5)
    c = c - ((z < low) & (c > 0)).float() + (z >= high).float()
    return c.clamp(max=float(levels)).view(-1), scale


def _adamw_plain(s):
    case = s["case"]
    s["t"] += 1
    m, v = (s["m"], s["v"]) if case["bits"] == 32 else _decode(s)
    g = s["g"].float()
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + g * g * (1.0 - BETA2)
    r = torch.sqrt(v)
    denom = r * (1.0 / math.sqrt(1.0 - BETA2 ** s["t"])) + EPS
    s["p"].mul_(1.0 - LR * DECAY).sub_(m / denom * (LR / (1.0 - BETA1 ** s["t"])))
    s["copy"].copy_(s["p"])
    if case["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return dict(p=s["p"], copy=s["copy"], m=s["m"], v=s["v"])
    c, s["m_scale"] = _encode(m.abs(), 127)
    s["m_code"] = (c * torch.sign(m)).to(torch.int8)
    c, s["r_scale"] = _encode(r, 255)
    s["r_code"] = torch.where(r > 0, c.clamp(min=1.0), c).to(torch.uint8)
    m, v = _decode(s)
    return dict(p=s["p"], copy=s["copy"], m=m, v=v)


# ------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    b = 2
    if op == "adamw":
        n = sum(_sizes(case))
        states = 16 if case["bits"] == 32 else 4 + 8 + 16 / BLOCK  # codes in and out, values out
        return dict(bytes=n * (8 + 2 * b + states), flops=14 * n)
    R = case["rows"]
    if op.startswith("swiglu"):
        cols = 3 if op == "swiglu" else 5
        return dict(bytes=R * case["I"] * cols * b + 4 * R * (2 if case["weights"] else 0),
                    flops=R * case["I"] * (8 if op == "swiglu" else 18))
    E, n, k = case["E"], case["n"], case["k"]
    used = int((_counts(case, 1) > 0).sum())    # experts that have rows, for one seed
    flops = 2 * R * n * k
    if op == "wgrad":
        per = 8 if case["out"] == "f32" else b
        return dict(bytes=R * (n + k) * b + (used if per == 8 else E) * n * k * per, flops=flops)
    return dict(bytes=R * (n + k) * b + used * n * k * b, flops=flops)


# ----------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions in 64 bits, expert by expert."""
    s = prepare(dict(case), seed)
    op = case["op"]
    if op == "adamw":
        return _exact_adamw(case, s)
    counts, first, segments = s["counts"].tolist(), 0, []
    for c in counts:
        segments.append((first, first + c))
        first += -(-c // case["align"]) * case["align"]
    if op in ("fwd", "dgrad"):
        out = s["out"].double()
        for (lo, hi), w in zip(segments, s["w"]):
            if hi > lo:
                out[lo:hi] = s["x"][lo:hi].double() @ (w.double().t() if op == "fwd" else w.double())
        return out
    if op == "wgrad":
        out = s["acc"].double() if "acc" in s else torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        for e, (lo, hi) in enumerate(segments):
            if hi > lo:
                out[e] += s["dy"][lo:hi].double().t() @ s["x"][lo:hi].double()
        return out
    I = case["I"]
    h = torch.zeros(s["rows"], I, dtype=torch.float64, device=DEV)
    dgu = torch.zeros(s["rows"], 2 * I, dtype=torch.float64, device=DEV)
    drow = torch.zeros(s["rows"], dtype=torch.float64, device=DEV)
    for lo, hi in segments:
        g, u = s["gu"][lo:hi, :I].double(), s["gu"][lo:hi, I:].double()
        w = s["row_w"][lo:hi, None].double() if case["weights"] else 1.0
        sig = torch.special.expit(g)
        if op == "swiglu":
            h[lo:hi] = w * u * g * sig
            continue
        dh = s["dh"][lo:hi].double()
        dgu[lo:hi, :I] = w * dh * u * sig * (1 + g * torch.special.expit(-g))
        dgu[lo:hi, I:] = w * dh * g * sig
        drow[lo:hi] = torch.einsum("rc,rc->r", dh, u * g * sig)
    if op == "swiglu":
        return h
    return dict(dgu=dgu, drow_w=drow if case["weights"] else None)


def _exact_adamw(case, s):
    if case["bits"] == 32:
        m, r2 = s["m"].double(), s["v"].double()
    else:
        rep = lambda t: t.double().repeat_interleave(BLOCK)  # noqa: E731
        q = s["m_code"].double() / 127
        m = torch.sign(q) * q ** 2 * rep(s["m_scale"])
        r2 = ((s["r_code"].double() / 255) ** 2 * rep(s["r_scale"])) ** 2
    g = s["g"].double()
    m = BETA1 * m + (1 - BETA1) * g
    r2 = BETA2 * r2 + (1 - BETA2) * g ** 2
    p = s["p"].double()
    p = p - LR * DECAY * p - LR * (m / (1 - BETA1)) / (torch.sqrt(r2 / (1 - BETA2)) + EPS)
    if case["bits"] == 32:
        return dict(p=p, copy=p, m=m, v=r2)
    return dict(p=p, copy=p, m=None, v=None)
