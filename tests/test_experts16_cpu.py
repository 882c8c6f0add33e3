"""The entry points for experts in 16-bit storage without a GPU: structure layout, host
argument checks, and the binding's refusals."""
import ctypes
import os

import pytest
import torch

from combine_moe_route_03_gb300 import _lib, api

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P16, P2 = 4096, 4098   # addresses: 16-byte aligned, and not


@pytest.fixture(scope="module")
def L():
    from combine_moe_route_03_gb300 import build
    build.build()
    return _lib.load()


STRUCTS = {"Segments": "moe_segments", "GgemmArgs": "moe_ggemm_args",
           "WgradArgs": "moe_wgrad_args", "SwigluArgs": "moe_swiglu_args",
           "AdamwCfg": "moe_adamw_cfg", "AdamwTensor": "moe_adamw_tensor"}


def test_binding_structs_match_the_c_layout(tmp_path):
    import subprocess
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "moe.h"', 'int main(void){']
    for py, c in STRUCTS.items():
        lines.append(f'printf("{py} . %zu %zu\\n", sizeof({c}), (size_t)0);')
        for f, _ in getattr(_lib, py)._fields_:
            lines.append(f'printf("{py} {f} %zu %zu\\n", offsetof({c}, {f}), sizeof((({c} *)0)->{f}));')
    lines.append("return 0;}")
    (tmp_path / "l.c").write_text("\n".join(lines) + "\n")
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                           str(tmp_path / "l.c"), "-o", str(tmp_path / "l")])
    for line in filter(None, subprocess.check_output([str(tmp_path / "l")], text=True).split("\n")):
        py, f, a, b = line.split()
        cls = getattr(_lib, py)
        if f == ".":
            assert ctypes.sizeof(cls) == int(a), py
        else:
            assert (getattr(cls, f).offset, getattr(cls, f).size) == (int(a), int(b)), (py, f)


INVALID, UNSUPPORTED = -1, -2
SEG = dict(counts=P16, E=4, align=1, cap=0, rows=100)


def seg(**kw):
    return _lib.Segments(*[{**SEG, **kw}[f] for f, _ in _lib.Segments._fields_])


def make(cls, **kw):
    a = cls()
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_SEGMENTS = [(dict(counts=None), INVALID), (dict(E=0), INVALID), (dict(E=1025), UNSUPPORTED),
                (dict(align=0), INVALID), (dict(cap=-1), INVALID), (dict(rows=-1), INVALID),
                (dict(rows=2 ** 31 - 1), UNSUPPORTED)]


def test_grouped_gemm_refusals(L):
    ok = dict(seg=seg(), n=16, k=24, trans=0, type=0, x=P16, w=P16, out=P16)
    call = lambda **kw: L.moe_grouped_gemm(ctypes.byref(make(_lib.GgemmArgs, **{**ok, **kw})), None)  # noqa: E731
    assert L.moe_grouped_gemm(None, None) == INVALID
    for kw, rc in BAD_SEGMENTS:
        assert call(seg=seg(**kw)) == rc, kw
    for kw in (dict(n=0), dict(k=-8), dict(trans=2), dict(type=2), dict(type=-1), dict(x=None), dict(w=None),
               dict(out=None), dict(x=P2), dict(w=P2), dict(out=P2)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(n=12), dict(k=20)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(seg=seg(rows=0), x=None, out=None) == 0       # no rows: nothing enqueued


def test_grouped_wgrad_refusals(L):
    ok = dict(seg=seg(), n=16, k=24, type=0, out_type=0, dy=P16, x=P16, out=P16)
    call = lambda **kw: L.moe_grouped_wgrad(ctypes.byref(make(_lib.WgradArgs, **{**ok, **kw})), None)  # noqa: E731
    assert L.moe_grouped_wgrad(None, None) == INVALID
    for kw, rc in BAD_SEGMENTS:
        assert call(seg=seg(**kw)) == rc, kw
    for kw in (dict(n=0), dict(type=2), dict(out_type=1), dict(out_type=3), dict(accumulate=1), dict(dy=None),
               dict(x=None), dict(out=None), dict(dy=P2), dict(x=P2), dict(out=P2)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(n=12), dict(k=20)):
        assert call(**kw) == UNSUPPORTED, kw


def test_default_status_refusals(L):
    assert L.moe_read_default_status(None, 0) == INVALID


def test_swiglu_refusals(L):
    ok = dict(seg=seg(), I=16, type=0, gu=P16, out=P16)
    for name, more in (("moe_swiglu", {}), ("moe_swiglu_backward", dict(dh=P16, drow_w=P16))):
        f = getattr(L, name)
        call = lambda **kw: f(ctypes.byref(make(_lib.SwigluArgs, **{**ok, **more, **kw})), None)  # noqa: E731
        assert f(None, None) == INVALID
        for kw, rc in BAD_SEGMENTS[1:]:
            assert call(seg=seg(**kw)) == rc, kw
        for kw in (dict(I=0), dict(type=2), dict(gu=None), dict(out=None), dict(gu=P16 + 1), dict(row_w=P2)):
            assert call(**kw) == INVALID, kw
        assert call(I=2 ** 24 + 1) == UNSUPPORTED
        assert call(seg=seg(rows=0), gu=None) == 0
    assert L.moe_swiglu(ctypes.byref(make(_lib.SwigluArgs, **ok, dh=P16)), None) == INVALID
    assert L.moe_swiglu_backward(ctypes.byref(make(_lib.SwigluArgs, **ok)), None) == INVALID


def test_adamw_refusals(L):
    cfg = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1, state_bits=32)
    ten = dict(n=10, p=P16, g=P16, m=P16, v=P16)

    def call(t={}, n=1, **kw):
        arr = (_lib.AdamwTensor * 1)(make(_lib.AdamwTensor, **{**ten, **t}))
        return L.moe_adamw(ctypes.byref(make(_lib.AdamwCfg, **{**cfg, **kw})), arr, n, None)
    arr = (_lib.AdamwTensor * 1)()
    assert L.moe_adamw(None, arr, 1, None) == INVALID
    assert L.moe_adamw(ctypes.byref(make(_lib.AdamwCfg, **cfg)), None, 1, None) == INVALID
    for kw in (dict(step=0), dict(state_bits=16), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0),
               dict(beta1=float("nan")), dict(grad_scale=P2), dict(n=-1)):
        assert call(**kw) == INVALID, kw
    for t in (dict(n=-1), dict(p=None), dict(g=None), dict(m=None), dict(v=None), dict(p=P2), dict(m=P2),
              dict(g_type=3), dict(copy=P16, copy_type=-1), dict(g=P2 + 1), dict(g=P2, g_type=2)):
        assert call(t) == INVALID, t
    assert call(state_bits=8) == INVALID                       # no scales
    assert call(dict(n=2 ** 41)) == UNSUPPORTED
    assert call(n=0) == 0 and call(dict(n=0, p=None)) == 0     # nothing to do
    for f in (L.moe_adamw_decode, L.moe_adamw_encode):
        assert f(0, *[None] * 7) == 0
        assert f(-1, *[None] * 7) == INVALID and f(5, *[None] * 7) == INVALID


def test_binding_refuses_host_tensors_and_shapes(L):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    c4 = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: api.swiglu(bf(4, 32), out=bf(4, 16)),
                 lambda: api.grouped_gemm(bf(8, 24), bf(4, 16, 24), c4, out=bf(8, 16),
                                          status=torch.zeros(1, dtype=torch.int32)),
                 lambda: api.AdamW([torch.zeros(4)])):
        with pytest.raises(ValueError, match="device parameter"):
            call()
    w = bf(4, 16, 24)
    for call in (lambda: api.grouped_gemm(bf(8, 16), w, c4),                          # k
                 lambda: api.grouped_gemm(bf(8, 24), w, c4, trans=True),              # n
                 lambda: api.grouped_gemm(bf(8, 24).half(), w, c4),                   # type
                 lambda: api.grouped_gemm(bf(8, 24), w.float(), c4),
                 lambda: api.grouped_gemm(bf(8, 24), w, c4[:3]),                      # experts
                 lambda: api.grouped_gemm(bf(8, 24), w, c4.long()),
                 lambda: api.grouped_gemm(bf(8, 24), w, c4, out=bf(7, 16)),
                 lambda: api.grouped_wgrad(bf(8, 16), bf(9, 24), c4),                 # rows
                 lambda: api.grouped_wgrad(bf(8, 16), bf(8, 24), c4, accumulate=True),
                 lambda: api.grouped_wgrad(bf(8, 16), bf(8, 24), c4, out=bf(4, 16, 24), accumulate=True),
                 lambda: api.grouped_wgrad(bf(8, 16), bf(8, 24), c4, out=bf(4, 24, 16)),
                 lambda: api.swiglu(bf(8, 15)),
                 lambda: api.swiglu(bf(8, 16), row_w=torch.zeros(7)),
                 lambda: api.swiglu_backward(bf(8, 16), bf(8, 16)),
                 lambda: api.AdamW([torch.zeros(4, dtype=torch.bfloat16)]),
                 lambda: api.AdamW([torch.zeros(4)], copies=[torch.zeros(5)]),
                 lambda: api.AdamW([torch.zeros(4)], copies=[]),
                 lambda: api.AdamW([torch.zeros(4)], state_bits=16),
                 lambda: api.AdamW([])):
        with pytest.raises(ValueError, match="expected"):
            call()


class Calls:
    """Stands in for the library: records the calls, touches nothing."""

    def __init__(self):
        self.names = []

    def __getattr__(self, name):
        return lambda *a: self.names.append(name) or 0


@pytest.fixture
def calls(monkeypatch):
    """The binding over host tensors and a library that only records."""
    c = Calls()
    address = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    monkeypatch.setattr(api, "load", lambda: c)
    monkeypatch.setattr(api, "ptr", address)
    monkeypatch.setattr(api, "ptrs", lambda *ts: ([address(t) for t in ts], 0))
    return c


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_refuses_tensors_that_moved(calls, bits):
    """A parameter, copy or moment whose storage was replaced: the step would write where it
    lay before."""
    def new():
        return api.AdamW([torch.zeros(3, 5), torch.zeros(300)], state_bits=bits,
                         copies=[torch.zeros(3, 5, dtype=torch.bfloat16), None])
    grads = [torch.zeros(3, 5), torch.zeros(300)]

    def data(t, value):
        t.data = value
    name = "v" if bits == 32 else "r_scale"
    for move in (lambda o: data(o.params[1], torch.zeros(300)),
                 lambda o: data(o.params[0], o.params[0].data.view(5, 3).t()),
                 lambda o: data(o.params[1], o.params[1].data[:200]),
                 lambda o: data(o.copies[0], torch.zeros(3, 5, dtype=torch.bfloat16)),
                 lambda o: data(o.copies[0], o.copies[0].data.view(torch.float16)),
                 lambda o: setattr(o, name, getattr(o, name).clone())):
        opt = new()
        opt.step(grads)
        assert calls.names.pop() == "moe_adamw" and opt.steps == 1
        move(opt)
        with pytest.raises(ValueError, match="expected"):
            opt.step([torch.zeros(p.shape) for p in opt.params])
        assert calls.names == [] and opt.steps == 1


def test_adamw_refuses_gradients_that_are_no_tensors(calls):
    opt = api.AdamW([torch.zeros(4), torch.zeros(5)])
    for bad in (None, 1.0, [0.0] * 5):
        with pytest.raises(TypeError, match="torch tensor"):
            opt.step([torch.zeros(4), bad])
    assert calls.names == [] and opt.steps == 0


def test_binding_refuses_what_is_no_tensor_and_other_status_words(calls):
    """Neither ends in an attribute error or reaches the library: the kernels write 32 bits."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    c4, w = torch.zeros(4, dtype=torch.int32), bf(4, 16, 24)
    for call in (lambda: api.grouped_gemm(None, w, c4), lambda: api.grouped_gemm(bf(8, 24), None, c4),
                 lambda: api.grouped_gemm(bf(8, 24), w, None), lambda: api.grouped_wgrad(None, bf(8, 24), c4),
                 lambda: api.grouped_wgrad(bf(8, 16), None, c4), lambda: api.swiglu(None),
                 lambda: api.swiglu_backward(None, bf(8, 16)), lambda: api.swiglu_backward(bf(8, 32), None)):
        with pytest.raises(TypeError, match="torch tensor"):
            call()
    for status in (torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.int16), torch.zeros(1),
                   torch.zeros(0, dtype=torch.int32)):
        for call in (lambda: api.grouped_gemm(bf(8, 24), w, c4, status=status),
                     lambda: api.grouped_wgrad(bf(8, 16), bf(8, 24), c4, status=status),
                     lambda: api.swiglu(bf(8, 32), counts=c4, status=status),
                     lambda: api.swiglu_backward(bf(8, 32), bf(8, 16), counts=c4, status=status)):
            with pytest.raises(ValueError, match="status"):
                call()
    assert calls.names == []
    api.grouped_gemm(bf(8, 24), w, c4, status=torch.zeros((), dtype=torch.int32))
    assert calls.names == ["moe_grouped_gemm"]
