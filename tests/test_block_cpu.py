"""The entry points for operators around the experts without a GPU: structure layout, host
argument checks, and the binding's refusals."""
import ctypes
import os

import pytest
import torch

from combine_moe_route_03_gb300 import _lib, api, configs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P16, P2 = 4096, 4098   # addresses: 16-byte aligned, and not
INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def L():
    from combine_moe_route_03_gb300 import build
    build.build()
    return _lib.load()


STRUCTS = {"NormArgs": "moe_norm_args", "NormGradArgs": "moe_norm_grad_args",
           "LinearArgs": "moe_linear_args", "ActGradArgs": "moe_act_grad_args",
           "LinearGradArgs": "moe_linear_grad_args"}


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


def make(cls, **kw):
    a = cls()
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_norm_refusals(L):
    ok = dict(rows=10, H=256, eps=1e-6, type=0, res_type=0, fmt=1, x=P16, w=P16, y=P16)
    call = lambda **kw: L.moe_rms_norm(ctypes.byref(make(_lib.NormArgs, **{**ok, **kw})), None)  # noqa: E731
    assert L.moe_rms_norm(None, None) == INVALID
    for kw in (dict(rows=-1), dict(H=0), dict(eps=-1e-6), dict(eps=float("nan")), dict(type=2), dict(type=-1),
               dict(res_type=1), dict(res_type=3), dict(fmt=3), dict(fmt=-1), dict(x=None), dict(w=None), dict(y=None),
               dict(x=P16 + 1), dict(w=P2), dict(y=P16 + 1), dict(sum=P16), dict(A=P16), dict(A_sf=P16),
               dict(residual=P2, res_type=2), dict(residual=P16, sum=P2, res_type=2),
               dict(fmt=0), dict(fmt=0, A=P16), dict(fmt=2, A_sf=P16), dict(fmt=0, A=P2, A_sf=P16),
               dict(fmt=0, A=P16, A_sf=P2), dict(fmt=0, A=P16, A_sf=P16, x=P2), dict(fmt=2, A=P16, A_sf=P16, w=P16 + 4)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(H=16385), dict(rows=2 ** 31), dict(fmt=0, A=P16, A_sf=P16, H=192)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(rows=0, x=None, w=None, y=None) == 0


def test_norm_backward_refusals(L):
    ok = dict(rows=10, H=256, eps=1e-6, type=0, res_type=0, h=P16, dy=P16, w=P16, dx=P16, dw=P16)

    def call(ws=P16, size=1 << 40, **kw):
        return L.moe_rms_norm_backward(ctypes.byref(make(_lib.NormGradArgs, **{**ok, **kw})), ws, size, None)
    assert L.moe_rms_norm_backward(None, P16, 1 << 40, None) == INVALID
    for kw in (dict(rows=-1), dict(H=-8), dict(eps=-1.0), dict(type=2), dict(res_type=1), dict(h=None), dict(dy=None),
               dict(w=None), dict(dx=None), dict(h=P2, res_type=2), dict(dres=P16 + 1), dict(dw=P2), dict(ws=None),
               dict(ws=P2), dict(size=0)):
        assert call(**kw) == INVALID, kw
    assert call(H=16385) == UNSUPPORTED
    assert call(rows=0, dw=None, h=None) == 0
    assert call(rows=0, accumulate=1, h=None) == 0
    for kw in (dict(), dict(H=1001), dict(H=16384, rows=100000)):   # without a GPU: as for one SM and more
        assert L.moe_rms_norm_workspace_size(ctypes.byref(make(_lib.NormGradArgs, **{**ok, **kw}))) % 4 == 0
    for kw in (dict(rows=0), dict(H=0), dict(type=5)):
        assert L.moe_rms_norm_workspace_size(ctypes.byref(make(_lib.NormGradArgs, **{**ok, **kw}))) == 0
    assert L.moe_rms_norm_workspace_size(None) == 0


def topk_cfg(**kw):
    return _lib.RouteCfg(*[{**dict(B=4, H=0, N=32, K=4, n_group=1, topk_group=1, score_fn=1, renorm=1, route_scale=1.0),
                            **kw}[f] for f, _ in _lib.RouteCfg._fields_])


BAD_TOPK = [(dict(B=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(score_fn=2), INVALID),
            (dict(N=513), UNSUPPORTED), (dict(N=64, K=17), UNSUPPORTED), (dict(N=3), UNSUPPORTED),
            (dict(n_group=3, topk_group=1), UNSUPPORTED), (dict(n_group=32, topk_group=4), UNSUPPORTED),
            (dict(n_group=4, topk_group=0), UNSUPPORTED), (dict(n_group=4, topk_group=5), UNSUPPORTED),
            (dict(n_group=8, topk_group=1, K=5), UNSUPPORTED)]


def test_route_topk_refusals(L):
    def call(type=2, z=P16, bias=None, idx=P16, w=P16, counts=None, **kw):
        return L.moe_route_topk(ctypes.byref(topk_cfg(**kw)), type, z, bias, idx, w, counts, None)
    assert L.moe_route_topk(None, 2, P16, None, P16, P16, None, None) == INVALID
    for kw, rc in BAD_TOPK:
        assert call(**kw) == rc, kw
    for kw in (dict(type=3), dict(type=-1), dict(z=None), dict(idx=None), dict(w=None), dict(z=P2), dict(type=0, z=P16 + 1),
               dict(idx=P2), dict(w=P2), dict(counts=P2), dict(bias=P2), dict(bias=P16, score_fn=0)):
        assert call(**kw) == INVALID, kw
    assert call(B=0, z=None, idx=None, w=None) == 0


def test_route_topk_backward_refusals(L):
    def call(type=2, z=P16, idx=P16, dw=P16, out_type=2, out=P16, **kw):
        return L.moe_route_topk_backward(ctypes.byref(topk_cfg(**kw)), type, z, idx, dw, out_type, out, None)
    for kw, rc in BAD_TOPK:
        assert call(**kw) == rc, kw
    for kw in (dict(type=3), dict(type=0, out_type=1), dict(type=1, out_type=0), dict(out_type=3), dict(z=None),
               dict(idx=None), dict(dw=None), dict(out=None), dict(out=P2), dict(dw=P2), dict(idx=P2)):
        assert call(**kw) == INVALID, kw
    assert call(B=0, z=None, idx=None, dw=None, out=None) == 0


def test_binding_refuses_norm_arguments():
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256)
    for kw in (dict(w=torch.ones(255)), dict(w=w.bfloat16()), dict(x=x.float()), dict(residual=x[:3]), dict(residual=x.half()),
               dict(y16=False), dict(fmt=7), dict(fmt=api.FMT_FP8_F32, out=dict(A=torch.zeros(4, 256, dtype=torch.uint8))),
               dict(out=dict(y=x.float())), dict(residual=x, out=dict(residual=x.float()))):
        with pytest.raises(ValueError):
            api.rms_norm(**{**dict(x=x, w=w), **kw})
    with pytest.raises(TypeError):
        api.rms_norm(None, w)
    with pytest.raises(ValueError, match="device parameter"):
        api.rms_norm(x, w)                                       # host tensors
    for kw in (dict(h=x[:2]), dict(h=x.half()), dict(dres=x.float()), dict(dx=x.float()), dict(dw=torch.ones(3)),
               dict(accumulate=True), dict(w=w[:8])):
        with pytest.raises(ValueError):
            api.rms_norm_backward(**{**dict(h=x, w=w, dy=x), **kw})


def test_binding_refuses_routing_arguments():
    cfg = configs.TINY
    z, i, d = torch.zeros(4, cfg.N), torch.zeros(4, cfg.K, dtype=torch.int32), torch.zeros(4, cfg.K)
    for a in ((z[:, :4],), (z.double(),), (z.int(),), (z, torch.zeros(cfg.N - 1)), (z, torch.zeros(cfg.N).half())):
        with pytest.raises(ValueError):
            api.route_topk(cfg, *a)
    for a, kw in (((z, i[:2], d), {}), ((z, i.long(), d), {}), ((z, i, d.half()), {}), ((z.half(), i, d), dict(out_dtype=torch.bfloat16)),
                  ((z, i, d), dict(out=torch.zeros(4, 3))), ((z, i, d), dict(out=z, out_dtype=torch.float16))):
        with pytest.raises(ValueError):
            api.route_topk_backward(cfg, *a, **kw)


def test_linear_refusals(L):
    ok = dict(rows=10, n=16, k=24, trans=0, type=0, out_type=0, act=0, x=P16, w=P16, out=P16)
    call = lambda **kw: L.moe_linear(ctypes.byref(make(_lib.LinearArgs, **{**ok, **kw})), None)  # noqa: E731
    assert L.moe_linear(None, None) == INVALID
    for kw in (dict(rows=-1), dict(n=0), dict(k=-8), dict(trans=2), dict(type=2), dict(type=-1), dict(out_type=1), dict(out_type=3),
               dict(act=4), dict(act=-1), dict(x=None), dict(w=None), dict(out=None), dict(x=P2), dict(w=P2), dict(out=P2),
               dict(residual=P2), dict(pre=P2), dict(bias=P2)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(n=12), dict(k=20), dict(n=2 ** 24 + 8), dict(k=2 ** 24 + 8), dict(n=2 ** 20, k=2 ** 18), dict(rows=2 ** 31 - 1)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(rows=0, x=None, w=None, out=None) == 0


def test_act_backward_refusals(L):
    ok = dict(rows=10, n=16, type=0, act=2, dy=P16, pre=P16, dz=P16, dbias=P16)

    def call(ws=P16, size=1 << 40, **kw):
        return L.moe_act_backward(ctypes.byref(make(_lib.ActGradArgs, **{**ok, **kw})), ws, size, None)
    assert L.moe_act_backward(None, P16, 1 << 40, None) == INVALID
    for kw in (dict(rows=-1), dict(n=0), dict(type=2), dict(act=4), dict(act=-1), dict(dy=None), dict(pre=None), dict(dz=None),
               dict(dy=P16 + 1), dict(dbias=P2), dict(ws=None), dict(ws=P2), dict(size=0), dict(act=0), dict(act=0, dz=None, dbias=None)):
        assert call(**kw) == INVALID, kw
    assert call(n=2 ** 24 + 1) == UNSUPPORTED and call(rows=2 ** 31 - 1) == UNSUPPORTED
    assert call(rows=0, dbias=None) == 0 and call(rows=0, accumulate=1) == 0
    assert L.moe_act_backward_workspace_size(None) == 0
    assert L.moe_act_backward_workspace_size(ctypes.byref(make(_lib.ActGradArgs, **{**ok, "rows": 0}))) == 0


def test_linear_backward_refusals(L):
    ok = dict(rows=10, n=16, k=24, type=0, dw_type=0, act=2, dy=P16, x=P16, w=P16, pre=P16, dx=P16, dw=P16, dbias=P16)

    def call(ws=P16, size=1 << 40, **kw):
        return L.moe_linear_backward(ctypes.byref(make(_lib.LinearGradArgs, **{**ok, **kw})), ws, size, None)
    assert L.moe_linear_backward(None, P16, 1 << 40, None) == INVALID
    for kw in (dict(rows=-1), dict(n=0), dict(k=0), dict(type=2), dict(dw_type=1), dict(dw_type=3), dict(act=4), dict(accumulate=1),
               dict(dy=None), dict(x=None), dict(w=None), dict(pre=None), dict(dy=P2), dict(x=P2), dict(w=P2), dict(pre=P16 + 1),
               dict(dx=P2), dict(dw=P2), dict(add=P2), dict(dbias=P2), dict(ws=None), dict(ws=P2), dict(size=0)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(n=12), dict(k=20), dict(n=2 ** 24 + 8), dict(k=2 ** 24 + 8), dict(n=2 ** 20, k=2 ** 18), dict(rows=2 ** 31 - 1)):
        assert call(**kw) == UNSUPPORTED, kw
    size = lambda **kw: L.moe_linear_backward_workspace_size(ctypes.byref(make(_lib.LinearGradArgs, **{**ok, **kw})))  # noqa: E731
    assert size(act=0, dbias=None) == 0 and size(rows=0) == 0 and size(n=0) == 0 and size(dbias=None) == 512
    assert L.moe_linear_backward_workspace_size(None) == 0


def test_binding_refuses_linear_arguments():
    x, w, y = torch.zeros(4, 16).bfloat16(), torch.zeros(24, 16).bfloat16(), torch.zeros(4, 24).bfloat16()
    for kw in (dict(x=x.half()), dict(w=w.float()), dict(x=y), dict(trans=True), dict(bias=torch.zeros(16)), dict(bias=y[0]),
               dict(act="tanh"), dict(residual=y.float()), dict(residual=y[:2]), dict(pre=y.float()), dict(out=y.half()),
               dict(out_dtype=torch.float16), dict(out=y, out_dtype=torch.float32), dict(residual=y, out_dtype=torch.float32),
               dict(status=torch.zeros(1))):
        with pytest.raises(ValueError):
            api.linear(**{**dict(x=x, w=w), **kw})
    with pytest.raises(ValueError, match="device parameter"):
        api.linear(x, w)
    for kw in (dict(act="gelu"), dict(act="silu", pre=x), dict(dz=y), dict(accumulate=True), dict(dbias=torch.zeros(3)),
               dict(act="relu", pre=y, dz=y.half())):
        with pytest.raises((ValueError, TypeError)):
            api.act_backward(y, **kw)
    for kw in (dict(dy=x), dict(add=y), dict(accumulate=True), dict(dw=torch.zeros(24, 16), dw_dtype=torch.bfloat16),
               dict(dw=torch.zeros(16, 24)), dict(dw=torch.zeros(24, 16), bias=True, accumulate=True), dict(w=w.half())):
        with pytest.raises(ValueError):
            api.linear_backward(**{**dict(dy=y, x=x, w=w), **kw})


def test_binding_refuses_norm_buffers_that_nothing_fills():
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256)
    for out in (dict(residual=x), dict(sum=x), dict(y=x, A=torch.zeros(128, 256, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="out: buffers for"):
            api.rms_norm(x, w, out=out)


def test_dense_tile_lists():
    t = api.dense_tiles(300, device="cpu").tolist()
    assert t[:8] == [3, 384, 1, 1, 2, 0, 0, 0]
    assert t[8:32] == [0, 0, 128, 0, 3, 0, 0, 0, 128, 0, 128, 0, 3, 0, 0, 0, 256, 0, 44, 0, 3, 0, 0, 0]
    assert t[32:48] == [0, 1, 0, 2, 1, 0, 0, 0, 2, -1, 0, 2, 0, 0, 0, 0] and len(t) == 8 + 16 * 3
    assert api.dense_tiles(0, device="cpu").tolist() == [0] * 8
    with pytest.raises(ValueError):
        api.dense_tiles(-1)


def test_a_layer_with_a_norm_refuses_calls_that_would_leave_it_out():
    lay = object.__new__(api.MoELayer)                            # built by hand: no GPU here
    lay.norm_w = torch.ones(8)
    buf = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: lay.forward_host(buf, buf), lambda: lay.forward_host_pipelined([buf], [buf]),
                 lambda: api.LayerGraph(lay, None), lambda: api.LayerGraph(lay, None, buf, buf)):
        with pytest.raises(ValueError, match="norm"):
            call()


@pytest.mark.parametrize("rows,H,res_type", [(8192, 7168, 0), (8192, 7168, 2), (100000, 16384, 0), (3, 16384, 2), (50, 512, 0),
                                             (9000, 1001, 2), (9000, 100, 0), (1, 1, 0)])
def test_norm_workspace_is_what_the_parts_take(L, rows, H, res_type):
    """A part of dw a block, and at most 8 blocks an SM."""
    size = L.moe_rms_norm_workspace_size(ctypes.byref(make(_lib.NormGradArgs, rows=rows, H=H, eps=1e-6, type=0, res_type=res_type)))
    assert 4 * H <= size <= 4 * H * min(rows, 8 * L.moe_num_sms())
