"""CPU-side checks of the norm's, the router's and the 4-bit layer's entry
points: sizes, and arguments refused on the host before any launch. No kernel
is launched here."""
import ctypes

import pytest

from combine_get_layout_amd import ep
from test_experts_abi import ODD, P, OnDevice, StreamOf, lib, refused, shape  # noqa: F401 (fixtures)

byref = ctypes.byref
NAN, INF = float("nan"), float("inf")


def test_norm_refusals(lib, shape):
    O = ep.ep_norm_out

    def call(s=shape, x=P, res=P, kind=0, gain=P, eps=1e-6, out=O(P, P, P, P, P)):
        return lib.ep_rms_norm(byref(s) if s else None, x, res, kind, gain, eps, byref(out) if out else None, None)

    for bad in (dict(s=None), dict(x=None), dict(gain=None), dict(kind=2), dict(kind=-1), dict(eps=0.0), dict(eps=-1e-6),
                dict(eps=NAN), dict(eps=INF), dict(out=None), dict(out=O()), dict(out=O(P, P, P, None, P)),
                dict(out=O(P, P, None, P, P)), dict(x=ODD), dict(res=ODD), dict(gain=ODD), dict(out=O(ODD)),
                dict(out=O(None, ODD)), dict(out=O(None, None, ODD, P)), dict(out=O(None, None, P, P + 2)),
                dict(out=O(None, None, None, None, P + 2)), dict(s=ep.make_shape(4, 200, 1, 1, 1)),
                dict(s=ep.make_shape(4, 12, 1, 1, 1), out=O(P)), dict(s=ep.make_shape(-1, 256, 1, 1, 1))):
        refused(call(**bad))
    refused(call(s=ep.make_shape(4, (1 << 20) + 128, 1, 1, 1)), ep.EP_ERR_UNSUPPORTED)
    # Without tokens nothing is read or written.
    assert call(s=ep.make_shape(0, 256, 1, 1, 1), x=None, res=None, gain=None, out=O()) == ep.EP_OK


def test_norm_grad_refusals_and_workspace(lib, shape):
    n = ep.ep_norm_workspace_bytes(shape)
    assert n >= 256 + 4 * shape.H and n % 256 == 0

    def call(s=shape, h=P, kind=0, gain=P, r=P, dy=P, ds=P, dh=P + 256, dx=P + 512, dg=P, ws=P, wsb=n):
        return lib.ep_rms_norm_grad(byref(s), h, kind, gain, r, dy, ds, dh, dx, dg, ws, wsb, None)

    for bad in (dict(h=None), dict(gain=None), dict(r=None), dict(dy=None), dict(dh=None, dx=None, dg=None), dict(kind=2),
                dict(h=ODD), dict(gain=ODD), dict(r=P + 2), dict(dy=ODD), dict(ds=ODD), dict(dh=ODD), dict(dx=ODD),
                dict(dg=ODD), dict(ws=None), dict(ws=P + 16), dict(wsb=n - 1), dict(s=ep.make_shape(32, 252, 2, 8, 1)),
                dict(h=P + 256), dict(h=P + 512), dict(dy=P + 256), dict(dy=P + 512), dict(gain=P + 256), dict(gain=P + 512)):
        refused(call(**bad))
    refused(call(s=ep.make_shape(4, (1 << 20) + 8, 1, 1, 1)), ep.EP_ERR_UNSUPPORTED)
    for s in (ep.make_shape(4, 250, 1, 1, 1), ep.make_shape(4, (1 << 20) + 8, 1, 1, 1)):
        assert ep.ep_norm_workspace_bytes(s) == 0
        with pytest.raises(RuntimeError):
            ep.alloc_norm_workspace(s)
    # The parts of the gain's gradient stay bounded however many tokens there are.
    assert ep.ep_norm_workspace_bytes(ep.make_shape(1 << 20, 8192, 1, 1, 1)) <= 256 + 4 * 8192 * 1024


def router(**f):
    return ep.ep_router(**{**dict(score=0, top_groups=1, group_top=1, normalize=1, scale=1.0), **f})


BAD_ROUTERS = (None, router(score=2), router(score=-1), router(top_groups=0), router(top_groups=2), router(group_top=0),
               router(group_top=3), router(normalize=2), router(normalize=-1), router(scale=NAN), router(scale=INF),
               router(bias=P + 2))


def test_route_refusals(lib, shape):
    def call(s=shape, l=P, r=router(bias=P), idx=P, w=P, ws=P, wsb=1 << 20):
        return lib.ep_route(byref(s), l, byref(r) if r else None, idx, w, ws, wsb, None)

    for r in BAD_ROUTERS:
        refused(call(r=r))
    for bad in (dict(l=None), dict(idx=None), dict(l=P + 2), dict(idx=ODD), dict(w=P + 2), dict(ws=None), dict(ws=P + 16),
                dict(wsb=16), dict(s=ep.make_shape(4, 250, 2, 8, 1))):
        refused(call(**bad))
    many = ep.make_shape(4, 256, 2, 256, 128, 128)
    refused(call(s=many, r=router(top_groups=3)), ep.EP_ERR_UNSUPPORTED)
    refused(call(s=ep.make_shape(4, 256, 65, 256, 1)), ep.EP_ERR_UNSUPPORTED)
    z = ep.make_shape(0, 256, 2, 8, 1)
    assert call(s=z, l=None, idx=None, w=None) == ep.EP_OK


def test_route_grad_refusals(lib, shape):
    def call(s=shape, l=P, r=router(), idx=P, dw=P, d=P, dtype=1, ws=P, wsb=1 << 20):
        return lib.ep_route_grad(byref(s), l, byref(r) if r else None, idx, dw, d, dtype, ws, wsb, None)

    for r in BAD_ROUTERS:
        refused(call(r=r))
    for bad in (dict(l=None), dict(idx=None), dict(dw=None), dict(d=None), dict(dtype=2), dict(dtype=-1), dict(l=P + 2),
                dict(idx=ODD), dict(dw=P + 2), dict(d=ODD), dict(ws=None), dict(ws=P + 16), dict(wsb=16)):
        refused(call(**bad))
    z = ep.make_shape(0, 256, 2, 8, 1)
    assert call(s=z, l=None, idx=None, dw=None, d=None) == ep.EP_OK


def test_few_w4_refusals_and_workspace(lib, shape):
    X = ep.ep_experts_w4

    def call(s=shape, tk=ep.ep_tokens(P, None, None, P, P), x=X(128, 0, P, P, P, P), out=P, ws=P, wsb=1 << 30):
        return lib.ep_moe_few_w4(byref(s), byref(tk) if tk else None, byref(x) if x else None, out, ws, wsb, None)

    for bad in (dict(x=None), dict(tk=None), dict(x=X(0, 0, P, P, P, P)), dict(x=X(96, 0, P, P, P, P)),
                dict(x=X(128, 2, P, P, P, P)), dict(x=X(128, -1, P, P, P, P)), dict(x=X(16, 1, P, P, P, P)),
                dict(x=X(48, 1, P, P, P, P)), dict(x=X(-32, 1, P, P, P, P)), dict(x=X(128, 0, None, P, P, P)),
                dict(x=X(128, 0, P, None, P, P)), dict(x=X(128, 0, P, P, None, P)), dict(x=X(128, 0, P, P, P, None)),
                dict(x=X(128, 0, ODD, P, P, P)), dict(x=X(128, 0, P, ODD, P, P)), dict(x=X(128, 1, P, P, ODD, P)),
                dict(x=X(128, 1, P, P, P, ODD)), dict(tk=ep.ep_tokens(None, None, None, P, P)),
                dict(tk=ep.ep_tokens(P, None, None, None, P)), dict(tk=ep.ep_tokens(P, None, None, P, None)),
                dict(tk=ep.ep_tokens(ODD, None, None, P, P)), dict(out=None), dict(out=ODD), dict(ws=None),
                dict(ws=P + 16), dict(wsb=256), dict(s=ep.make_shape(32, 224, 2, 8, 1)),
                dict(s=ep.make_shape(32, 208, 2, 8, 1), x=X(128, 1, P, P, P, P))):
        refused(call(**bad))
    refused(call(s=ep.make_shape(129, 256, 2, 8, 1)), ep.EP_ERR_UNSUPPORTED)
    refused(call(x=X((1 << 20) + 128, 0, P, P, P, P)), ep.EP_ERR_UNSUPPORTED)
    refused(call(s=ep.make_shape(4, (1 << 20) + 128, 2, 8, 1)), ep.EP_ERR_UNSUPPORTED)
    refused(call(s=ep.make_shape(128, 256, 4, 8, 1), x=X(1 << 20, 0, P, P, P, P)), ep.EP_ERR_UNSUPPORTED)
    n = ep.ep_few_w4_workspace_bytes(shape, 128)
    assert n >= 256 + 32 * 2 * 128 * 2 and n % 256 == 0
    refused(call(wsb=n - 1))
    for s, F in ((ep.make_shape(129, 256, 2, 8, 1), 128), (shape, 0), (shape, (1 << 20) + 32),
                 (ep.make_shape(128, 256, 4, 8, 1), 1 << 20)):
        assert ep.ep_few_w4_workspace_bytes(s, F) == 0
    with pytest.raises(RuntimeError):
        ep.alloc_few_w4_workspace(ep.make_shape(129, 256, 2, 8, 1), 128)


ROUTER = dict(score=0)
FOUR = dict(F=128, form=0, w13=P, w13_scales=P, w2=P, w2_scales=P)
CALLS = dict(
    grad_h=lambda s, t, ws, st: ep.ep_rms_norm_grad(s, t, 0, P, P, P, P, P, P, P, ws, stream=st),
    grad_gain=lambda s, t, ws, st: ep.ep_rms_norm_grad(s, P, 0, P, P, P, P, P, P, t, ws, stream=st),
    route=lambda s, t, ws, st: ep.ep_route(s, t, ROUTER, P, P, ws, stream=st),
    route_bias=lambda s, t, ws, st: ep.ep_route(s, P + 2, dict(ROUTER, bias=t), P, P, ws, stream=st),
    route_idx=lambda s, t, ws, st: ep.ep_route(s, P + 2, ROUTER, t, P, ws, stream=st),
    route_grad=lambda s, t, ws, st: ep.ep_route_grad(s, P, ROUTER, P, P, t, 1, ws, stream=st),
    few=lambda s, t, ws, st: ep.ep_moe_few_w4(s, dict(x=t, topk_idx=P, topk_weights=P), FOUR, P, ws, stream=st),
    few_scales=lambda s, t, ws, st: ep.ep_moe_few_w4(s, dict(x=P, topk_idx=P, topk_weights=P), dict(FOUR, w2_scales=t), P,
                                                     ws, stream=st),
    norm=lambda s, t, x, st: ep.ep_rms_norm(s, x, t, 0, P, 1e-6, dict(y=P), stream=st),
    norm_out=lambda s, t, x, st: ep.ep_rms_norm(s, x, None, 0, P, 1e-6, dict(y=t), stream=st),
)


@pytest.mark.parametrize("name", CALLS)
def test_binding_refuses_tensors_of_another_device(lib, shape, monkeypatch, name):
    """As for the expert operators: tensors, workspace (of the norm: x) and stream on one device."""
    import torch

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x30 + device)
    monkeypatch.setattr(torch, "Tensor", (torch.Tensor, OnDevice))
    call = CALLS[name]
    for stream, own, other in ((None, 0, 1), (StreamOf(1), 1, 0), (0, 0, 1)):
        for devices in ((other, own), (own, other), (other, other)):
            with pytest.raises(ValueError, match="device"):
                call(shape, OnDevice(devices[0]), OnDevice(devices[1]), stream)
        with pytest.raises(RuntimeError, match="invalid|argument"):
            call(shape, OnDevice(own), OnDevice(own), stream)


def test_binding_refuses_host_and_short_tensors(lib, shape):
    import torch

    t = torch.zeros(8)
    with pytest.raises(ValueError, match="GPU tensor"):
        ep.ep_rms_norm(shape, t, None, 0, P, 1e-6, dict(y=P))
    with pytest.raises(ValueError, match="GPU tensor"):
        ep.ep_route(shape, t, ROUTER, P, P, t)
    with pytest.raises(ValueError, match="GPU tensor"):
        ep.ep_moe_few_w4(shape, dict(x=t, topk_idx=P, topk_weights=P), FOUR, P, t)


class Short(OnDevice):
    """A tensor one byte shorter than the call needs."""
    def __init__(self, need):
        super().__init__(0)
        self.need = need

    def numel(self):
        return self.need - 1


@pytest.mark.parametrize("form", [0, 1], ids=["int", "e2m1"])
def test_binding_knows_the_sizes(lib, monkeypatch, form):
    import torch

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x30)
    monkeypatch.setattr(torch, "Tensor", (torch.Tensor, OnDevice))
    T, H, K, E, F = 6, 384, 2, 8, 256
    s, ws = ep.make_shape(T, H, K, E, 1), OnDevice(0)
    per, size = (128, 2) if form == 0 else (32, 1)
    for name, need in dict(w13=E * 2 * F * H // 2, w2=E * H * F // 2, w13_scales=E * 2 * F * (H // per) * size,
                           w2_scales=E * H * (F // per) * size).items():
        with pytest.raises(ValueError, match=f"{name}: .* needs {need}"):
            ep.ep_moe_few_w4(s, dict(x=P, topk_idx=P, topk_weights=P), dict(FOUR, F=F, form=form, **{name: Short(need)}), P, ws)
    wide = form == 1
    w = 4 if wide else 2
    for name, need in dict(h=w * T * H, y=2 * T * H, y_fp8=T * H, y_scales=4 * T * H // 128, rstd=4 * T).items():
        with pytest.raises(ValueError, match=f"{name}: .* needs {need}"):
            ep.ep_rms_norm(s, OnDevice(0), P, int(wide), P, 1e-6, {name: Short(need)})
    with pytest.raises(ValueError, match=f"residual: .* needs {w * T * H}"):
        ep.ep_rms_norm(s, OnDevice(0), Short(w * T * H), int(wide), P, 1e-6, dict(y=P))
    for at, need in ((1, 4 * T * E), (3, 8 * T * K), (4, 4 * T * K)):
        args = [s, P + 2, ROUTER, P, P, ws]
        args[at] = Short(need)
        with pytest.raises(ValueError, match=f"needs {need}"):
            ep.ep_route(*args)
    with pytest.raises(ValueError, match=f"d_logits: .* needs {w * T * E}"):
        ep.ep_route_grad(s, P, ROUTER, P, P, Short(w * T * E), int(wide), ws)
