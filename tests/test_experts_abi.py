"""CPU-side checks of the expert products' entry points: sizes, and arguments
refused on the host before any launch. No kernel is launched here."""
import ctypes
import os

import pytest

from combine_get_layout_amd import ep

P = 0x100000          # an aligned address that no call dereferences
ODD = P + 4           # 4 B aligned only
byref = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ep.LIB_PATH):
        from combine_get_layout_amd import build
        build.build()
    return ep.lib()


@pytest.fixture(scope="module")
def shape():
    return ep.make_shape(32, 256, 2, 8, 1)


def layout(**f):
    return ep.ep_layout(**f)


def refused(rc, want=ep.EP_ERR_ARG):
    assert rc == want, rc


def matmul(lib, s, L=None, x=P, rows=10, k=64, w=P, n=128, order=0, y=P, ws=P, wsb=None):
    L = layout(expert_offsets=P) if L is None else L
    return lib.ep_expert_matmul(byref(s), byref(L), x, rows, k, w, n, order, y, ws,
                                ep.ep_workspace_bytes(s) if wsb is None else wsb, None)


def test_matmul_refusals(lib, shape):
    refused(matmul(lib, shape, L=layout()))
    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(x=ODD), dict(w=ODD), dict(y=ODD), dict(k=60),
                dict(n=4), dict(k=0), dict(n=-8), dict(order=2), dict(order=-1), dict(rows=-1), dict(ws=None),
                dict(ws=P + 16), dict(wsb=16), dict(L=layout(expert_offsets=P + 2))):
        refused(matmul(lib, shape, **bad))
    for big in (dict(k=(1 << 20) + 8), dict(n=(1 << 20) + 8), dict(rows=1 << 31),
                dict(rows=(1 << 31) - 1, n=1 << 20)):
        refused(matmul(lib, shape, **big), ep.EP_ERR_UNSUPPORTED)
    assert lib.ep_expert_matmul(None, None, P, 1, 8, P, 8, 0, P, P, 1 << 20, None) == ep.EP_ERR_ARG
    assert lib.ep_expert_matmul(byref(shape), None, P, 1, 8, P, 8, 0, P, P, 1 << 20, None) == ep.EP_ERR_ARG


def test_swiglu_refusals(lib, shape):
    def call(s=shape, L=layout(expert_offsets=P), x=P, rows=10, w=P, F=128, act=P, q=P, sc=P, ws=P):
        return lib.ep_expert_swiglu(byref(s), byref(L), x, rows, w, F, act, q, sc, ws, ep.ep_workspace_bytes(s), None)

    for bad in (dict(L=layout()), dict(x=None), dict(w=None), dict(act=None), dict(q=None), dict(sc=None),
                dict(F=136), dict(F=12, q=None, sc=None), dict(F=0), dict(q=ODD), dict(sc=ODD), dict(act=ODD),
                dict(rows=-1), dict(ws=None)):
        refused(call(**bad))
    wide = ep.make_shape(32, 65536, 2, 8, 1)  # 4 F H passes 31 bits
    refused(call(s=wide, F=8192), ep.EP_ERR_UNSUPPORTED)
    refused(call(rows=1 << 31), ep.EP_ERR_UNSUPPORTED)


def test_swiglu_grad_refusals(lib, shape):
    def call(L=layout(expert_slot=P), F=128, q=P, sc=P, d=P, rows=10, w=P, dg=P, a=P, dw=P, ws=P):
        return lib.ep_swiglu_grad(byref(shape), byref(L), F, q, sc, d, rows, w, dg, a, dw, ws,
                                  ep.ep_workspace_bytes(shape), None)

    for bad in (dict(L=layout()), dict(F=64), dict(F=200), dict(q=None), dict(sc=None), dict(d=None), dict(w=None),
                dict(dg=None), dict(q=ODD), dict(sc=ODD), dict(d=ODD), dict(dg=ODD), dict(a=ODD), dict(w=P + 2),
                dict(dw=P + 2), dict(rows=-1), dict(ws=None)):
        refused(call(**bad))
    refused(call(rows=1 << 31), ep.EP_ERR_UNSUPPORTED)


def test_wgrad_refusals(lib, shape):
    def call(L=layout(expert_offsets=P), dy=P, rows=10, n=64, x=ep.ep_rows(P, None, None), k=128, dw=P, dtype=0, ws=P):
        return lib.ep_expert_wgrad(byref(shape), byref(L), dy, rows, n, None if x is None else byref(x), k, dw, dtype,
                                   ws, ep.ep_workspace_bytes(shape), None)

    R = ep.ep_rows
    for bad in (dict(L=layout()), dict(dy=None), dict(x=None), dict(x=R()), dict(x=R(P, P, P)), dict(x=R(P, None, P)),
                dict(x=R(None, P, None)), dict(x=R(None, None, P)), dict(x=R(None, P, P), k=136), dict(dw=None),
                dict(dtype=2), dict(n=12), dict(k=12), dict(dy=ODD), dict(dw=ODD), dict(x=R(ODD, None, None)),
                dict(x=R(None, ODD, P)), dict(x=R(None, P, ODD)), dict(rows=-5), dict(ws=None)):
        refused(call(**bad))
    for big in (dict(rows=1 << 31), dict(n=(1 << 20) + 8), dict(k=1 << 21)):
        refused(call(**big), ep.EP_ERR_UNSUPPORTED)
    many = ep.make_shape(32, 256, 2, 4096, 1)  # too many tiles for one launch
    assert lib.ep_expert_wgrad(byref(many), byref(layout(expert_offsets=P)), P, 10, 1 << 20, byref(R(P, None, None)),
                               1 << 20, P, 0, P, ep.ep_workspace_bytes(many), None) == ep.EP_ERR_UNSUPPORTED


def test_few_refusals_and_workspace(lib, shape):
    def call(s=shape, tk=ep.ep_tokens(P, None, None, P, P), x=ep.ep_experts(128, P, P), out=P, ws=P, wsb=1 << 30):
        return lib.ep_moe_few(byref(s), byref(tk), None if x is None else byref(x), out, ws, wsb, None)

    X = ep.ep_experts
    eight = X(128, None, None, P, P, P, P)
    for bad in (dict(x=None), dict(x=X(0, P, P)), dict(x=X(12, P, P)), dict(x=X(128, P, None)), dict(x=X(128, None, P)),
                dict(x=X(128, P, P, P, P, P, P)), dict(x=X(128, P, P, None, P)), dict(x=X(128, None, None, P, P, P, None)),
                dict(x=X(128, P, None, None, None, P, P)), dict(x=X(72, None, None, P, P, P, P)),
                dict(x=X(128, ODD, P)), dict(x=X(128, P, ODD)), dict(x=X(128, None, None, P, ODD, P, P)),
                dict(tk=ep.ep_tokens(None, None, None, P, P)), dict(tk=ep.ep_tokens(P, None, None, None, P)),
                dict(tk=ep.ep_tokens(P, None, None, P, None)), dict(tk=ep.ep_tokens(ODD, None, None, P, P)),
                dict(out=None), dict(out=ODD), dict(ws=None), dict(ws=P + 16), dict(wsb=256),
                dict(s=ep.make_shape(32, 200, 2, 8, 1), x=eight)):
        refused(call(**bad))
    refused(call(s=ep.make_shape(129, 256, 2, 8, 1)), ep.EP_ERR_UNSUPPORTED)
    refused(call(x=X((1 << 20) + 8, P, P)), ep.EP_ERR_UNSUPPORTED)
    n = ep.ep_few_workspace_bytes(shape, 128)
    assert n >= 256 + 32 * 2 * 128 * 2 and n % 256 == 0
    refused(call(wsb=n - 1))
    for s, F in ((ep.make_shape(129, 256, 2, 8, 1), 128), (shape, 0), (shape, 12), (shape, (1 << 20) + 8),
                 (ep.make_shape(4, 250, 2, 8, 1), 128)):
        assert ep.ep_few_workspace_bytes(s, F) == 0
    with pytest.raises(RuntimeError):
        ep.alloc_few_workspace(ep.make_shape(129, 256, 2, 8, 1), 128)


def test_binding_refuses_host_and_short_tensors(lib, shape):
    import torch

    L = dict(expert_offsets=P)
    t = torch.zeros(8)
    with pytest.raises(ValueError, match="GPU tensor"):
        ep.ep_expert_matmul(shape, L, t, 1, 8, P, 8, 0, P, t)
    with pytest.raises(ValueError, match="GPU tensor"):
        ep.ep_moe_few(shape, dict(x=t, topk_idx=P, topk_weights=P), dict(F=128, w13=P, w2=P), P, t)


def test_stream_lookup_keeps_torchs_checks(monkeypatch):
    """A call without a stream goes through torch's own initialisation, which refuses a process
    forked from one that holds the GPU; a given stream is taken as it is."""
    import torch

    class Stream:
        cuda_stream = 0x51

    def refuse():
        raise RuntimeError("Cannot re-initialize CUDA in forked subprocess")

    assert ep._stream(7) == 7 and ep._stream(Stream) == 0x51
    if torch.cuda.is_initialized():
        pytest.skip("torch has made these checks in this process already")
    monkeypatch.setattr(torch.cuda, "_lazy_init", refuse)
    with pytest.raises(RuntimeError, match="forked subprocess"):
        ep._stream(None)


class OnDevice:
    """What the binding asks of a tensor, on a given device."""
    is_cuda = True

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True

    def numel(self):
        return 1 << 40

    def element_size(self):
        return 1

    def data_ptr(self):
        return P + 4  # the library refuses it: no launch


class StreamOf:
    cuda_stream = 0x51

    def __init__(self, device):
        self.device_index = device


# Each entry point with one tensor (and its workspace) on given devices.
CALLS = dict(
    matmul=lambda s, L, t, ws, st: ep.ep_expert_matmul(s, L, t, 1, 64, P, 128, 0, P, ws, stream=st),
    matmul_y=lambda s, L, t, ws, st: ep.ep_expert_matmul(s, L, P, 1, 64, P, 128, 0, t, ws, stream=st),
    matmul_offsets=lambda s, L, t, ws, st: ep.ep_expert_matmul(s, dict(expert_offsets=t), P, 1, 64, P, 128, 0, P, ws,
                                                               stream=st),
    swiglu=lambda s, L, t, ws, st: ep.ep_expert_swiglu(s, L, P, 1, t, 128, P, P, P, ws, stream=st),
    swiglu_scales=lambda s, L, t, ws, st: ep.ep_expert_swiglu(s, L, P, 1, P, 128, P, P, t, ws, stream=st),
    grad=lambda s, L, t, ws, st: ep.ep_swiglu_grad(s, dict(expert_slot=P), 128, P, P, P, 1, t, P, P, P, ws, stream=st),
    grad_d_w=lambda s, L, t, ws, st: ep.ep_swiglu_grad(s, dict(expert_slot=P), 128, P, P, P, 1, P, P, P, t, ws, stream=st),
    wgrad=lambda s, L, t, ws, st: ep.ep_expert_wgrad(s, L, P, 1, 64, dict(x=t), 128, P, 0, ws, stream=st),
    wgrad_dw=lambda s, L, t, ws, st: ep.ep_expert_wgrad(s, L, P, 1, 64, dict(x=P), 128, t, 0, ws, stream=st),
    few=lambda s, L, t, ws, st: ep.ep_moe_few(s, dict(x=P, topk_idx=t, topk_weights=P), dict(F=128, w13=P, w2=P), P, ws,
                                              stream=st),
    few_w2=lambda s, L, t, ws, st: ep.ep_moe_few(s, dict(x=P, topk_idx=P, topk_weights=P), dict(F=128, w13=P, w2=t), P,
                                                 ws, stream=st),
)


@pytest.mark.parametrize("name", CALLS)
def test_binding_refuses_tensors_of_another_device(lib, shape, monkeypatch, name):
    """The kernel runs on its stream's device (the current one without a stream), where
    another device's memory would fault. A tensor of the right device reaches the library, which
    refuses the address."""
    import torch

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x30 + device)
    call, L = CALLS[name], dict(expert_offsets=P)
    for stream, own, other in ((None, 0, 1), (StreamOf(1), 1, 0), (0, 0, 1)):
        for devices in ((other, own), (own, other), (other, other)):
            with pytest.raises(ValueError, match="device"):
                call(shape, L, OnDevice(devices[0]), OnDevice(devices[1]), stream)
        with pytest.raises(RuntimeError, match="invalid|argument"):
            call(shape, L, OnDevice(own), OnDevice(own), stream)
