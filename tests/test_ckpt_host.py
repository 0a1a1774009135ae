"""Refusals of the 8-bit activation checkpoint, on the host."""
import ctypes as C
import gc
import weakref

import pytest
import torch

from routing_grouped_expert_router_amd import _lib as L
from routing_grouped_expert_router_amd.block import MoEBlock
from routing_grouped_expert_router_amd.layer import MoELayer

INVALID, UNSUPPORTED = -1, -2
FAKE = 0x1000


def tensor(q=FAKE, s=FAKE):
    t = L.moe_mx_tensor()
    t.q, t.s = q, s
    return t


def test_bf16_gemms():
    lib = L.lib()

    def call(op=L.MOE_GG_FWD_GATE_UP, dtype=L.MOE_BF16, d=256, F=256, n=64, g=tensor(), u=tensor(), **f):
        desc = L.make_gg_desc(op, dtype, 4, d, F, n, 16)
        names = ("x_perm", "w_gate", "w_up", "h") if op == L.MOE_GG_FWD_GATE_UP else ("dy_perm", "w_down", "dg", "du")
        for m in names:
            setattr(desc, m, FAKE)
        for m, v in f.items():
            setattr(desc, m, v)
        return lib.moe_grouped_gemm_ckpt(C.byref(desc), C.byref(g) if g else None, C.byref(u) if u else None, None)

    bwd = L.MOE_GG_DGRAD_DOWN
    assert lib.moe_grouped_gemm_ckpt(None, None, None, None) == INVALID
    assert call(g=None) == INVALID and call(u=None) == INVALID
    for op in (L.MOE_GG_FWD_DOWN, L.MOE_GG_DGRAD_GATE_UP, L.MOE_GG_WGRAD_DOWN, 9):
        assert call(op=op) == INVALID
    for kw in (dict(q=None), dict(s=None), dict(q=FAKE + 8), dict(s=FAKE + 2)):
        assert call(g=tensor(**kw)) == INVALID and call(bwd, u=tensor(**kw)) == INVALID
    assert call(**dict(h=None)) == INVALID                     # the forward's H is read next
    for op in (L.MOE_GG_FWD_GATE_UP, bwd):
        assert call(op, **dict([("g", tensor())]), d=264) == UNSUPPORTED
        assert call(op, F=128) == UNSUPPORTED
        assert call(op, dtype=L.MOE_F32) == UNSUPPORTED
        assert call(op, capacity=17) == INVALID
        assert call(op, n=0, capacity=0, group_offsets=FAKE) == 0
    assert call(bwd, dg=None) == INVALID and call(bwd, h=FAKE + 8) == INVALID
    desc = L.make_gg_desc(bwd, L.MOE_BF16, 4, 256, 256, 64, 16)
    desc.dy_perm = desc.w_down = desc.dg = desc.du = FAKE
    desc.g = FAKE                                              # bf16 g beside the copies
    t = tensor()
    assert lib.moe_grouped_gemm_ckpt(C.byref(desc), C.byref(t), C.byref(t), None) == INVALID


def test_mx_gemms():
    lib = L.lib()

    def call(op, g=tensor(), n=64, **f):
        desc = L.make_mx_gg_desc(op, 4, 256, 256, n, None)
        desc.group_offsets = FAKE
        for m in ("a0", "b0", "b1"):
            getattr(desc, m).q = getattr(desc, m).s = FAKE
        if op == L.MOE_GG_FWD_GATE_UP:
            desc.out2 = FAKE
        else:
            desc.out0 = desc.out1 = FAKE
        for m, v in f.items():
            setattr(desc, m, v)
        t = tensor()
        return lib.moe_grouped_gemm_mx_ckpt(C.byref(desc), C.byref(g), C.byref(t), None)

    fwd, bwd = L.MOE_GG_FWD_GATE_UP, L.MOE_GG_DGRAD_DOWN
    assert call(fwd, n=0) == 0 and call(bwd, n=0) == 0
    assert call(fwd, out0=FAKE) == INVALID and call(fwd, out1=FAKE) == INVALID and call(fwd, out2=None) == INVALID
    assert call(bwd, g=tensor(q=None)) == INVALID and call(bwd, out0=None) == INVALID
    assert call(L.MOE_GG_FWD_DOWN) == INVALID
    desc = L.make_mx_gg_desc(bwd, 4, 256, 256, 64, None)
    t = tensor()
    desc.u = FAKE
    assert lib.moe_grouped_gemm_mx_ckpt(C.byref(desc), C.byref(t), C.byref(t), None) == INVALID


def test_binding_checks_the_copies():
    desc = L.make_gg_desc(L.MOE_GG_FWD_GATE_UP, L.MOE_BF16, 4, 256, 256, 64, 16)
    u8 = torch.uint8
    ok = L.MxTensor(torch.empty(64, 256, dtype=u8), torch.empty(512, dtype=u8))
    with pytest.raises(L.MoEError, match="u.s: 511 elements"):
        L.moe_grouped_gemm_ckpt(desc, ok, L.MxTensor(ok.q, ok.s[:511]))
    with pytest.raises(L.MoEError, match="g.q: dtype"):
        L.moe_grouped_gemm_ckpt(desc, L.MxTensor(ok.q.float(), ok.s), ok)
    with pytest.raises(L.MoEError, match="device tensors"):
        L.moe_grouped_gemm_ckpt(desc, ok, ok)


@pytest.mark.parametrize("kw", [dict(recompute=True), dict(dtype=torch.float32), dict(d=384), dict(F=128),
                                dict(shared_ff=128)], ids=str)
def test_layer_refuses(kw):
    args = {**dict(T=8, d=256, E=4, k=2, F=256), **kw}
    with pytest.raises(ValueError, match="act8"):
        MoELayer(**args, device="cpu", act8=True)


def test_layer_takes_rows_only_with_act8():
    lay = MoELayer(8, 256, 4, 2, 256, device="cpu", routing="given")
    with pytest.raises(ValueError, match="act8"):
        lay.forward(None, None, None, None, x8=object())


@pytest.mark.parametrize("opts", [dict(), dict(act8=True), dict(mx_bf16_intermediates=False),
                                  dict(act8=True, mx_bf16_intermediates=False)], ids=str)
def test_release_lets_go_of_the_mxfp8_experts_tensors_too(opts):
    """What the layer releases is held by nothing else: the MXFP8 experts
    write into the same tensors under names of their own."""
    lay = MoELayer(8, 256, 4, 2, 256, device="cpu", routing="given", mxfp8=True, **opts)
    lay.forward_buffers()
    lay.backward_buffers()
    held = {}
    for name in ("g", "u", "h", "y_perm", "y", "dy_perm", "dg", "du", "dx_perm"):
        if getattr(lay, name) is not None:
            held[name] = weakref.ref(getattr(lay, name))
    for name in ("g8", "u8") if lay.act8 else ():
        held[name] = weakref.ref(getattr(lay, name).q)
    assert len(held) >= 6
    lay.release_intermediates()
    gc.collect()
    assert [n for n, r in held.items() if r() is not None] == []
    lay.forward_buffers()                                       # and the next step has them again
    lay.backward_buffers()
    assert lay.mx.y_perm is lay.y_perm and lay.mx.dx_perm is lay.dx_perm and lay.mx.dg is lay.dg
    assert (lay.mx.g8 is lay.g8 and lay.g8 is not None) if lay.act8 else lay.mx.g is lay.g


@pytest.mark.parametrize("opts,reads", [(dict(), False), (dict(act8=True), True), (dict(act8=True, mxfp8=True), True),
                                        (dict(act8=True, routing="given"), True),
                                        (dict(act8=True, mxfp8=True, routing="given"), False)], ids=str)
def test_block_writes_the_rows_its_layer_reads(opts, reads, monkeypatch):
    """The norm writes the 8-bit rows only where the backward reads them."""
    blk = MoEBlock(8, 256, 4, 2, 256, device="cpu", **opts)
    seen = {}
    monkeypatch.setattr(L, "moe_add_rmsnorm", lambda x, w, eps, **kw: seen.update(kw))
    monkeypatch.setattr(blk.layer, "forward", lambda n, *a, **kw: seen.update(x8=kw.get("x8")))
    x, w = torch.zeros(8, 256, dtype=torch.bfloat16), torch.ones(256, dtype=torch.bfloat16)
    blk.forward(x, None, w)
    assert (seen["q"] is not None) == (seen["x8"] is not None) == reads and seen["q"] is seen["x8"]


class OnDevice:
    """What the binding asks of a contiguous device tensor; never dereferenced."""

    def __init__(self, dtype, shape, at):
        self.dtype, self.shape, self.is_cuda, self.at = dtype, shape, True, at

    numel = lambda self: int(torch.tensor(self.shape).prod())
    element_size = lambda self: self.dtype.itemsize
    is_contiguous = lambda self: True
    data_ptr = lambda self: FAKE
    get_device = lambda self: self.at


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("name", [None, "x", "w", "offsets", "copy"])
def test_every_tensor_has_to_be_on_the_current_device(mx, name, monkeypatch):
    monkeypatch.setattr(L, "_one_device", False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(L, "_stream", lambda s=None: None)
    called = []
    monkeypatch.setattr(L, "_call", lambda f, *a: called.append(f))
    at = lambda n: 1 if n == name else 0
    t = lambda n, *shape, dtype=torch.bfloat16: OnDevice(dtype, shape, at(n))
    q = lambda n, rows, cols: L.MxTensor(t(n, rows, cols, dtype=torch.uint8), t(n, rows * cols // 32, dtype=torch.uint8))
    off = t("offsets", 5, dtype=torch.int32)
    if mx:
        desc = L.make_mx_gg_desc(L.MOE_GG_FWD_GATE_UP, 4, 256, 256, 64, off, a0=q("x", 64, 256), b0=q("w", 256, 1024),
                                 b1=q("w", 256, 1024), out2=t("h", 64, 256))
        call = L.moe_grouped_gemm_mx_ckpt
    else:
        desc = L.make_gg_desc(L.MOE_GG_FWD_GATE_UP, L.MOE_BF16, 4, 256, 256, 64, 0, off, x_perm=t("x", 64, 256),
                              w_gate=t("w", 4, 256, 256), w_up=t("w", 4, 256, 256), h=t("h", 64, 256))
        call = L.moe_grouped_gemm_ckpt
    copies = q("copy", 64, 256), q("other copy", 64, 256)
    if name is None:
        call(desc, *copies)
        assert called == [call.__name__]
    else:
        with pytest.raises(L.MoEError, match="on cuda:1, the current device is cuda:0"):
            call(desc, *copies)
        assert called == []
