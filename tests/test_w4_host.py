"""Refusals of the 4-bit experts, on the host, and the header's constants."""
import ctypes as C
import os
import re

import pytest
import torch

from routing_grouped_expert_router_amd import _lib as L
from routing_grouped_expert_router_amd.decode import MoEDecoder

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
FAKE = 0x1000
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe.h")


def test_constants_and_layout():
    text = open(HEADER).read()
    for name in ("MOE_MAX_NORM_D", "MOE_W4_MAX_SLOTS"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(L, name)
    # five ints, three pointers, three (codes, scales) pairs, y_add, y, ws, ws_bytes
    assert C.sizeof(L.moe_w4_desc) == 24 + 8 * (3 + 6 + 4)


def test_sizes():
    lib = L.lib()
    assert lib.moe_w4_code_bytes(256, 48) == 256 * 24
    assert lib.moe_w4_scale_bytes(512, 16) == 256 and lib.moe_w4_scale_bytes(640, 32) == 1024
    assert lib.moe_w4_code_bytes(0, 16) == 0 and lib.moe_w4_scale_bytes(128, -1) == 0
    assert lib.moe_experts_w4_workspace_bytes(0, 2, 128, 128) == 0
    assert lib.moe_experts_w4_workspace_bytes(3, 2, 256, 128) == 6 * 128 * 4 + 6 * 256 * 4


def test_quantize_argument_errors():
    f = L.lib().moe_w4_quantize
    assert f(FAKE, 2, 192, 64, FAKE, FAKE, None) == INVALID       # K % 128
    assert f(FAKE, 2, 256, 40, FAKE, FAKE, None) == INVALID       # N % 16
    assert f(FAKE, -1, 256, 64, FAKE, FAKE, None) == INVALID
    assert f(None, 2, 256, 64, FAKE, FAKE, None) == INVALID
    assert f(FAKE + 2, 2, 256, 64, FAKE, FAKE, None) == INVALID
    assert f(FAKE, 2, 256, 64, FAKE + 8, FAKE, None) == INVALID
    assert f(FAKE, 2, 256, 64, FAKE, FAKE + 2, None) == INVALID
    assert f(None, 0, 256, 64, None, None, None) == 0


def desc(**kw):
    g = L.moe_w4_desc(4, 256, 8, 2, 384)
    for n in ("x", "topk_idx", "topk_w", "w_gate_q", "w_gate_s", "w_up_q", "w_up_s", "w_down_q", "w_down_s", "y", "ws"):
        setattr(g, n, FAKE)
    g.ws_bytes = 1 << 30
    for n, v in kw.items():
        setattr(g, n, v)
    return g


def test_experts_argument_errors():
    lib = L.lib()
    call = lambda **kw: lib.moe_experts_w4(C.byref(desc(**kw)), None)
    assert lib.moe_experts_w4(None, None) == INVALID
    assert call(T=0) == 0 and call(T=0, x=None, ws=None) == 0
    assert call(T=-1) == INVALID and call(k=0) == INVALID and call(E=0) == INVALID
    assert call(d=192) == INVALID and call(F=64) == INVALID
    assert call(E=1025) == UNSUPPORTED and call(k=17) == UNSUPPORTED
    assert call(T=2049) == UNSUPPORTED                                 # 4098 slots
    for n in ("x", "topk_idx", "topk_w", "y", "w_gate_q", "w_up_s", "w_down_q"):
        assert call(**{n: None}) == INVALID
    for n in ("x", "y", "y_add", "w_up_q"):
        assert call(**{n: FAKE + 8}) == INVALID
    assert call(topk_idx=FAKE + 2) == INVALID and call(w_gate_s=FAKE + 1) == INVALID
    need = lib.moe_experts_w4_workspace_bytes(4, 2, 256, 384)
    assert call(ws=None) == WORKSPACE and call(ws_bytes=need - 1) == WORKSPACE and call(ws=FAKE + 8) == WORKSPACE


def test_binding_refuses_mismatched_tensors():
    T, d, E, k, F = 3, 256, 4, 2, 128
    bf = torch.bfloat16
    x, y = torch.zeros(T, d, dtype=bf), torch.zeros(T, d, dtype=bf)
    idx, p = torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k)
    wg, wd = L.W4Tensor.empty(E, d, F, device="cpu"), L.W4Tensor.empty(E, F, d, device="cpu")
    ws = torch.empty(L.moe_experts_w4_workspace_bytes(T, k, d, F), dtype=torch.uint8)
    with pytest.raises(L.MoEError, match="device tensors"):
        L.moe_experts_w4(x, idx, p, wg, wg, wd, y, ws)
    with pytest.raises(L.MoEError, match="w_down"):
        L.moe_experts_w4(x, idx, p, wg, wg, wg, y, ws)
    with pytest.raises(L.MoEError, match="topk_idx: dtype"):
        L.moe_experts_w4(x, idx.long(), p, wg, wg, wd, y, ws)
    with pytest.raises(L.MoEError, match="topk_w: shape"):
        L.moe_experts_w4(x, idx, p[:2], wg, wg, wd, y, ws)
    with pytest.raises(L.MoEError, match="w_up.s"):
        L.moe_experts_w4(x, idx, p, wg, L.W4Tensor(wg.q, wg.s[:-1], E, d, F), wd, y, ws)
    with pytest.raises(L.MoEError, match="y: dtype"):
        L.moe_experts_w4(x, idx, p, wg, wg, wd, y.float(), ws)
    with pytest.raises(L.MoEError, match="w: shape|out"):
        L.moe_w4_quantize(torch.zeros(E, d, F, dtype=bf), wd)


def test_decoder_refuses_batches_past_the_slot_limit():
    with pytest.raises(ValueError, match="4096"):
        MoEDecoder(None, None, torch.empty(8, 128, 128), None, None, k=4, max_tokens=1025)


def test_widths_past_one_launch_are_refused():
    """A launch counts its threads in 32 bits."""
    lib = L.lib()
    need = 1 << 40
    call = lambda **kw: lib.moe_experts_w4(C.byref(desc(ws_bytes=need, **kw)), None)
    assert call(T=1024, k=1, E=1024, F=1 << 20) == UNSUPPORTED            # 1024 experts of 65536 tiles
    assert call(T=1024, k=1, E=1024, d=1 << 20) == UNSUPPORTED
    assert call(T=4096, k=1, E=1, d=1 << 22) == UNSUPPORTED               # the weighted sum's threads
    assert lib.moe_w4_quantize(FAKE, 1 << 14, 1 << 14, 1 << 9, FAKE, FAKE, None) == UNSUPPORTED


@pytest.mark.parametrize("rows", [slice(0, 3), slice(1, 4), slice(4, 5)], ids=str)
@pytest.mark.parametrize("swap", [False, True])
def test_decoder_hands_the_norm_no_rows_that_it_overwrites(rows, swap, monkeypatch):
    """Rows of the decoder's own h may come back as res (or x): the norm may
    write h over them only where each row is its own."""
    monkeypatch.setattr(L, "moe_w4_quantize", lambda w, out: None)
    b = lambda *s: torch.randn(*s).to(torch.bfloat16)
    dec = MoEDecoder(b(128), b(128, 4), b(4, 128, 128), b(4, 128, 128), b(4, 128, 128), k=2, max_tokens=5)
    for name in ("moe_router_gemm", "moe_route", "moe_experts_w4"):
        monkeypatch.setattr(L, name, lambda *a, **kw: None)
    calls = []
    monkeypatch.setattr(L, "moe_add_rmsnorm", lambda x, w, eps, **kw: calls.append((x, kw["res"], kw["h"])))
    x, res = dec.y[rows], dec.h[rows]
    x.copy_(b(*x.shape))
    res.copy_(b(*res.shape))
    want = (res.clone(), x.clone()) if swap else (x.clone(), res.clone())
    dec.step(*((res, x) if swap else (x, res)))
    (gx, gres, h), = calls
    assert torch.equal(gx, want[0]) and torch.equal(gres, want[1])
    size = h.numel() * h.element_size()
    for t in (gx, gres):
        assert t.data_ptr() == h.data_ptr() or abs(t.data_ptr() - h.data_ptr()) >= size


def test_missing_workspace_is_the_librarys_error():
    T, d, E, k, F = 3, 256, 4, 2, 128
    bf = torch.bfloat16
    x, idx, p = torch.zeros(T, d, dtype=bf), torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k)
    wg, wd = L.W4Tensor.empty(E, d, F, device="cpu"), L.W4Tensor.empty(E, F, d, device="cpu")
    with pytest.raises(L.MoEError):
        L.moe_experts_w4(x, idx, p, wg, wg, wd, x.clone(), None)


@pytest.mark.parametrize("given", [("w_gate_s",), ("w_up_s", "w_down_s"), ("w_down_s",)], ids=str)
def test_decoder_refuses_part_of_a_shared_expert(given, monkeypatch):
    monkeypatch.setattr(L, "moe_w4_quantize", lambda w, out: None)
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    shared = dict(w_gate_s=b(128, 128), w_up_s=b(128, 128), w_down_s=b(128, 128))
    args = (b(128), b(128, 4), b(4, 128, 128), b(4, 128, 128), b(4, 128, 128))
    with pytest.raises(ValueError, match="shared expert"):
        MoEDecoder(*args, k=2, max_tokens=5, **{n: shared[n] for n in given})
    assert MoEDecoder(*args, k=2, max_tokens=5, **shared).shared is not None
    assert MoEDecoder(*args, k=2, max_tokens=5).shared is None
