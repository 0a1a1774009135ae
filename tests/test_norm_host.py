"""Refusals of the norm and of the row restore, on the host: before anything
is launched, with the documented codes."""
import pytest
import torch

from routing_grouped_expert_router_amd import _lib as L

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
FAKE = 0x1000   # 16-byte aligned, never dereferenced


def test_norm_argument_errors():
    f = L.lib().moe_add_rmsnorm
    #       dtype x     res   w     T  d    eps   h     y     q     s     rstd  stream
    good = [1, FAKE, FAKE, FAKE, 4, 256, 1e-6, FAKE, FAKE, FAKE, FAKE, FAKE, None]

    def call(**kw):
        a = list(good)
        for k, v in kw.items():
            a[["dtype", "x", "res", "w", "T", "d", "eps", "h", "y", "q", "s", "rstd", "stream"].index(k)] = v
        return f(*a)

    assert call(T=0) == 0
    assert call(T=0, x=None, w=None) == 0                  # nothing to read
    assert call(T=-1) == INVALID
    assert call(dtype=2) == INVALID
    assert call(d=12) == INVALID                           # d % 8
    assert call(d=0) == INVALID
    assert call(d=136) == INVALID                          # the MXFP8 copy needs d % 128 == 0
    assert call(d=12288 + 128) == UNSUPPORTED
    assert call(dtype=0) == INVALID                        # no MXFP8 copy of binary32
    assert call(s=None) == INVALID and call(q=None) == INVALID
    assert call(res=None) == INVALID                       # h is written only beside res
    assert call(h=None) == INVALID
    assert call(y=None, q=None, s=None) == INVALID         # no output
    for eps in (0.0, -1e-6, float("inf"), float("nan")):
        assert call(eps=eps) == INVALID
    for n in ("x", "res", "w", "h", "y", "q"):
        assert call(**{n: FAKE + 8}) == INVALID            # alignment
    assert call(s=FAKE + 2) == INVALID and call(rstd=FAKE + 2) == INVALID
    assert call(x=None) == INVALID and call(w=None) == INVALID


def test_norm_bwd_argument_errors():
    lib = L.lib()
    need = lib.moe_add_rmsnorm_bwd_workspace_bytes(300, 256)
    assert need > 0 and need % 16 == 0
    assert lib.moe_add_rmsnorm_bwd_workspace_bytes(0, 256) == 0
    names = ["dtype", "dy", "h", "w", "rstd", "dh", "T", "d", "dx", "dw", "ws", "ws_bytes", "stream"]
    good = [1, FAKE, FAKE, FAKE, FAKE, FAKE, 300, 256, FAKE, FAKE, FAKE, need, None]

    def call(**kw):
        a = list(good)
        for k, v in kw.items():
            a[names.index(k)] = v
        return lib.moe_add_rmsnorm_bwd(*a)

    assert call(T=0, dw=None) == 0
    assert call(T=-1) == INVALID and call(dtype=5) == INVALID and call(d=12) == INVALID
    assert call(d=12296) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(ws_bytes=need - 1) == WORKSPACE and call(ws=FAKE + 4) == WORKSPACE
    for n in ("dy", "h", "w", "dh", "dx", "dw"):
        assert call(**{n: FAKE + 8}) == INVALID
    for n in ("dy", "h", "w", "rstd", "dx"):
        assert call(**{n: None}) == INVALID


def test_restore_argument_errors():
    lib = L.lib()
    f = lib.moe_permute_from_mx
    #            q     s     T   d    k  row_of src_slot n_rows x x_perm
    assert f(FAKE, FAKE, 10, 256, 2, FAKE, None, 21, FAKE, FAKE, None) == INVALID      # dropless rows
    assert f(FAKE, FAKE, 10, 192, 2, FAKE, None, 20, FAKE, FAKE, None) == INVALID      # d % 128
    assert f(FAKE, FAKE, 10, 256, 17, FAKE, None, 170, FAKE, FAKE, None) == UNSUPPORTED
    assert f(FAKE + 8, FAKE, 10, 256, 2, FAKE, None, 20, FAKE, FAKE, None) == INVALID
    assert f(FAKE, FAKE + 2, 10, 256, 2, FAKE, None, 20, FAKE, FAKE, None) == INVALID
    assert f(FAKE, FAKE, 10, 256, 2, None, None, 20, FAKE, FAKE, None) == INVALID
    assert f(FAKE, FAKE, 10, 256, 2, FAKE, None, 20, FAKE + 8, FAKE, None) == INVALID
    assert f(FAKE, FAKE, 10, 256, 2, FAKE, None, 20, FAKE, None, None) == INVALID
    assert f(None, None, 0, 256, 2, None, None, 0, None, None, None) == 0
    g = lib.moe_mx_dequantize
    assert g(FAKE, FAKE, 4, 192, FAKE, None) == INVALID
    assert g(FAKE, FAKE, -1, 256, FAKE, None) == INVALID
    assert g(None, FAKE, 4, 256, FAKE, None) == INVALID
    assert g(FAKE, FAKE, 4, 256, FAKE + 2, None) == INVALID
    assert g(None, None, 0, 256, None, None) == 0


def test_binding_refuses_mismatched_tensors():
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    x, w = torch.zeros(4, 256, dtype=bf), torch.ones(256, dtype=bf)
    y = torch.empty_like(x)
    with pytest.raises(L.MoEError, match="w: shape"):
        L.moe_add_rmsnorm(x, w[:128], 1e-6, y=y)
    with pytest.raises(L.MoEError, match="w: dtype"):
        L.moe_add_rmsnorm(x, w.float(), 1e-6, y=y)
    with pytest.raises(L.MoEError, match="res: shape"):
        L.moe_add_rmsnorm(x, w, 1e-6, res=x[:3], h=y, y=y)
    with pytest.raises(L.MoEError, match="contiguous"):
        L.moe_add_rmsnorm(torch.zeros(256, 4, dtype=bf).t(), w, 1e-6, y=y)
    with pytest.raises(L.MoEError, match="q.s"):
        L.moe_add_rmsnorm(x, w, 1e-6, y=y, q=L.MxTensor(torch.empty(4, 256, dtype=u8), torch.empty(8, dtype=u8)))
    with pytest.raises(L.MoEError, match="rstd"):
        L.moe_add_rmsnorm(x, w, 1e-6, y=y, rstd=torch.empty(3))
    with pytest.raises(L.MoEError, match="needs device tensors"):
        L.moe_add_rmsnorm(x, w, 1e-6, y=y)
    with pytest.raises(L.MoEError, match="dw: dtype"):
        L.moe_add_rmsnorm_bwd(x, x, w, torch.empty(4), y, dw=torch.empty(256))
    mx = L.MxTensor(torch.empty(4, 256, dtype=u8), torch.empty(32, dtype=u8))
    with pytest.raises(L.MoEError, match="q: 1024 elements"):
        L.moe_mx_dequantize(mx, torch.empty(5, 256, dtype=bf))
    rows = torch.zeros(10, dtype=torch.int32)
    with pytest.raises(L.MoEError, match="elements"):
        L.moe_permute_from_mx(mx, 2, rows, None, torch.empty(10, 256, dtype=bf))
    with pytest.raises(L.MoEError, match="x: shape"):
        L.moe_permute_from_mx(mx, 2, rows[:8], None, torch.empty(8, 256, dtype=bf), x=torch.empty(4, 128, dtype=bf))


def test_rows_past_one_launch_are_refused():
    """A launch counts its threads in 32 bits: 64 for each row of a wave."""
    lib = L.lib()
    A = [0x1000 * i for i in range(1, 12)]

    def norm(dtype, T, d, mx=False):
        return lib.moe_add_rmsnorm(dtype, A[0], A[1], A[2], T, d, 1e-6, A[3], A[4], A[5] if mx else None,
                                   A[6] if mx else None, A[7], None)

    assert norm(1, 1 << 26, 8) == UNSUPPORTED and norm(0, 1 << 26, 8) == UNSUPPORTED
    assert norm(1, 1 << 26, 128, True) == UNSUPPORTED and norm(1, (1 << 31) - 1, 2048) == UNSUPPORTED
    assert norm(1, 1 << 25, 2056) == UNSUPPORTED and norm(0, 1 << 25, 1032) == UNSUPPORTED     # two waves a row
    assert norm(1, 1 << 24, 8192) == UNSUPPORTED and norm(0, 5592406, 12288) == UNSUPPORTED    # four, twelve
    f = lib.moe_permute_from_mx
    assert f(A[0], A[1], 1 << 26, 128, 1, A[2], None, 1 << 26, A[3], A[4], None) == UNSUPPORTED
    assert f(A[0], A[1], 8, 128, 1, A[2], A[5], 1 << 26, A[3], A[4], None) == UNSUPPORTED      # pad rows
    assert f(A[0], A[1], (1 << 31) - 1, 128, 1, A[2], None, (1 << 31) - 1, A[3], A[4], None) == UNSUPPORTED
    assert lib.moe_mx_dequantize(A[0], A[1], 1 << 26, 128, A[2], None) == UNSUPPORTED
    assert lib.moe_mx_dequantize(A[0], A[1], (1 << 31) - 1, 128, A[2], None) == UNSUPPORTED


def test_binding_refuses_row_counts_past_32_bits():
    """2^32 + 4 rows are not 4: a row count is an int of the library's."""
    T, bf = (1 << 32) + 4, torch.bfloat16
    x, w = torch.empty(T, 8, dtype=bf, device="meta"), torch.ones(8, dtype=bf)
    with pytest.raises(L.MoEError, match="rows"):
        L.moe_add_rmsnorm(x, w, 1e-6, y=x)
    with pytest.raises(L.MoEError, match="rows"):
        L.moe_add_rmsnorm_bwd(x, x, w, torch.empty(T, device="meta"), x, dw=w)
    with pytest.raises(L.MoEError, match="rows"):
        L.moe_add_rmsnorm_bwd_workspace_bytes(T, 8)


def test_norm_of_no_rows_needs_no_tensor():
    """A tensor of no row may have no address."""
    f = L.lib().moe_add_rmsnorm
    for dtype in (0, 1):
        assert f(dtype, None, None, FAKE, 0, 256, 1e-6, None, None, None, None, None, None) == 0
        assert f(dtype, None, None, FAKE, 0, 12, 1e-6, None, None, None, None, None, None) == INVALID
        assert f(dtype, None, None, FAKE, 0, 12296, 1e-6, None, None, None, None, None, None) == UNSUPPORTED
    assert f(1, None, FAKE, FAKE, 4, 256, 1e-6, None, FAKE, None, None, None, None) == INVALID
