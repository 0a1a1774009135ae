"""G and U kept in 8 bits between the passes: the two GEMMs, the layer and the
block that use them.

The GEMMs' sums are those of the calls that keep bf16 (the same K loop), so
their outputs are compared bit for bit with those calls on the copies' values;
H, which the backward computes again, is compared with 64 bits (half a bf16
step, 2^-8, and the hardware exponential and reciprocal, 2^-20 at most)."""
import numpy as np
import pytest
import torch

import oracle.moe as om
from moe_inputs import make_inputs, workload
from oracle.norm import add_rmsnorm, add_rmsnorm_bwd
from oracle.numerics import f64_to_bf16_bits, mx_quantize, mx_roundtrip, round_bf16, round_f32
from routing_grouped_expert_router_amd import _lib as L
from routing_grouped_expert_router_amd.block import MoEBlock
from routing_grouped_expert_router_amd.layer import MoELayer
from routing_grouped_expert_router_amd.mx_layer import MxExperts

from parity import assert_close, dev, host

pytestmark = pytest.mark.gpu

BF, U8 = torch.bfloat16, torch.uint8


def bf(a):
    return dev(f64_to_bf16_bits(a), "bf16")


def rows8(n, F, fill=0xAA):
    return L.MxTensor(torch.full((n, F), fill, dtype=U8, device="cuda"),
                      torch.full((n * F // 32,), fill, dtype=U8, device="cuda"))


def grouped(s):
    R, nb = s.shape
    return np.ascontiguousarray(s.reshape(R, nb // 4, 4).transpose(1, 0, 2)).reshape(-1)


def problem(counts, d, F, seed, spare=0):
    g = np.random.default_rng([seed, d, F, len(counts)])
    E, n = len(counts), int(sum(counts)) + spare
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x, dy = (bf(g.standard_normal((n, d))) for _ in range(2))
    wg, wu = (bf(g.standard_normal((E, d, F)) * d ** -0.5) for _ in range(2))
    wd = bf(g.standard_normal((E, F, d)) * F ** -0.5)
    return E, n, dev(off, "i32"), x, dy, wg, wu, wd


# the last for tiles of 64 rows (F 256), of 128 (F 1024), and of both (F 768)
COUNTS = [[1], [0, 3, 0], [129, 0, 127, 1, 256], [5, 300, 0, 64], [700], [2100, 0, 1999]]


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("d,F", [(256, 256), (512, 768), (256, 1024)])
@pytest.mark.parametrize("spare", [0, 5])
def test_gemms(counts, d, F, spare):
    E, n, off, x, dy, wg, wu, wd = problem(counts, d, F, 1, spare)
    used = n - spare
    new = lambda: torch.full((n, F), 9.0, dtype=BF, device="cuda")
    desc = lambda op, **t: L.make_gg_desc(op, L.MOE_BF16, E, d, F, n, 0, off, **t)
    g, u, h, h8 = new(), new(), new(), new()
    L.moe_grouped_gemm(desc(L.MOE_GG_FWD_GATE_UP, x_perm=x, w_gate=wg, w_up=wu, g=g, u=u, h=h))
    g8, u8 = rows8(n, F), rows8(n, F)
    L.moe_grouped_gemm_ckpt(desc(L.MOE_GG_FWD_GATE_UP, x_perm=x, w_gate=wg, w_up=wu, h=h8), g8, u8)
    assert torch.equal(h, h8)
    for t, t8 in ((g, g8), (u, u8)):
        q, s = mx_quantize(host(t))
        q[used:], s[used:] = 0xAA, 0xAA             # rows past the last group stay as they were
        assert np.array_equal(host(t8.q), q) and np.array_equal(host(t8.s), grouped(s))
    # the backward: as with the bf16 tensors of the copies' values
    gd, ud = new(), new()
    L.moe_mx_dequantize(g8, gd)
    L.moe_mx_dequantize(u8, ud)
    want, got = (new(), new()), (new(), new(), new())
    L.moe_grouped_gemm(desc(L.MOE_GG_DGRAD_DOWN, dy_perm=dy, w_down=wd, g=gd, u=ud, dg=want[0], du=want[1]))
    L.moe_grouped_gemm_ckpt(desc(L.MOE_GG_DGRAD_DOWN, dy_perm=dy, w_down=wd, dg=got[0], du=got[1], h=got[2]), g8, u8)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    v = host(gd)[:used], host(ud)[:used]
    ref = v[0] * v[1] / (1 + np.exp(-v[0]))
    assert np.all(np.abs(host(got[2])[:used] - ref) <= (2.0 ** -8 + 2.0 ** -19) * np.abs(ref))
    assert np.all(host(got[2])[used:] == 9.0)
    dg, du = new(), new()
    L.moe_grouped_gemm_ckpt(desc(L.MOE_GG_DGRAD_DOWN, dy_perm=dy, w_down=wd, dg=dg, du=du), g8, u8)   # h not wanted
    assert torch.equal(dg, got[0]) and torch.equal(du, got[1])


def test_gemms_against_the_oracle_and_padded():
    """Capacity groups, the whole chain in 64 bits from the same bf16 inputs."""
    E, cap, d, F = 5, 24, 256, 512
    g = np.random.default_rng(3)
    n = E * cap
    r = round_bf16
    x, dy = r(g.standard_normal((n, d))), r(g.standard_normal((n, d)))
    x[20:24] = 0                                       # pad rows
    wg, wu = r(g.standard_normal((E, d, F)) * d ** -0.5), r(g.standard_normal((E, d, F)) * d ** -0.5)
    wd = r(g.standard_normal((E, F, d)) * F ** -0.5)
    groups = [(e * cap, cap) for e in range(E)]
    G, Uv = (r(np.concatenate([x[a:a + m] @ w[e] for e, (a, m) in enumerate(groups)])) for w in (wg, wu))
    G8, U8v = mx_roundtrip(G), mx_roundtrip(Uv)
    dH = np.concatenate([dy[a:a + m] @ wd[e].T for e, (a, m) in enumerate(groups)])
    s = 1 / (1 + np.exp(-G8))
    ref = dict(dg=dH * U8v * s * (1 + G8 * (1 - s)), du=dH * G8 * s, h=G8 * s * U8v)
    g8, u8 = rows8(n, F), rows8(n, F)
    out = {m: torch.empty(n, F, dtype=BF, device="cuda") for m in ref}
    desc = lambda op, **t: L.make_gg_desc(op, L.MOE_BF16, E, d, F, n, cap, None, **t)
    L.moe_grouped_gemm_ckpt(desc(L.MOE_GG_FWD_GATE_UP, x_perm=bf(x), w_gate=bf(wg), w_up=bf(wu), h=out["h"]), g8, u8)
    assert_close(host(out["h"]), G / (1 + np.exp(-G)) * Uv, "bf16", "h")
    L.moe_grouped_gemm_ckpt(desc(L.MOE_GG_DGRAD_DOWN, dy_perm=bf(dy), w_down=bf(wd), **out), g8, u8)
    # a G at the border of two codes may fall either way (its binary32 sum and
    # the oracle's differ): compare where the copies are the same
    gd, ud = (torch.empty(n, F, dtype=BF, device="cuda") for _ in range(2))
    L.moe_mx_dequantize(g8, gd)
    L.moe_mx_dequantize(u8, ud)
    same = (host(gd) == G8) & (host(ud) == U8v)
    assert same.mean() > 0.99
    for m, v in ref.items():
        assert_close(np.where(same, host(out[m]), 0), np.where(same, v, 0), "bf16", m)


@pytest.mark.parametrize("counts", [[0, 3, 0], [129, 0, 127, 256], [500]], ids=str)
@pytest.mark.parametrize("keep", [True, False])
def test_mx_gemms(counts, keep):
    d, F = 256, 512
    E, n, off, x, dy, wg, wu, wd = problem(counts, d, F, 2)
    a = MxExperts(n, d, E, F, bf16_intermediates=keep)
    b = MxExperts(n, d, E, F, bf16_intermediates=keep)
    b.g8, b.u8 = rows8(n, F), rows8(n, F)
    a.forward(x, off, wg, wu, wd)
    b.forward(x, off, wg, wu, wd)
    assert torch.equal(a.y_perm, b.y_perm) and (not keep or torch.equal(a.h, b.h))
    for t, t8 in ((a.g, b.g8), (a.u, b.u8)):
        q, s = mx_quantize(host(t))
        assert np.array_equal(host(t8.q), q) and np.array_equal(host(t8.s), grouped(s))
        L.moe_mx_dequantize(t8, t)                     # a's backward reads the copies' values
    a.backward(dy)
    b.backward(dy)
    for name in ("dx_perm", "dw_gate", "dw_up", "dw_down") + (("dg", "du") if keep else ()):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


def _inputs(wl):
    inp = make_inputs(wl)
    out = {}
    for name, v in inp.items():
        if name == "topk_idx":
            out[name] = dev(v.astype(np.int32), "i32")
        else:
            out[name] = dev(v, "f32" if name == "topk_w" else "bf16")
    return out


SMALL = dict(T=301, d=256, F=256, E=8)
OPTS = {
    "given": dict(name="e128_uniform_bf16"), "learned": dict(name="e8_learned_bf16"),
    "padded": dict(name="e128_zipf_bf16", over=dict(zero_cold=2), capacity=60),
    "shared": dict(name="e8_learned_bf16", over=dict(shared_ff=512)),
    "mxfp8": dict(name="e8_learned_bf16", opts=dict(mxfp8=True)),
    "mxfp8 given": dict(name="e128_uniform_bf16", opts=dict(mxfp8=True, mx_bf16_intermediates=False)),
}


@pytest.mark.parametrize("case", OPTS)
@pytest.mark.parametrize("x8", [True, False])
def test_layer(case, x8):
    """y is the plain layer's bit for bit; the gradients are the plain
    layer's backward at the copies' values."""
    c = OPTS[case]
    wl = workload(c["name"]).scaled(**SMALL, **c.get("over", {}))
    t, opts = _inputs(wl), dict(c.get("opts", {}))
    kw = {n: t[n] for n in ("w_r", "topk_idx", "topk_w", "w_gate_s", "w_up_s", "w_down_s") if n in t}
    mk = lambda **o: MoELayer(wl.T, wl.d, wl.E, wl.k, wl.F, routing="learned" if "w_r" in t else "given",
                              capacity=c.get("capacity", 0), shared_ff=wl.shared_ff, **opts, **o)
    a, b = mk(), mk(act8=True)
    a.forward(t["x"], t["w_gate"], t["w_up"], t["w_down"], **kw)
    q = rows8(wl.T, wl.d)
    L.moe_mx_quantize(t["x"], 0, q.q, q.s)
    b.forward(t["x"], t["w_gate"], t["w_up"], t["w_down"], **kw, **(dict(x8=q) if x8 else {}))
    assert torch.equal(a.y, b.y)
    assert b.x is None and b.g is None and b.x_perm is None and (b.h is None or b.mxfp8)
    # the plain layer's tensors replaced by the copies' values
    if not a.mxfp8 or "w_r" in t:
        a.x = torch.empty_like(t["x"])
        L.moe_mx_dequantize(q, a.x)
    if not a.mxfp8:
        L.moe_permute(a.x, wl.k, a.row_of, a.src_slot if a.capacity else None, a.x_perm)
    silu = lambda g, u: (g.float() * u.float() * torch.sigmoid(g.float())).to(BF)
    for g, u, h, g8, u8 in (("g", "u", "h", b.g8, b.u8), ("g_s", "u_s", "h_s", b.g8_s, b.u8_s)):
        if g8 is None:
            continue
        L.moe_mx_dequantize(g8, getattr(a, g))
        L.moe_mx_dequantize(u8, getattr(a, u))
    dgrads = {}
    b.hook = lambda name: dgrads.update({m: getattr(b, m).clone() for m in ("h", "h_s")
                                         if getattr(b, m, None) is not None}) if "bwd_data" in name or "dgrad_down" in name else None
    b.backward(t["dy"])
    if not a.mxfp8:
        ref = silu(a.g, a.u).float()
        # both within half a step and a few units of the exponential of 64 bits: a step apart at most
        off = (dgrads["h"].float() - ref).abs()
        n = int(a.offsets[-1]) if a.capacity == 0 else a.n_rows
        assert bool((off[:n] <= 2.0 ** -7 * ref[:n].abs()).all())
        a.h = dgrads["h"]
        if wl.shared_ff:
            a.h_s = dgrads["h_s"]
    a.backward(t["dy"])
    torch.cuda.synchronize()
    for name, v in a.grads().items():
        assert torch.equal(v, b.grads()[name]), name
    assert b.x is None and b.x_perm is None
    # a second step gives the same
    first = {n: v.clone() for n, v in b.grads().items()}
    b.hook = None
    b.forward(t["x"], t["w_gate"], t["w_up"], t["w_down"], **kw, **(dict(x8=q) if x8 else {}))
    b.backward(t["dy"])
    assert all(torch.equal(v, first[n]) for n, v in b.grads().items())


def test_layer_keeps_half_the_memory():
    T, d, E, k, F = 2048, 1024, 8, 4, 1024
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF) * 0.05
    x, ws = rand(T, d), (rand(E, d, F), rand(E, d, F), rand(E, F, d))
    idx = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    p = torch.full((T, k), 1 / k, device="cuda")
    held = {}
    for act8 in (False, True):
        lay = MoELayer(T, d, E, k, F, routing="given", act8=act8, keep_intermediates=False)
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        lay.forward(x, *ws, topk_idx=idx, topk_w=p)
        held[act8] = torch.cuda.memory_allocated() - before
        lay.backward(torch.randn(T, d, device="cuda").to(BF))
        del lay
    R = T * k
    # y_perm and y in both; x_perm, G, U, H against x8, G8, U8
    assert held[False] >= 2 * (2 * R * d + T * d + 3 * R * F)
    assert held[True] <= 2 * (R * d + T * d) + (T * d + 2 * R * F) * 33 / 32 + (1 << 20)


# ----------------------------------------------------------------------------- block
@pytest.mark.parametrize("opts", [{}, dict(act8=True), dict(act8=True, mxfp8=True), dict(recompute=True)], ids=str)
@pytest.mark.parametrize("first", [False, True])
def test_block(opts, first):
    """Norm, learned router and experts together, as a stack runs them: the
    norm against the oracle on the block's own inputs, its copy handed to the
    layer, the layer's backward into the norm's adjoint."""
    wl = workload("e8_learned_bf16").scaled(T=77, d=256, F=256, E=8)
    t = _inputs(wl)
    g = np.random.default_rng(11)
    res = None if first else round_bf16(3 * g.standard_normal((wl.T, wl.d)))
    w = round_bf16(1 + 0.1 * g.standard_normal(wl.d))
    dh = round_bf16(g.standard_normal((wl.T, wl.d)))
    blk = MoEBlock(wl.T, wl.d, wl.E, wl.k, wl.F, **opts)
    W, R, DH = bf(w), None if first else bf(res), bf(dh)
    args = (t["w_gate"], t["w_up"], t["w_down"])
    y, h = blk.forward(t["x"], R, W, *args, w_r=t["w_r"])
    x = host(t["x"])
    h_ref, n_ref, rs_ref = add_rmsnorm(x, res, w, 1e-6, lambda a: round_bf16(round_f32(a)))
    assert np.array_equal(host(h), h_ref)
    lay = MoELayer(wl.T, wl.d, wl.E, wl.k, wl.F, **opts)
    n = torch.empty_like(t["x"])
    L.moe_add_rmsnorm(h, W, 1e-6, y=n)
    assert np.all(np.abs(host(n) - n_ref) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(n_ref))
    assert torch.equal(lay.forward(n, *args, w_r=t["w_r"]), y)
    dx = blk.backward(t["dy"], DH)
    dn = lay.backward(t["dy"])
    for name, v in lay.grads().items():
        assert torch.equal(v, blk.layer.grads()[name]), name
    rs = host(blk.rstd)
    dx_ref, dw_ref = add_rmsnorm_bwd(host(dn), h_ref, w, rs, dh)
    assert_close(host(dx), dx_ref, "bf16", "dx")
    assert_close(host(blk.dw_norm), dw_ref, "bf16", "dw_norm")
    first_dx = dx.clone()
    blk.forward(t["x"], R, W, *args, w_r=t["w_r"])
    assert torch.equal(blk.backward(t["dy"], DH), first_dx)


def test_two_blocks_against_autograd():
    """A stack of two blocks in binary32 against automatic differentiation of
    the definition in 64 bits: every gradient that a training step takes.
    Sums of up to 160 terms, through four of them in turn: 1e-4 of the largest
    element is 10^3 roundings of 2^-24."""
    T, d, E, k, F = 33, 64, 4, 2, 160
    g = torch.Generator().manual_seed(12)
    rn = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    x0 = rn(T, d)
    par = [dict(w=1 + 0.1 * rn(d), wg=rn(E, d, F, std=d ** -0.5), wu=rn(E, d, F, std=d ** -0.5),
                wd=rn(E, F, d, std=F ** -0.5),
                idx=torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32),
                p=torch.rand(T, k, generator=g)) for _ in range(2)]
    dy, dh = rn(T, d), rn(T, d)
    # the definition, differentiated
    X = x0.double().requires_grad_()
    P = [{n: (v if n == "idx" else v.double().requires_grad_()) for n, v in q.items()} for q in par]
    x, res = X, None
    for q in P:
        h = x if res is None else x + res
        n = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * q["w"]
        y = torch.zeros(T, d, dtype=torch.float64)
        for j in range(k):
            e = q["idx"][:, j].long()
            a, b = (torch.einsum("td,tdf->tf", n, q[m][e]) for m in ("wg", "wu"))
            y = y + q["p"][:, j:j + 1] * torch.einsum("tf,tfd->td", a * torch.sigmoid(a) * b, q["wd"][e])
        x, res = y, h
    ((x * dy).sum() + (res * dh).sum()).backward()
    # the blocks
    C = lambda v: v.detach().float().cuda() if v.dtype != torch.int32 else v.cuda()
    blocks = [MoEBlock(T, d, E, k, F, torch.float32, routing="given") for _ in par]
    cx, cres = C(x0), None
    dev_par = [{n: C(v) for n, v in q.items()} for q in par]
    for blk, q in zip(blocks, dev_par):
        cx, cres = blk.forward(cx, cres, q["w"], q["wg"], q["wu"], q["wd"], topk_idx=q["idx"], topk_w=q["p"])
    close = lambda got, ref, name: np.testing.assert_allclose(host(got), ref.detach().numpy(), rtol=0,
                                                              atol=1e-4 * float(ref.detach().abs().max()), err_msg=name)
    close(cx, x, "y")
    close(cres, res, "h")
    up, along = C(dy), C(dh)
    for blk, q in list(zip(blocks, P))[::-1]:
        dx = blk.backward(up, along)
        grads = blk.layer.grads()
        for name, ref in (("dw_gate", "wg"), ("dw_up", "wu"), ("dw_down", "wd"), ("dtopk_w", "p")):
            close(grads[name], q[ref].grad, name)
        close(blk.dw_norm, q["w"].grad, "dw_norm")
        up = along = dx          # the sum's gradient is that of both of its terms
    close(up, X.grad, "dx")


def test_block_captured_and_replayed():
    """Forward and backward of a block in one graph, replayed beside eager runs
    of the same buffers' inputs."""
    wl = workload("e8_learned_bf16").scaled(T=130, d=256, F=256, E=8)
    t = _inputs(wl)
    w = bf(np.ones(wl.d))
    args = (t["w_gate"], t["w_up"], t["w_down"])
    res = t["dy"].clone()

    def step(blk):
        y, h = blk.forward(t["x"], res, w, *args, w_r=t["w_r"])
        return y, h, blk.backward(t["dy"], t["x"])

    eager = MoEBlock(wl.T, wl.d, wl.E, wl.k, wl.F, act8=True)
    held = MoEBlock(wl.T, wl.d, wl.E, wl.k, wl.F, act8=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(held)
    for i in range(3):
        t["x"].copy_(torch.roll(t["x"], 1, 0))
        want = [v.clone() for v in step(eager)] + [v.clone() for v in eager.layer.grads().values()]
        graph.replay()
        torch.cuda.synchronize()
        got = list(out) + list(held.layer.grads().values())
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("act8", [False, True])
def test_mxfp8_layer_releases_its_step(act8):
    """With keep_intermediates=False nothing but the gradients is left of a
    step, and a second step peaks where the first did."""
    T, d, E, k, F = 2048, 1024, 8, 4, 1024
    g = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF) * 0.05
    x, dy, ws = rand(T, d), rand(T, d), (rand(E, d, F), rand(E, d, F), rand(E, F, d))
    idx = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    p = torch.full((T, k), 1 / k, device="cuda")
    lay = MoELayer(T, d, E, k, F, routing="given", mxfp8=True, act8=act8, keep_intermediates=False)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    peaks = []
    for _ in range(3):
        torch.cuda.reset_peak_memory_stats()
        lay.forward(x, *ws, topk_idx=idx, topk_w=p)
        lay.backward(dy)
        peaks.append(torch.cuda.max_memory_allocated())
        left = torch.cuda.memory_allocated() - before
        # a cached block may be up to 1 MiB larger than what it is given for; a tensor of R x d is 16
        assert left <= sum(v.numel() * v.element_size() for v in lay.grads().values()) + (8 << 20)
    assert max(peaks) <= peaks[0] + (8 << 20)


def test_block_of_mxfp8_experts_with_given_routing():
    """No 8-bit rows of n are kept here: the layer's gradients are those of the
    same layer called by itself."""
    wl = workload("e128_uniform_bf16").scaled(**SMALL)
    t = _inputs(wl)
    kw = dict(topk_idx=t["topk_idx"], topk_w=t["topk_w"])
    args, W = (t["w_gate"], t["w_up"], t["w_down"]), bf(np.linspace(0.5, 1.5, wl.d))
    opts = dict(routing="given", mxfp8=True, act8=True)
    blk, lay = MoEBlock(wl.T, wl.d, wl.E, wl.k, wl.F, **opts), MoELayer(wl.T, wl.d, wl.E, wl.k, wl.F, **opts)
    n = torch.empty_like(t["x"])
    L.moe_add_rmsnorm(t["x"], W, 1e-6, y=n)
    for _ in range(2):
        y, _ = blk.forward(t["x"], None, W, *args, **kw)
        assert blk.n8 is None and torch.equal(y, lay.forward(n, *args, **kw))
        dx, dn = blk.backward(t["dy"]), lay.backward(t["dy"])
        for name, v in lay.grads().items():
            assert torch.equal(v, blk.layer.grads()[name]), name
        want, dw = torch.empty_like(dx), torch.empty_like(W)
        L.moe_add_rmsnorm_bwd(dn, t["x"], W, blk.rstd, want, dw=dw, ws=blk.ws_norm)
        assert torch.equal(dx, want) and torch.equal(blk.dw_norm, dw)


@pytest.mark.parametrize("act8", [False, True])
def test_block_fed_its_own_output_without_a_residual(act8):
    """x is the block's own y buffer, which the pass writes: h, which is x then,
    must still be x when the backward reads it."""
    wl = workload("e128_uniform_bf16").scaled(T=33, d=256, F=256, E=8)
    t = _inputs(wl)
    kw = dict(topk_idx=t["topk_idx"], topk_w=t["topk_w"])
    args, W = (t["w_gate"], t["w_up"], t["w_down"]), bf(np.linspace(0.5, 1.5, wl.d))
    mk = lambda: MoEBlock(wl.T, wl.d, wl.E, wl.k, wl.F, routing="given", act8=act8)
    a, b = mk(), mk()
    y, _ = a.forward(t["x"], None, W, *args, **kw)
    x = y.clone()
    y_a, h_a = a.forward(y, None, W, *args, **kw)
    y_b, h_b = b.forward(x, None, W, *args, **kw)
    assert torch.equal(y_a, y_b) and torch.equal(h_a, x) and h_b is x
    dx_a, dx_b = a.backward(t["dy"]), b.backward(t["dy"])
    assert torch.equal(dx_a, dx_b) and torch.equal(a.dw_norm, b.dw_norm)


@pytest.mark.parametrize("opts", [{}, dict(act8=True), dict(act8=True, mxfp8=True), dict(act8=True, capacity=8),
                                  dict(act8=True, shared_ff=256)], ids=str)
def test_block_without_tokens(opts):
    """A rank that is given no token: empty outputs, and gradients of zero."""
    d, E, k, F = 256, 4, 2, 256
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF) * 0.05
    kw = {}
    if "shared_ff" in opts:
        kw = dict(w_gate_s=rand(d, 256), w_up_s=rand(d, 256), w_down_s=rand(256, d))
    blk = MoEBlock(0, d, E, k, F, routing="given", **opts)
    e = torch.empty(0, d, dtype=BF, device="cuda")
    idx, p = torch.empty(0, k, dtype=torch.int32, device="cuda"), torch.empty(0, k, device="cuda")
    y, h = blk.forward(e, e.clone(), rand(d), rand(E, d, F), rand(E, d, F), rand(E, F, d), topk_idx=idx, topk_w=p, **kw)
    dx = blk.backward(torch.empty_like(e))
    assert y.shape == h.shape == dx.shape == (0, d)
    grads = dict(blk.layer.grads(), dw_norm=blk.dw_norm)
    for name, v in grads.items():
        assert not bool(v.any()), name
