"""The 4-bit experts on the GPU: the quantiser bit for bit, the products and
the decode step against the float64 oracle on the quantised weights.

Tolerance of y: its own rounding, half a bf16 step (2^-8); H's in two bf16
terms, 2^-16 of H; a sum of K products carries at most K roundings of 2^-24 of
the sum of their magnitudes (2 K where H has two terms); the sigmoid a few (8)
units. The oracle gives the sums of
magnitudes."""
import numpy as np
import pytest
import torch

import oracle.moe as om
from oracle.norm import add_rmsnorm
from oracle.numerics import f64_to_bf16_bits, round_bf16, round_f32
from oracle.w4 import experts, w4_dequantize, w4_quantize
from routing_grouped_expert_router_amd import _lib as L
from routing_grouped_expert_router_amd.decode import MoEDecoder, quantize_experts

from parity import dev, host

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U = 2.0 ** -24


def bf(a):
    return dev(f64_to_bf16_bits(a), "bf16")


def laid_out(codes, scales):
    """The documented layout, written from its index formula."""
    M, K, N = codes.shape
    c = codes.reshape(M, K // 128, 4, 16, 2, N // 16, 16)      # m, step, g, j, half, tile, n
    q = (c[:, :, :, :, 0] | c[:, :, :, :, 1] << 4).transpose(0, 4, 1, 2, 5, 3)
    k5 = -(-K // 512)
    s = np.zeros((M, k5 * 16, N), dtype=np.uint8)
    s[:, :K // 32] = scales
    s = s.reshape(M, k5, 4, 4, N // 16, 16).transpose(0, 4, 1, 3, 5, 2)   # m, tile, chunk, g, n, step
    return np.ascontiguousarray(q).reshape(-1), np.ascontiguousarray(s).reshape(-1)


@pytest.mark.parametrize("M,K,N", [(1, 128, 16), (3, 640, 48), (2, 512, 80), (1, 2048, 128), (5, 384, 64)])
def test_quantize_bitwise(M, K, N):
    g = np.random.default_rng([1, M, K, N])
    w = g.standard_normal((M, K, N)) * np.exp2(g.integers(-40, 40, (M, 1, N)))
    w[0, :32, 0] = 0                                            # an all-zero block
    w[0, 32:64, 1] = np.ldexp(1.0, -131)                        # subnormal ones
    w[0, :32, 2] = 4.0                                          # scale 1: every tie, and saturation
    w[0, 1:21, 2] = [.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6.5, 7.5, 6, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -7.9, 0.0, -0.0]
    w[0, 64:96, 3] = np.ldexp(1.5, 127)                         # the largest binade
    w = round_bf16(w)
    t = quantize_experts(bf(w))
    q, s = laid_out(*w4_quantize(w))
    assert np.array_equal(host(t.s), s)
    assert np.array_equal(host(t.q), q)


def problem(T, d, E, k, F, seed, holes=0.0, twice=False, hot=False):
    g = np.random.default_rng([seed, T, d, E, k, F])
    ws = [round_bf16(g.standard_normal(s) * std) for s, std in
          (((E, d, F), d ** -0.5), ((E, d, F), d ** -0.5), ((E, F, d), F ** -0.5))]
    x = round_bf16(g.standard_normal((T, d)))
    idx = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    if hot:
        idx[:, 0] = 0                                           # one expert takes every token
    if twice:
        idx[:, -1] = idx[:, 0]                                  # the same expert in two slots
    if holes:
        idx[g.random((T, k)) < holes] = -1
        idx[0, 0] = E                                           # past the last expert
        idx[T // 2] = -1                                        # a token without any
    p = (g.random((T, k)) + 0.05).astype(np.float32)
    p /= p.sum(1, keepdims=True)
    return x, idx, p, ws, g


def check(y, ref, mag, hmag, K_d, K_F):
    tol = mag * (2.0 ** -16 + (2 * K_F + 20) * U) + hmag * (K_d + 8) * U
    assert np.all(np.isfinite(y))
    assert np.all(np.abs(y - ref) <= 2.0 ** -8 * (np.abs(ref) + tol) + tol)


CASES = [  # T, d, E, k, F: one token; slots up to the experts; more; rows past 16 and 64; K of 1 to 9 steps; one
    # expert; a thousand tokens
    (1, 256, 8, 2, 128), (1, 2048, 4, 4, 1024), (1, 128, 1, 1, 128), (3, 1152, 12, 4, 640), (2, 128, 4, 4, 512),
    (16, 256, 4, 1, 256), (17, 256, 1, 1, 384), (70, 640, 3, 2, 128), (150, 128, 2, 2, 256), (9, 1024, 64, 8, 128),
    (64, 256, 128, 4, 128), (40, 384, 8, 8, 1152), (1, 4096, 2, 2, 128), (130, 1152, 3, 2, 384), (200, 256, 2, 2, 640),
    (1000, 640, 8, 4, 128), (900, 1152, 3, 2, 256),
]


@pytest.mark.parametrize("T,d,E,k,F", CASES)
@pytest.mark.parametrize("kind", ["plain", "holes", "twice", "hot", "add"])
def test_products(T, d, E, k, F, kind):
    x, idx, p, ws, g = problem(T, d, E, k, F, 2, holes=0.3 if kind == "holes" else 0.0, twice=kind == "twice",
                               hot=kind == "hot")
    add = round_bf16(g.standard_normal((T, d))) if kind in ("add", "holes") else None
    w4 = [quantize_experts(bf(w)) for w in ws]
    vals = [w4_dequantize(*w4_quantize(w)) for w in ws]
    ref, mag, hmag = experts(x, idx, p, *vals, lambda a: a, add)
    y = torch.full((T, d), float("nan"), dtype=BF, device="cuda")
    ws_buf = torch.full((L.moe_experts_w4_workspace_bytes(T, k, d, F),), 0xFF, dtype=torch.uint8, device="cuda")
    P = dev(p, "f32")
    if kind == "holes":
        P[dev(idx, "i32") < 0] = float("nan")                   # the weight of an empty slot is not read
    args = (bf(x), dev(idx, "i32"), P, *w4)
    A = None if add is None else bf(add)
    L.moe_experts_w4(*args, y, ws_buf, y_add=A)
    check(host(y), ref, mag, hmag, d, F)
    if kind == "holes":
        assert torch.equal(y[T // 2], A[T // 2])
    first = y.clone()
    ws_buf.fill_(0x7F)
    L.moe_experts_w4(*args, y, ws_buf, y_add=A)
    assert torch.equal(y, first)                                # the same bits whatever the workspace held
    if A is not None:
        L.moe_experts_w4(*args, A, ws_buf, y_add=A)             # y over y_add
        assert torch.equal(A, first)


def test_batch_rows_do_not_depend_on_each_other():
    """A token alone and in a batch of one row per expert differ by nothing
    but the order of sums: the same bits, as the order is the same."""
    T, d, E, k, F = 12, 512, 16, 3, 256
    x, idx, p, ws, _ = problem(T, d, E, k, F, 3)
    w4 = [quantize_experts(bf(w)) for w in ws]
    buf = torch.empty(L.moe_experts_w4_workspace_bytes(T, k, d, F), dtype=torch.uint8, device="cuda")
    X, I, P = bf(x), dev(idx, "i32"), dev(p, "f32")
    y, one = torch.empty(T, d, dtype=BF, device="cuda"), torch.empty(1, d, dtype=BF, device="cuda")
    L.moe_experts_w4(X, I, P, *w4, y, buf)
    for t in range(T):
        L.moe_experts_w4(X[t:t + 1], I[t:t + 1], P[t:t + 1], *w4, one, buf)
        assert torch.equal(one[0], y[t]), t


def test_infinite_token_stays_in_its_row():
    T, d, E, k, F = 6, 256, 4, 2, 128
    x, idx, p, ws, _ = problem(T, d, E, k, F, 4)
    w4 = [quantize_experts(bf(w)) for w in ws]
    buf = torch.empty(L.moe_experts_w4_workspace_bytes(T, k, d, F), dtype=torch.uint8, device="cuda")
    X, I, P = bf(x), dev(idx, "i32"), dev(p, "f32")
    a, b = (torch.empty(T, d, dtype=BF, device="cuda") for _ in range(2))
    L.moe_experts_w4(X, I, P, *w4, a, buf)
    X[2] = float("inf")
    X[4, 3] = float("nan")
    L.moe_experts_w4(X, I, P, *w4, b, buf)
    keep = [0, 1, 3, 5]
    assert torch.equal(a[keep], b[keep]) and not bool(b[4].isfinite().any())


def test_largest_batch():
    """The slot limit, one expert with every row."""
    T, d, E, k, F = 1024, 128, 8, 4, 128
    x, idx, p, ws, _ = problem(T, d, E, k, F, 5, hot=True)
    w4 = [quantize_experts(bf(w)) for w in ws]
    vals = [w4_dequantize(*w4_quantize(w)) for w in ws]
    ref, mag, hmag = experts(x, idx, p, *vals, lambda a: a)
    y = torch.empty(T, d, dtype=BF, device="cuda")
    buf = torch.empty(L.moe_experts_w4_workspace_bytes(T, k, d, F), dtype=torch.uint8, device="cuda")
    L.moe_experts_w4(bf(x), dev(idx, "i32"), dev(p, "f32"), *w4, y, buf)
    check(host(y), ref, mag, hmag, d, F)


@pytest.mark.parametrize("T,d,E,k,F", [(4096, 128, 1, 1, 128), (256, 128, 1000, 16, 128), (1, 128, 1024, 16, 128)])
def test_limits(T, d, E, k, F):
    """Every slot on one expert, and the most experts and slots a token."""
    x, idx, p, ws, _ = problem(T, d, E, k, F, 7)
    w4 = [quantize_experts(bf(w)) for w in ws]
    vals = [w4_dequantize(*w4_quantize(w)) for w in ws]
    ref, mag, hmag = experts(x, idx, p, *vals, lambda a: a)
    y = torch.empty(T, d, dtype=BF, device="cuda")
    buf = torch.empty(L.moe_experts_w4_workspace_bytes(T, k, d, F), dtype=torch.uint8, device="cuda")
    L.moe_experts_w4(bf(x), dev(idx, "i32"), dev(p, "f32"), *w4, y, buf)
    check(host(y), ref, mag, hmag, d, F)


def test_offsets_past_32_bits():
    """A pool of more than 4 GB of codes: its last experts give what they give
    in a pool of their own."""
    E, d, F, k, T = 1024, 2048, 4096, 2, 3
    g = torch.Generator(device="cuda").manual_seed(8)
    rnd = lambda n: torch.randint(0, 256, (n,), generator=g, device="cuda", dtype=torch.uint8)
    x = torch.randn(T, d, generator=g, device="cuda").to(BF)
    idx = torch.tensor([[1023, 1], [1022, 1023], [0, 1021]], dtype=torch.int32, device="cuda")
    p = torch.rand(T, k, generator=g, device="cuda")
    used, at = torch.unique(idx.view(-1).long(), return_inverse=True)
    big, small = [], []
    for K, N in ((d, F), (d, F), (F, d)):
        nq, ns = L.moe_w4_code_bytes(K, N), L.moe_w4_scale_bytes(K, N)
        q = torch.zeros(E, nq, dtype=torch.uint8, device="cuda")
        q[used] = rnd(len(used) * nq).view(len(used), nq)
        s = torch.full((E, ns), 119, dtype=torch.uint8, device="cuda")
        assert E * nq > 1 << 31
        big.append(L.W4Tensor(q.view(-1), s.view(-1), E, K, N))
        small.append(L.W4Tensor(q[used].contiguous().view(-1), s[used].contiguous().view(-1), len(used), K, N))
    out = []
    for w4, i in ((big, idx), (small, at.view(T, k).to(torch.int32))):
        y = torch.empty(T, d, dtype=BF, device="cuda")
        buf = torch.empty(L.moe_experts_w4_workspace_bytes(T, k, d, F), dtype=torch.uint8, device="cuda")
        L.moe_experts_w4(x, i, p, *w4, y, buf)
        out.append(y)
    assert bool(out[0].isfinite().all()) and bool((out[0] != 0).any()) and torch.equal(out[0], out[1])


# ----------------------------------------------------------------------------- decode step
def decoder(shared, max_tokens=20):
    g = np.random.default_rng(6)
    d, E, k, F, Fs = 256, 16, 4, 384, 128
    r = lambda *s, std=1.0: round_bf16(g.standard_normal(s) * std)
    w = dict(w_norm=r(d, std=0.1) + 1, w_r=r(d, E, std=d ** -0.5), w_gate=r(E, d, F, std=d ** -0.5),
             w_up=r(E, d, F, std=d ** -0.5), w_down=r(E, F, d, std=F ** -0.5))
    w["w_norm"] = round_bf16(w["w_norm"])
    if shared:
        w.update(w_gate_s=r(d, Fs, std=d ** -0.5), w_up_s=r(d, Fs, std=d ** -0.5), w_down_s=r(Fs, d, std=Fs ** -0.5))
    return MoEDecoder(**{n: bf(v) for n, v in w.items()}, k=k, max_tokens=max_tokens), w, k, g


@pytest.mark.parametrize("T", [1, 2, 20])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("first", [False, True])
def test_decode_step(T, shared, first):
    """Norm, router and experts as a serving loop runs them."""
    dec, w, k, g = decoder(shared)
    d = 256
    x = round_bf16(g.standard_normal((T, d)))
    res = None if first else round_bf16(2 * g.standard_normal((T, d)))
    y, h = dec.step(bf(x), None if first else bf(res))
    h_ref, n_ref, _ = add_rmsnorm(x, res, w["w_norm"], 1e-6, lambda a: round_bf16(round_f32(a)))
    assert np.array_equal(host(h), h_ref)
    n = host(dec.n[:T])
    assert np.all(np.abs(n - n_ref) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(n_ref))
    logits = host(dec.logits[:T])
    assert np.all(np.abs(logits - n @ w["w_r"]) <= d * U * (np.abs(n) @ np.abs(w["w_r"])))
    idx, p = om.route(logits.astype(np.float32), k)
    assert np.array_equal(host(dec.topk_idx[:T]), idx)
    p = host(dec.topk_w[:T])
    q = lambda a: w4_dequantize(*w4_quantize(a))
    vals = [q(w[n_]) for n_ in ("w_gate", "w_up", "w_down")]
    tol_add, add = 0.0, None
    if shared:
        sv = [q(w[n_][None]) for n_ in ("w_gate_s", "w_up_s", "w_down_s")]
        add, m, hm = experts(n, np.zeros((T, 1), dtype=int), np.ones((T, 1)), *sv, lambda a: a)
        tol_add = m * (2.0 ** -16 + 276 * U) + hm * (d + 8) * U
        tol_add = tol_add + 2.0 ** -8 * (np.abs(add) + tol_add)      # stored in bf16 in between
    ref, mag, hmag = experts(n, idx, p, *vals, lambda a: a, add)
    tol = tol_add + mag * (2.0 ** -16 + (768 + 20) * U) + hmag * (d + 8) * U
    assert np.all(np.abs(host(y) - ref) <= 2.0 ** -8 * (np.abs(ref) + tol) + tol)


def test_decode_step_captured_and_replayed():
    dec, _, _, g = decoder(True)
    eager, _, _, _ = decoder(True)
    x, res = bf(g.standard_normal((3, 256))), bf(g.standard_normal((3, 256)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dec.step(x, res)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = dec.step(x, res)
    for i in range(4):
        x.copy_(torch.roll(x, 1, 1))
        want = [v.clone() for v in eager.step(x, res)]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(h, want[1]), i
        eager.step(res, x)                                       # other eager work between the replays


def test_decode_step_of_no_tokens():
    dec, _, _, _ = decoder(True)
    e = torch.empty(0, 256, dtype=BF, device="cuda")
    for out in (dec.step(e), dec.step(e, e)):
        assert out[0].shape == out[1].shape == (0, 256)
    with pytest.raises(ValueError, match="made for 20"):
        dec.step(torch.empty(21, 256, dtype=BF, device="cuda"))


def test_decode_on_another_stream():
    dec, _, _, g = decoder(False)
    eager, _, _, _ = decoder(False)
    x = bf(g.standard_normal((5, 256)))
    want = eager.step(x)[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = dec.step(x)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("shared", [False, True])
def test_decode_step_fed_its_own_output_without_a_residual(shared):
    """x is the decoder's own y, which the step writes: the h it returns is still x."""
    dec, _, _, g = decoder(shared)
    other, _, _, _ = decoder(shared)
    y, _ = dec.step(bf(g.standard_normal((5, 256))))
    x = y.clone()
    y1, h1 = dec.step(y)
    y2, h2 = other.step(x)
    assert torch.equal(y1, y2) and torch.equal(h1, x) and h2 is x
    z = y1.clone()
    y1, h1 = dec.step(y1[1:3])                                   # some of its rows
    assert torch.equal(h1, z[1:3])
    y1, h1 = dec.step(y1, h1)
    y2, h2 = other.step(z[1:3].clone())
    y2, h2 = other.step(y2.clone(), h2)
    assert torch.equal(y1, y2) and torch.equal(h1, h2)


@pytest.mark.parametrize("rows", [slice(0, 12), slice(1, 20), slice(7, 8)], ids=str)
def test_decode_step_fed_rows_of_its_own_output(rows):
    """Sequences that end leave a batch: the rows that stay are read from where
    other rows' h goes."""
    dec, _, _, g = decoder(False)
    other, _, _, _ = decoder(False)
    x, res = bf(g.standard_normal((20, 256))), bf(g.standard_normal((20, 256)))
    y, h = dec.step(x, res)
    want = other.step(y[rows].clone(), h[rows].clone())
    want = other.step(want[1].clone(), want[0].clone())
    got = dec.step(y[rows], h[rows])
    got = dec.step(got[1], got[0])                               # h as x: its own rows again
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_decode_step_without_a_residual_captured():
    """The copy of an own output inside a graph, replayed beside eager steps."""
    dec, _, _, g = decoder(True)
    eager, _, _, _ = decoder(True)
    x = bf(g.standard_normal((3, 256)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dec.step(dec.step(x)[0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = dec.step(dec.step(x)[0])
    for i in range(4):
        x.copy_(torch.roll(x, 1, 1))
        first = eager.step(x)[0].clone()
        want = eager.step(first)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(h, first), i
