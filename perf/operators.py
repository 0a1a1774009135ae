"""What is measured of the operators around the expert layer: the residual
addition with its root-mean-square norm (forward, with an optional MXFP8 copy,
and backward), the expert activations kept in 8 bits between the passes, the
layer input rebuilt from its 8-bit copy, and the experts' products with 4-bit
weights for decode batches.

``run`` computes them in their plain form, or where ``own`` is set through the
framework's entry points. Both take what ``prepare`` gives.
"""
import math

import torch

own = False

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6


def listed():
    return [
        # one token of a decode step entering the layer: latency alone
        dict(name="norm_one_token", op="norm", T=1, d=2048, dtype="bf16", res=True, mx=False),
        # the training batch of the headline layer, with the 8-bit copy that its backward keeps
        dict(name="norm_train_mx", op="norm", T=16384, d=2048, dtype="bf16", res=True, mx=True),
        # a ragged batch in binary32 at a width that fills no whole wave, first layer (no residual yet)
        dict(name="norm_f32_odd", op="norm", T=1237, d=1000, dtype="f32", res=False, mx=False),
        # its backward in the headline layer, with the residual stream's gradient
        dict(name="norm_bwd_train", op="norm_bwd", T=16384, d=2048, dtype="bf16", dh=True),
        # a short wide batch in binary32, the last norm of a stack (nothing arrives along the residual)
        dict(name="norm_bwd_wide_f32", op="norm_bwd", T=333, d=8200, dtype="f32", dh=False),
        # the experts of a small layer, rows uneven, two experts without rows
        dict(name="experts8_small", op="experts8", R=1021, d=256, F=256, E=16, skew=0.5, empty=2),
        # the experts of the headline layer: 16384 tokens, four of 128 experts each
        dict(name="experts8_headline", op="experts8", R=65536, d=2048, F=1024, E=128, skew=0.0, empty=0),
        # the layer input of a short batch rebuilt in its experts' rows
        dict(name="restore_short", op="restore", T=257, d=1024, k=2, E=8),
        # the same for the headline layer
        dict(name="restore_headline", op="restore", T=16384, d=2048, k=4, E=128),
        # one token through four of 128 experts: latency, and the weights of four experts
        dict(name="w4_one_token", op="w4", T=1, d=2048, F=1024, E=128, k=4, add=False, holes=0.0),
        # a decode batch that reaches most of the experts with a row or two each
        dict(name="w4_decode_batch", op="w4", T=64, d=2048, F=1024, E=128, k=4, add=False, holes=0.0),
        # a padded batch of a small pool (some slots hold no expert, one token none at all) beside a shared expert
        dict(name="w4_small_pool", op="w4", T=37, d=2048, F=1024, E=8, k=4, add=True, holes=0.2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "experts8", "restore", "w4", "w4"])
    if op in ("norm", "norm_bwd"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        mx = op == "norm" and dtype == "bf16" and rng.random() < 0.5
        d = 128 * _log(rng, 1, 64) if mx else 8 * _log(rng, 8, 1100)
        T = _log(rng, 1, max(1, min(16384, (1 << 24) // d)))
        if op == "norm":
            return dict(op=op, T=T, d=d, dtype=dtype, res=rng.random() < 0.7, mx=mx)
        return dict(op=op, T=T, d=d, dtype=dtype, dh=rng.random() < 0.7)
    if op == "experts8":
        E = rng.choice([1, 4, 8, 32, 64])
        return dict(op=op, R=_log(rng, 1, 16384), d=256 * rng.randint(1, 8), F=256 * rng.randint(1, 4), E=E,
                    skew=rng.choice([0.0, 0.5]), empty=rng.randint(0, E // 4))
    if op == "restore":
        E = rng.choice([8, 16, 64, 128])
        return dict(op=op, T=_log(rng, 1, 8192), d=128 * _log(rng, 1, 32), k=rng.randint(1, 6), E=E)
    E = rng.choice([1, 8, 16, 32, 64, 128])
    d, F = 128 * _log(rng, 1, 32), 128 * _log(rng, 1, 16)
    if E > 32:
        d, F = min(d, 2048), min(F, 1024)
    return dict(op=op, T=_log(rng, 1, 128), d=d, F=F, E=E, k=rng.randint(1, min(E, 8)), add=rng.random() < 0.3,
                holes=rng.choice([0.0, 0.0, 0.25]))


def _es(case):
    return 4 if case["dtype"] == "f32" else 2


def work(case):
    op = case["op"]
    if op == "norm":
        n, es = case["T"] * case["d"], _es(case)
        # x, res, h, y; the 8-bit copy is written and read back, and its values are written
        return {"bytes": n * es * (2 + 2 * case["res"]) + n * (2 * 33 / 32 + 2) * case["mx"] + 4 * case["T"]
                + case["d"] * es, "flops": 5 * n}
    if op == "norm_bwd":
        n, es = case["T"] * case["d"], _es(case)
        return {"bytes": n * es * (3 + case["dh"]) + 4 * case["T"] + 2 * case["d"] * es, "flops": 10 * n}
    if op == "experts8":
        R, d, F, E = case["R"], case["d"], case["F"], case["E"]
        full = min(E - case["empty"], R)
        # rows in, weights, H of both passes, dG, dU, and the two 8-bit copies written and read
        return {"bytes": 2 * R * d * 2 + 3 * full * d * F * 2 + 4 * R * F * 2 + 2 * 2 * R * F * 33 / 32,
                "flops": 6 * R * d * F}
    if op == "restore":
        n = case["T"] * case["d"]
        return {"bytes": n * 33 / 32 + 2 * n + 2 * n * case["k"] + 4 * case["T"] * case["k"], "flops": n}
    T, d, F, E, k = case["T"], case["d"], case["F"], case["E"], case["k"]
    R = T * k * (1 - case["holes"])
    reached = E * (1 - (1 - 1 / E) ** R)
    return {"bytes": reached * 3 * d * F * 17 / 32 + T * d * 2 * (2 + case["add"]) + 8 * T * k,
            "flops": 6 * R * d * F}


# ------------------------------------------------------------------ formats
def _pow2(code):
    """2^(code - 127) of scale bytes (code 0 stands beside zero codes only)."""
    return (code.to(torch.int32) << 23).view(F32)


def _mx_quantize(v):
    """Codes [R, K] and scale bytes in the framework's layout (the four scales of
    128 values of a row in one word, words of a column group together) of bf16 v."""
    R, K = v.shape
    b = v.float().view(R, K // 32, 32)
    x = (torch.frexp(b.abs().amax(-1))[1] - 9).clamp(-127, 127)
    x = torch.where(b.abs().amax(-1) == 0, torch.full_like(x, -127), x)
    code = (x + 127).to(torch.uint8)
    inv = _pow2(254 - code.to(torch.int32))
    q = (b * inv[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s = code.view(R, K // 128, 4).transpose(0, 1).contiguous()
    return q.view(R, K), s.view(-1)


def _mx_values(q, s):
    R, K = q.shape
    code = s.view(K // 128, R, 4).transpose(0, 1).reshape(R, K // 32, 1)
    return (q.view(torch.float8_e4m3fn).float().view(R, K // 32, 32) * _pow2(code)).view(R, K)


def _w4_quantize(w):
    """4-bit codes and scales of bf16 w [M, K, N]: blocks of 32 along K share 2^X, X = floor(log2 amax) - 2.

    Codes lie as the product reads them, [M][N/16][K/128][4 blocks][16 columns][16 bytes], two values a byte, the
    lower k in the low half; scales as [M][N/16][ceil(K/512)][4 blocks][16 columns][4 steps of 128]."""
    M, K, N = w.shape
    b = w.float().view(M, K // 32, 32, N)
    amax = b.abs().amax(2)
    x = torch.where(amax == 0, torch.full_like(amax, -127, dtype=torch.int32), torch.frexp(amax)[1] - 3)
    code = (x.clamp(-127, 127) + 127).to(torch.uint8)
    b = b * _pow2(254 - code.to(torch.int32))[:, :, None]
    v = b.abs()
    c = sum((v > m).to(torch.uint8) for m in (0.25, 1.25, 2.5, 5.0))
    c = c + sum((v >= m).to(torch.uint8) for m in (0.75, 1.75, 3.5)) + (b < 0).to(torch.uint8) * 8
    c = c.view(M, K // 128, 4, 16, 2, N // 16, 16)
    q = (c[:, :, :, :, 0] | c[:, :, :, :, 1] << 4).permute(0, 4, 1, 2, 5, 3).contiguous()
    k5 = -(-K // 512)
    code = torch.nn.functional.pad(code, (0, 0, 0, k5 * 16 - K // 32)).view(M, k5, 4, 4, N // 16, 16)
    return q.view(-1), code.permute(0, 4, 1, 3, 5, 2).contiguous().view(-1)


def _w4_values(q, s, K, N):
    """Values [M, K, N] in 32 bits of codes and scales [M, ...] laid out as above."""
    M, k5 = q.shape[0], -(-K // 512)
    c = q.view(M, N // 16, K // 128, 4, 16, 16, 1)
    c = torch.cat([c & 15, c >> 4], -1).permute(0, 2, 3, 5, 6, 1, 4).reshape(M, K // 32, 32, N)
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    table = torch.cat([table, -table])
    code = s.view(M, N // 16, k5, 4, 16, 4).permute(0, 2, 5, 3, 1, 4).reshape(M, k5 * 16, 1, N)
    return (table[c.int()] * _pow2(code[:, : K // 32])).view(M, K, N)


# ------------------------------------------------------------------ inputs
def _rand(g, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _empty(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device=DEV)


def _counts(case, seed):
    """Rows of each expert: popularity rank^-skew over a shuffled order, the last `empty` ranks without any."""
    g = torch.Generator().manual_seed(seed)
    E, R = case["E"], case["R"]
    p = torch.arange(1, E + 1, dtype=torch.float64) ** -case["skew"]
    if case["empty"]:
        p[-case["empty"]:] = 0
    p = p[torch.randperm(E, generator=g)]
    return torch.bincount(torch.multinomial(p, R, replacement=True, generator=g), minlength=E)


def _routes(g, T, E, k):
    return torch.rand(T, E, generator=g, device=DEV).topk(k, dim=1).indices.to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("norm", "norm_bwd"):
        T, d, dt = case["T"], case["d"], F32 if case["dtype"] == "f32" else BF16
        s["w"] = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(dt)
        # a residual stream: a few channels far larger than the others
        wide = 1 + 20 * (torch.rand(d, generator=g, device=DEV) < 0.01).float()
        if op == "norm":
            s["x"] = _rand(g, T, d, dtype=dt)
            s["res"] = (torch.randn(T, d, generator=g, device=DEV) * wide).to(dt) if case["res"] else None
            s["h"] = _empty(T, d, dtype=dt) if case["res"] else None
            s["y"], s["rstd"] = _empty(T, d, dtype=dt), _empty(T, dtype=F32)
            if case["mx"]:
                s["q"], s["s"] = _empty(T, d, dtype=torch.uint8), _empty(T * d // 32, dtype=torch.uint8)
                s["y8"] = _empty(T, d)
        else:
            s["dy"], s["dh"] = _rand(g, T, d, dtype=dt), _rand(g, T, d, dtype=dt) if case["dh"] else None
            s["h"] = (torch.randn(T, d, generator=g, device=DEV) * wide).to(dt)
            s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
            s["dx"], s["dw"] = _empty(T, d, dtype=dt), _empty(d, dtype=dt)
            # room for the sums of up to 1024 parts of the batch, as a user's plan holds it
            s["ws"] = _empty(1024 * d, dtype=F32)
    elif op == "experts8":
        R, d, F, E = case["R"], case["d"], case["F"], case["E"]
        n = _counts(case, seed)
        s["cap"] = int(n.max())
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).to(torch.int32).to(DEV)
        s["x"], s["dy"] = _rand(g, R, d), _rand(g, R, d)
        s["w_gate"], s["w_up"] = (_rand(g, E, d, F, std=d ** -0.5) for _ in range(2))
        s["w_down"] = _rand(g, E, F, d, std=F ** -0.5)
        for name in ("h", "dg", "du", "h_again"):
            s[name] = _empty(R, F)
        for name in ("g8", "u8"):
            s[name] = _empty(R, F, dtype=torch.uint8), _empty(R * F // 32, dtype=torch.uint8)
    elif op == "restore":
        T, d, k, E = case["T"], case["d"], case["k"], case["E"]
        s["q"], s["s"] = _mx_quantize(_rand(g, T, d))
        slots = _routes(g, T, E, k).view(-1).sort(stable=True).indices
        s["row_of"] = torch.empty_like(slots).scatter_(0, slots, torch.arange(T * k, device=DEV)).to(torch.int32)
        s["x"], s["x_perm"] = _empty(T, d), _empty(T * k, d)
    else:
        T, d, F, E, k = case["T"], case["d"], case["F"], case["E"], case["k"]
        for name, K, N in (("w_gate", d, F), ("w_up", d, F), ("w_down", F, d)):
            s[name] = _w4_quantize(_rand(g, E, K, N, std=K ** -0.5))
        s["x"] = _rand(g, T, d)
        idx = _routes(g, T, E, k)
        hole = torch.rand(T, k, generator=g, device=DEV) < case["holes"]
        if case["holes"]:
            hole[T // 2] = True   # a padding token: no expert at all
        s["idx"] = torch.where(hole, torch.full_like(idx, -1), idx)
        p = torch.rand(T, k, generator=g, device=DEV) + 0.1
        s["p"] = p / p.sum(1, keepdim=True)
        s["add"] = _rand(g, T, d) if case["add"] else None
        s["y"] = _empty(T, d)
        # room for every slot's hidden row and for its output row in a few parts
        s["ws"] = _empty(T * k * (32 * d + 16 * F) + 65536, dtype=torch.uint8)
    return s


# ------------------------------------------------------------------ passes
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "experts8": _own_experts8, "restore": _own_restore,
                "w4": _own_w4}[op](state)
    return {"norm": _norm, "norm_bwd": _norm_bwd, "experts8": _experts8, "restore": _restore, "w4": _w4}[op](state)


def _norm(s):
    x, dt = s["x"], s["x"].dtype
    h = x if s["res"] is None else (x.float() + s["res"].float()).to(dt)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(1) + EPS)
    y = (hf * rstd[:, None] * s["w"].float()).to(dt)
    out = dict(y=y, rstd=rstd)
    if s["res"] is not None:
        out["h"] = h
    if s["case"]["mx"]:
        out["y8"] = _mx_values(*_mx_quantize(y)).to(BF16)
    return out


def _norm_bwd(s):
    n = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - n * (g * n).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dict(dx=dx.to(s["h"].dtype), dw=(dy * n).sum(0).to(s["h"].dtype))


def _by_expert(s, rows, w):
    """rows[r] @ w[expert of r] in 32 bits, over rows padded to the fullest expert's count."""
    off, R = s["offsets"].long(), rows.shape[0]
    r = torch.arange(R, device=DEV)
    e = torch.searchsorted(off[1:].contiguous(), r, right=True)
    at = r - off[e]
    padded = torch.zeros(w.shape[0], s["cap"], rows.shape[1], device=DEV)
    padded[e, at] = rows.float()
    return torch.bmm(padded, w)[e, at]


def _experts8(s):
    g = _by_expert(s, s["x"], s["w_gate"].float()).to(BF16)
    u = _by_expert(s, s["x"], s["w_up"].float()).to(BF16)
    h = (g.float() * torch.sigmoid(g.float()) * u.float()).to(BF16)
    g, u = _mx_values(*_mx_quantize(g)), _mx_values(*_mx_quantize(u))   # what is kept between the passes
    dh = _by_expert(s, s["dy"], s["w_down"].float().transpose(1, 2).contiguous())
    sg = torch.sigmoid(g)
    return dict(h=h, dg=(dh * u * sg * (1 + g * (1 - sg))).to(BF16), du=(dh * g * sg).to(BF16),
                h_again=(g * sg * u).to(BF16))


def _restore(s):
    x = _mx_values(s["q"], s["s"]).to(BF16)
    x_perm = torch.empty_like(s["x_perm"])
    x_perm[s["row_of"].long()] = x.repeat_interleave(s["case"]["k"], 0)
    return dict(x=x, x_perm=x_perm)


def _silu(v):
    return v * torch.sigmoid(v)


def _w4(s):
    c = s["case"]
    T, d, F, E, k = c["T"], c["d"], c["F"], c["E"], c["k"]
    x, p = s["x"].float(), s["p"] * (s["idx"] >= 0)
    at = s["idx"].clamp(min=0).long()
    tables = [(q.view(E, -1), sc.view(E, -1), K, N)
              for (q, sc), K, N in ((s["w_gate"], d, F), (s["w_up"], d, F), (s["w_down"], F, d))]
    if T * k < E:      # the chosen experts' weights, one copy a slot
        wg, wu, wd = (_w4_values(q[at.view(-1)], sc[at.view(-1)], K, N) for q, sc, K, N in tables)
        xs = x.repeat_interleave(k, 0)[:, None]
        y = torch.bmm(_silu(torch.bmm(xs, wg)) * torch.bmm(xs, wu), wd).view(T, k, d)
        y = (y * p[..., None]).sum(1)
    else:              # every token through every expert, weighted by zero where it is not routed
        wg, wu, wd = (_w4_values(q, sc, K, N) for q, sc, K, N in tables)
        xs = x.expand(E, T, d)
        y = torch.bmm(_silu(torch.bmm(xs, wg)) * torch.bmm(xs, wu), wd)
        share = torch.zeros(T, E, device=DEV).scatter_add_(1, at, p)
        y = (y * share.t()[..., None]).sum(0)
    if s["add"] is not None:
        y = y + s["add"].float()
    return dict(y=y.to(BF16))


# ------------------------------------------------------------------ the framework's calls
def _own_norm(s):
    from routing_grouped_expert_router_amd import _lib as L
    q = L.MxTensor(s["q"], s["s"]) if s["case"]["mx"] else None
    L.moe_add_rmsnorm(s["x"], s["w"], EPS, res=s["res"], h=s["h"], y=s["y"], q=q, rstd=s["rstd"])
    out = dict(y=s["y"], rstd=s["rstd"])
    if s["res"] is not None:
        out["h"] = s["h"]
    if q is not None:
        L.moe_mx_dequantize(q, s["y8"])
        out["y8"] = s["y8"]
    return out


def _own_norm_bwd(s):
    from routing_grouped_expert_router_amd import _lib as L
    L.moe_add_rmsnorm_bwd(s["dy"], s["h"], s["w"], s["rstd"], s["dx"], dw=s["dw"], dh=s["dh"], ws=s["ws"])
    return dict(dx=s["dx"], dw=s["dw"])


def _own_experts8(s):
    from routing_grouped_expert_router_amd import _lib as L
    c = s["case"]
    shape = (L.MOE_BF16, c["E"], c["d"], c["F"], c["R"], 0, s["offsets"])
    g8, u8 = L.MxTensor(*s["g8"]), L.MxTensor(*s["u8"])
    L.moe_grouped_gemm_ckpt(L.make_gg_desc(L.MOE_GG_FWD_GATE_UP, *shape, x_perm=s["x"], w_gate=s["w_gate"],
                                           w_up=s["w_up"], h=s["h"]), g8, u8)
    L.moe_grouped_gemm_ckpt(L.make_gg_desc(L.MOE_GG_DGRAD_DOWN, *shape, dy_perm=s["dy"], w_down=s["w_down"],
                                           dg=s["dg"], du=s["du"], h=s["h_again"]), g8, u8)
    return dict(h=s["h"], dg=s["dg"], du=s["du"], h_again=s["h_again"])


def _own_restore(s):
    from routing_grouped_expert_router_amd import _lib as L
    L.moe_permute_from_mx(L.MxTensor(s["q"], s["s"]), s["case"]["k"], s["row_of"], None, s["x_perm"], x=s["x"])
    return dict(x=s["x"], x_perm=s["x_perm"])


def _own_w4(s):
    from routing_grouped_expert_router_amd import _lib as L
    c = s["case"]
    wg, wu = (L.W4Tensor(*s[n], c["E"], c["d"], c["F"]) for n in ("w_gate", "w_up"))
    wd = L.W4Tensor(*s["w_down"], c["E"], c["F"], c["d"])
    L.moe_experts_w4(s["x"], s["idx"], s["p"], wg, wu, wd, s["y"], s["ws"], y_add=s["add"])
    return dict(y=s["y"])


# ------------------------------------------------------------------ 64 bits
def _two(e):
    """2^e in 64 bits from its exponent field (a device's pow may be off in the last place)."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _grid(v, man, low, top):
    """v (64 bits) on a grid of `man` mantissa bits, least exponent `low`, largest value `top`; ties to even."""
    e = torch.frexp(v.abs().clamp(min=2.0 ** low))[1] - 1
    step = _two(e - man)
    return (torch.round(v / step) * step).clamp(-top, top)


def _exact_mx(v):
    """Values of the MXFP8 copy of bf16 v, block by block."""
    b = v.double().unflatten(1, (-1, 32))
    amax = b.abs().amax(2, keepdim=True)
    unit = _two((torch.frexp(amax)[1] - 9).clamp(min=-127))
    return (_grid(b / unit, 3, -6, 448.0) * unit).flatten(1)


def exact(case, seed):
    s = prepare(case, seed)
    D = {n: v.double() for n, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    op = case["op"]
    if op == "norm":
        full = D["x"] if s["res"] is None else D["x"] + D["res"]
        h = full.to(s["x"].dtype).double()
        rms = (h.pow(2).sum(1) / case["d"] + EPS).sqrt()
        y = h / rms[:, None] * D["w"]
        out = dict(y=y, rstd=1 / rms)
        if s["res"] is not None:
            out["h"] = full
        if case["mx"]:
            out["y8"] = _exact_mx(y.to(BF16))
        return out
    if op == "norm_bwd":
        r = D["rstd"][:, None]
        t = D["dy"] * D["w"]
        dx = r * t - D["h"] * r ** 3 * (t * D["h"]).sum(1, keepdim=True) / case["d"]
        return dict(dx=dx + D["dh"] if s["dh"] is not None else dx, dw=(D["dy"] * D["h"] * r).sum(0))
    if op == "experts8":
        out = {n: torch.zeros(case["R"], case["F"], dtype=torch.float64, device=DEV)
               for n in ("h", "dg", "du", "h_again")}
        off = s["offsets"].tolist()
        for e in range(case["E"]):
            i = slice(off[e], off[e + 1])
            if off[e] == off[e + 1]:
                continue
            g, u = ((D["x"][i] @ s[n][e].double()).to(BF16) for n in ("w_gate", "w_up"))
            out["h"][i] = u.double() * g.double() / (1 + torch.exp(-g.double()))
            g, u = _exact_mx(g), _exact_mx(u)
            sig = 1 / (1 + torch.exp(-g))
            dh = D["dy"][i] @ s["w_down"][e].double().t()
            out["h_again"][i] = g * sig * u
            out["du"][i] = dh * g * sig
            out["dg"][i] = dh * u * (sig + g * sig * (1 - sig))
        return out
    if op == "restore":
        T, d, k = case["T"], case["d"], case["k"]
        byte = s["q"].int()
        e, m = byte >> 3 & 15, (byte & 7).double()
        v = torch.where(e == 0, m / 512, (1 + m / 8) * _two(e - 7))
        v = torch.where(byte > 127, -v, v)
        col = torch.arange(d, device=DEV)
        word = (col // 128)[None] * T + torch.arange(T, device=DEV)[:, None]
        x = v * _two(s["s"][4 * word + (col % 128 // 32)[None]].int() - 127)
        x_perm = torch.zeros(T * k, d, dtype=torch.float64, device=DEV)
        x_perm[s["row_of"].long().view(T, k)] = x[:, None].expand(T, k, d)
        return dict(x=x, x_perm=x_perm)
    T, d, F, E, k = (case[n] for n in ("T", "d", "F", "E", "k"))
    y = D["add"].clone() if s["add"] is not None else torch.zeros(T, d, dtype=torch.float64, device=DEV)
    idx = s["idx"].cpu()

    def weights(name, e, K, N):
        kk, nn = torch.arange(K, device=DEV)[:, None], torch.arange(N, device=DEV)[None]
        q, sc = (t.view(E, -1)[e] for t in s[name])
        lane = nn % 16 + 16 * (kk % 128 // 32)
        c = q[((nn // 16 * (K // 128) + kk // 128) * 64 + lane) * 16 + kk % 32 // 2].int() >> 4 * (kk % 2) & 15
        m = c & 7
        v = torch.where(m < 2, m / 2.0, (1 + (m & 1) / 2.0) * _two((m >> 1) - 1))
        x = sc[((nn // 16 * -(-K // 512) + kk // 512) * 64 + lane) * 4 + kk % 512 // 128].int() - 127
        return torch.where(c > 7, -v, v) * _two(x)

    for e in sorted(set(idx[idx >= 0].tolist())):
        t, j = (v.to(DEV) for v in torch.nonzero(idx == e, as_tuple=True))
        a, b = (D["x"][t] @ weights(n, e, d, F) for n in ("w_gate", "w_up"))
        rows = (a * b / (1 + torch.exp(-a))) @ weights("w_down", e, F, d)
        y.index_add_(0, t, D["p"][t, j][:, None] * rows)
    return dict(y=y)
