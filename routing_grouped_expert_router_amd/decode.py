"""The pre-norm MoE block's decode step on one GPU, with the experts in 4 bits.

  h = x + res, n = rmsnorm(h) * w_norm, learned router (GEMM, softmax, top-k),
  y = the chosen experts' weighted products with MXFP4 weights (plus a shared
  expert's); returns (y, h), the next block's x and res

for one token up to ``max_tokens``, which times k is at most
MOE_W4_MAX_SLOTS. The expert weights are quantised once, here; the bf16 ones
are not kept. Five launches for a token (norm, router GEMM, top-k, gate/up, down
with the sum), six for a batch (the sum by itself), two or three more with a
shared expert; no host synchronisation, and no allocation unless rows of an
earlier step's h come back in another place, so a step can be captured into a
graph; a graph then owns this decoder's buffers.
"""
from __future__ import annotations

import torch

from . import _lib as L


def quantize_experts(w: torch.Tensor) -> L.W4Tensor:
    """w [E, K, N] bf16 as MXFP4 along K."""
    out = L.W4Tensor.empty(*w.shape, device=w.device)
    L.moe_w4_quantize(w, out)
    return out


def _lies_in(v: torch.Tensor, buf: torch.Tensor) -> bool:
    return 0 <= v.data_ptr() - buf.data_ptr() < buf.numel() * buf.element_size()


class MoEDecoder:
    def __init__(self, w_norm, w_r, w_gate, w_up, w_down, k: int, max_tokens: int, eps: float = 1e-6,
                 w_gate_s=None, w_up_s=None, w_down_s=None):
        """w_norm [d], w_r [d, E], w_gate and w_up [E, d, F], w_down [E, F, d];
        the shared expert's w_gate_s, w_up_s [d, Fs], w_down_s [Fs, d]."""
        E, d, F = w_gate.shape
        if max_tokens < 1 or max_tokens * k > L.MOE_W4_MAX_SLOTS:
            raise ValueError(f"1 <= max_tokens * k <= {L.MOE_W4_MAX_SLOTS}")
        if not (w_gate_s is None) == (w_up_s is None) == (w_down_s is None):
            raise ValueError("a shared expert needs all three of its weights")
        self.w_norm, self.w_r, self.k, self.eps = w_norm, w_r, k, eps
        self.T, self.d, self.E, self.F, self.dev = max_tokens, d, E, F, w_gate.device
        self.w4 = [quantize_experts(w) for w in (w_gate, w_up, w_down)]
        T = max_tokens
        e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=self.dev)
        self.h, self.n, self.y = e(T, d), e(T, d), e(T, d)
        self.logits, self.topk_w = e(T, E, dt=torch.float32), e(T, k, dt=torch.float32)
        self.topk_idx = e(T, k, dt=torch.int32)
        need = L.moe_experts_w4_workspace_bytes(T, k, d, F)
        self.shared = None
        if w_gate_s is not None:
            self.shared = [quantize_experts(w.unsqueeze(0)) for w in (w_gate_s, w_up_s, w_down_s)]
            need = max(need, L.moe_experts_w4_workspace_bytes(T, 1, d, w_gate_s.shape[1]))
            self.one_idx = torch.zeros(T, 1, dtype=torch.int32, device=self.dev)
            self.one_w = torch.ones(T, 1, device=self.dev)
        self.ws = e(need, dt=torch.uint8)   # the calls run in order on one stream

    def step(self, x, res=None):
        """x and res [T, d] bf16, T <= max_tokens (res None: the first block).
        Returns (y, h), views of this decoder's buffers (h is x itself without
        res), overwritten by the next step. They, and rows of them, may come
        back as x and res: a view that the step would overwrite before it is
        done with it is copied first."""
        T = x.shape[0]
        if T > self.T:
            raise ValueError(f"{T} tokens, made for {self.T}")
        if T == 0:
            return self.y[:0], x if res is None else self.h[:0]
        n, y, h = self.n[:T], self.y[:T], self.h[:T]
        if res is None:
            if _lies_in(x, self.y):      # what is returned as h
                h.copy_(x)
            else:
                h = x
        else:                            # the rows of h in another place than they are read from
            x, res = (v.clone() if _lies_in(v, self.h) and v.data_ptr() != h.data_ptr() else v for v in (x, res))
        L.moe_add_rmsnorm(x, self.w_norm, self.eps, res=res, h=None if res is None else h, y=n)
        logits, idx, p = self.logits[:T], self.topk_idx[:T], self.topk_w[:T]
        L.moe_router_gemm(n, self.w_r, logits)
        L.moe_route(logits, self.k, idx, p)
        add = None
        if self.shared is not None:
            L.moe_experts_w4(n, self.one_idx[:T], self.one_w[:T], *self.shared, y, self.ws)
            add = y
        L.moe_experts_w4(n, idx, p, *self.w4, y, self.ws, y_add=add)
        return y, h
