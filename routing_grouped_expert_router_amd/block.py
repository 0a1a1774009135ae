"""One pre-norm MoE block on one GPU: the residual addition with its norm, and
the expert layer, forward and backward.

  forward   h = x + res, n = rmsnorm(h) * w_norm, y = MoELayer(n): returns
            (y, h), the next block's x and res
  backward  the layer's backward gives the gradient of n; the norm's adjoint
            adds what arrives at h along the residual stream and returns the
            gradient of x and res (one tensor: they enter as a sum)

With ``act8=True`` the norm writes n also as MXFP8 rows, which is all the layer
keeps of it (see ``layer``; nothing where its MXFP8 experts alone read n): the
bf16 n is released after the forward.

Memory: h and the reciprocal roots stay from the forward to the backward. The
buffers are allocated by the first pass and reused by later ones.
"""
from __future__ import annotations

import torch

from . import _lib as L
from .layer import MoELayer


class MoEBlock:
    def __init__(self, T: int, d: int, E: int, k: int, F: int, dtype=torch.bfloat16, eps: float = 1e-6,
                 device: str = "cuda", **layer_opts):
        """layer_opts go to MoELayer (routing, recompute, shared_ff, mxfp8,
        act8, ...)."""
        self.layer = MoELayer(T, d, E, k, F, dtype, device=device, **layer_opts)
        self.T, self.d, self.eps, self.dtype, self.dev = T, d, eps, dtype, torch.device(device)
        e = lambda *s, dt=dtype: torch.empty(*s, dtype=dt, device=self.dev)
        self.rstd = e(T, dt=torch.float32)
        self.n = self.h = self.n8 = self._sum = None
        if self.layer.has_bwd:
            self.ws_norm = e(max(L.moe_add_rmsnorm_bwd_workspace_bytes(T, d), 16), dt=torch.uint8)
            self.dx, self.dw_norm = e(T, d), e(d)

    def forward(self, x, res, w_norm, *weights, **kw):
        """x and res [T, d] (res None: the first block, whose stream is x
        itself, which the backward reads again); weights and the rest as MoELayer.forward takes them after x.
        Returns (y, h)."""
        lay = self.layer
        if self.n is None:
            self.n = torch.empty(self.T, self.d, dtype=self.dtype, device=self.dev)
        if lay.reads_x8 and self.n8 is None:
            self.n8 = lay._rows8(self.T, self.d)
        # the layer writes over its own last y: as x without res it is copied first
        own = res is None and lay.y is not None and x.data_ptr() == lay.y.data_ptr()
        if res is None and not own:
            self.h = x
        else:
            if self._sum is None:
                self._sum = torch.empty(self.T, self.d, dtype=self.dtype, device=self.dev)
            self.h = self._sum.copy_(x) if own else self._sum
        self.w_norm = w_norm
        L.moe_add_rmsnorm(x, w_norm, self.eps, res=res, h=None if res is None else self.h, y=self.n, q=self.n8,
                          rstd=self.rstd)
        lay._mark("add_rmsnorm")
        if lay.reads_x8:
            kw["x8"] = self.n8
        y = lay.forward(self.n, *weights, **kw)
        if lay.act8:
            self.n = None
        return y, self.h

    def backward(self, dy, dh=None):
        """dy: gradient of y; dh: what arrives at h from the blocks above
        (None: nothing). Returns the gradient of x (and of res); w_norm's is
        left in dw_norm, the layer's in layer.grads()."""
        dn = self.layer.backward(dy)
        L.moe_add_rmsnorm_bwd(dn, self.h, self.w_norm, self.rstd, self.dx, dw=self.dw_norm, dh=dh, ws=self.ws_norm)
        self.layer._mark("add_rmsnorm_bwd")
        return self.dx
