"""Mixture-of-experts feed-forward layer on FP8 products, as a sequence of C-ABI
calls (every arithmetic step runs in the library's kernels).

    h | u = x W13[e]^T,  a = act(h) u,  y = a W2[e]^T        for each chosen e
    out[t] = residual[t] + sum over t's choices of w y

Fine-grained scales (1x128 groups times 128x128 blocks).  The forward pass:

  fp8_experts_sort             rows in expert order from the choices
  fp8_experts_gather           codes of x in that order (or the codes a norm
                               has written, moved)
  fp8_gemm_group_experts       h | u, one [M, 2 ffn] product
  fp8_act_checkpoint           codes of a; with keep=True also h and u in 8 bits
  fp8_gemm_group_experts       y
  fp8_experts_combine          out

and ``backward``, the gradients of x and of the routing weights (the experts'
weights stay as they are; their transposed codes are made once, backward=True):

  fp8_experts_combine_backward codes of w dout in expert order, dw = <dout, y>
  fp8_gemm_group_experts       da = (w dout) W2
  fp8_act_checkpoint_backward  codes of dh | du from the 8-bit checkpoints
  fp8_gemm_group_experts       dx rows = dh | du times W13
  fp8_experts_combine          dx, each token's rows added

The experts' weights get no gradient.  A call with keep=True holds h and u in 8 bits
and y, which dw reads, in bf16: ffn 2048 and d 7168 are 4.2 KB of checkpoints and
14.3 KB of y a row.

Ids outside [0, experts) drop their choice (experts of another device, a full
expert): it adds nothing and its gradients are zero.
"""
from __future__ import annotations

import torch

import fp8_quantized_gemm_gb300 as F


class ExpertsMLP:
    """w13 [E, 2 ffn, d] (gate rows, then up rows), w2 [E, d, ffn]; d and ffn
    multiples of 128, E at most 256.  sfmt: F.SCALE_F32 or SCALE_UE8M0, of the
    products' operands; keep_sfmt: of the checkpoints."""

    def __init__(self, w13: torch.Tensor, w2: torch.Tensor, act: int = F.ACT_SILU,
                 sfmt: int = F.SCALE_F32, backward: bool = False, keep_sfmt: int = F.SCALE_F32):
        e, ffn2, d = w13.shape
        ffn = ffn2 // 2
        if d % 128 or ffn2 % 256 or w2.shape != (e, d, ffn):
            raise ValueError("w13 [E, 2 ffn, d], w2 [E, d, ffn], d and ffn multiples of 128")
        self.E, self.d, self.ffn = e, d, ffn
        self.act, self.sfmt, self.keep_sfmt = act, sfmt, keep_sfmt
        self.w13, self.w2 = self._blocks(w13), self._blocks(w2)
        self.w13t = self._blocks(w13.transpose(1, 2)) if backward else None
        self.w2t = self._blocks(w2.transpose(1, 2)) if backward else None
        self.saved = None

    @staticmethod
    def _dt(sfmt):
        return torch.float32 if sfmt == F.SCALE_F32 else torch.uint8

    def _blocks(self, w):
        """Codes and 128x128 block scales of [E, N, K] weights."""
        e, n, k = w.shape
        q = torch.empty((e, n, k), dtype=torch.uint8, device=w.device)
        s = torch.empty((e, n // 128, k // 128), dtype=self._dt(self.sfmt), device=w.device)
        F.fp8_quantize_block(w.contiguous().view(e * n, k), F.E4M3, self.sfmt, q.view(e * n, k),
                             s.view(e * n // 128, k // 128))
        return q, s

    def _codes(self, m, k, dev, sfmt=None):
        sfmt = self.sfmt if sfmt is None else sfmt
        return (torch.empty((m, k), dtype=torch.uint8, device=dev),
                torch.empty((k // 128, m), dtype=self._dt(sfmt), device=dev))

    def _product(self, q, s, w, offsets):
        out = torch.empty((q.shape[0], w[0].shape[1]), dtype=torch.bfloat16, device=q.device)
        F.fp8_gemm_group_experts(q, s, *w, self.sfmt, offsets, out)
        return out

    def __call__(self, x, ids, weights, *, x_scales=None, residual=None, keep=False):
        """out [T, d] bf16.  x [T, d] bf16, or its codes with x_scales (1x128
        groups of sfmt); ids [T, S] int32 or int64; weights fp32 [T, S];
        residual bf16 [T, d].  keep: hold what ``backward`` reads."""
        t, s = ids.shape
        m, dev, n = t * s, x.device, self.ffn
        out = torch.empty((t, self.d), dtype=torch.bfloat16, device=dev)
        self.saved = (None, None, weights, None, None) if keep and t == 0 else None
        if t == 0:
            return out
        offsets = torch.empty(self.E + 1, dtype=torch.int32, device=dev)
        rows = torch.empty((t, s), dtype=torch.int32, device=dev)
        F.fp8_experts_sort(ids, self.E, offsets, rows)
        xq, xs = self._codes(m, self.d, dev)
        F.fp8_experts_gather(x, rows, q=xq, scales=xs, sfmt=self.sfmt, x_scales=x_scales)
        hu = self._product(xq, xs, self.w13, offsets)
        aq, as_ = self._codes(m, n, dev)
        kept = {}
        if keep:
            for name in ("h", "u"):
                kept[name + "_q"], kept[name + "_scales"] = self._codes(m, n, dev, self.keep_sfmt)
        F.fp8_act_checkpoint(hu[:, :n], hu[:, n:], self.act, aq, scales=as_, sfmt=self.sfmt,
                             keep_sfmt=self.keep_sfmt, valid_rows=offsets[self.E:], **kept)
        y = self._product(aq, as_, self.w2, offsets)
        F.fp8_experts_combine(y, rows, weights, out, residual=residual)
        if keep:
            self.saved = (offsets, rows, weights, y, kept)
        return out

    def backward(self, dout):
        """(dx [T, d] bf16, d_weights fp32 [T, S]) for the gradient dout [T, d]
        of the last call, made with keep=True.  (The residual's gradient is dout.)"""
        if self.w13t is None or self.saved is None:
            raise ValueError("backward needs ExpertsMLP(backward=True) and a call with keep=True")
        offsets, rows, weights, y, kept = self.saved
        if rows is None:  # no tokens
            return torch.empty_like(dout, dtype=torch.bfloat16), torch.empty_like(weights)
        m, dev, n = rows.numel(), dout.device, self.ffn
        dw = torch.empty_like(weights)
        yq, ys = self._codes(m, self.d, dev)
        F.fp8_experts_combine_backward(dout, rows, weights, x=y, d_weights=dw, q=yq, scales=ys,
                                       sfmt=self.sfmt)
        da = self._product(yq, ys, self.w2t, offsets)
        gq, gs = self._codes(m, 2 * n, dev)
        F.fp8_act_checkpoint_backward(da, self.act, **kept, keep_sfmt=self.keep_sfmt,
                                      dh_q=gq[:, :n], du_q=gq[:, n:], fmt=F.E4M3,
                                      dh_scales=gs[:n // 128], du_scales=gs[n // 128:],
                                      sfmt=self.sfmt, valid_rows=offsets[self.E:])
        rows_dx = self._product(gq, gs, self.w13t, offsets)
        dx = torch.empty((rows.shape[0], self.d), dtype=torch.bfloat16, device=dev)
        F.fp8_experts_combine(rows_dx, rows, None, dx)
        return dx, dw
