"""Pre-norm FP8 feed-forward block of a transformer, as a sequence of C-ABI
calls (every arithmetic step runs in the library's kernels).

    r = x + stream                                     the residual stream
    y = r / rms(r) * g                                 the norm
    z = y W1^T + b1,  a = act(z)                       up projection
    out = a W2^T + r                                   down projection

``PreNormMLPTrainer`` is the training step with delayed scaling: E4M3 codes for
activations and weights, E5M2 for gradients (Flax guide 3.3), an (amax history,
scale) pair per GEMM operand (5.1), each tensor quantized with the scale left
by the step before (2.3).  Since every scale is known before its tensor, each
operand reaches memory only as codes, written by the kernel that forms it:

  forward   fp8_rmsnorm_quantize         r, 1/rms, codes of y
            fp8_gemm_tensor_epilogue     bf16 z, codes of a       (bias, act)
            fp8_gemm_tensor_epilogue     out                      (residual r)
  backward  fp8_gemm_tensor_act_backward codes of dz, db1         (through act)
            fp8_gemm_tensor_grouped      dy = dz W1, dW1 = dz^T y, dW2 = dout^T a
            fp8_rmsnorm_backward         dr = norm gradient + dout, dg, and the
                                         E5M2 codes of dr: the output gradient
                                         that the block below starts from
  update    fp8_delayed_state_update_multi, fp8_adamw_multi (which also writes
            the next step's weight codes)

Blocks are chained from the top one down: ``drq`` holds the codes of dr under
``drq_scale``, the scale of their own step (``update`` replaces the live one), and
the block below takes both with dr, before this block's next backward pass:

  top.step(x1, dout, s1)
  below.step(x0, top.dr, s0, doutq=top.drq, dout_scale=top.drq_scale)

``PreNormMLP`` is the forward pass alone with fine-grained scales (1x128 groups
times 128x128 blocks), from one decoded token to a prefill chunk.

Buffers are allocated once (device memory through torch); the calls go to the
current stream, and a step can be captured as a CUDA graph.
"""
from __future__ import annotations

import torch

import fp8_quantized_gemm_gb300 as F

# delayed-scaling states: input of W1, W1, a, W2, dz, dout of this block, and
# dr, which the block below receives as its dout
Y, K1, A, K2, DZ, DOUT, DR = range(7)


class PreNormMLPTrainer:
    def __init__(self, w1: torch.Tensor, b1: torch.Tensor, w2: torch.Tensor, gain: torch.Tensor,
                 tokens: int, act: int = F.ACT_GELU_TANH, eps: float = 1e-5, history: int = 16,
                 lr=1e-4, beta1=0.9, beta2=0.999, adam_eps=1e-8, weight_decay=0.01):
        dev = w1.device
        ffn, d = w1.shape
        if w2.shape != (d, ffn) or b1.shape != (ffn,) or gain.shape != (d,):
            raise ValueError("w1 [ffn, d], b1 [ffn], w2 [d, ffn], gain [d]")
        self.act, self.eps, self.tokens = act, eps, tokens
        self.hp = dict(lr=lr, beta1=beta1, beta2=beta2, eps=adam_eps, weight_decay=weight_decay)
        new = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device=dev)  # noqa: E731
        u8, bf = torch.uint8, torch.bfloat16
        # fp32 masters: W1, W2, gain, b1
        self.params = [p.float().contiguous().clone() for p in (w1, w2, gain, b1)]
        self.grads = [torch.empty_like(p) for p in self.params]
        self.m = [torch.zeros_like(p) for p in self.params]
        self.v = [torch.zeros_like(p) for p in self.params]
        self.hist = torch.zeros((7, history), device=dev)
        self.scale = torch.ones(7, device=dev)
        self.amax = torch.zeros(7, device=dev)
        self.drq_scale = torch.ones(1, device=dev)
        T = tokens
        self.r, self.out, self.dr = (new(T, d, t=bf) for _ in range(3))
        self.inv, self.z, self.dy = new(T), new(T, ffn, t=bf), new(T, d, t=bf)
        self.yq, self.doutq, self.drq = (new(T, d, t=u8) for _ in range(3))
        self.aq, self.dzq = new(T, ffn, t=u8), new(T, ffn, t=u8)
        self.w1q, self.w2q = new(ffn, d, t=u8), new(d, ffn, t=u8)
        self.norm_ws = new(F.fp8_rmsnorm_backward_workspace(T, d), t=u8)
        self.act_ws = new(F.fp8_act_backward_workspace(T, ffn), t=u8)
        self.step_dev = torch.zeros(1, dtype=torch.int64, device=dev)
        wq = {0: (self.w1q, K1), 1: (self.w2q, K2)}
        self.items = [
            F.adamw_item(p, g, m, v, **(dict(q=wq[i][0], q_scale=self._s(wq[i][1]),
                                             q_amax=self._a(wq[i][1]), q_fmt=F.E4M3)
                                        if i in wq else {}))
            for i, (p, g, m, v) in enumerate(zip(self.params, self.grads, self.m, self.v))]
        # the first step's weight codes, by current scaling
        for i, (q, slot) in wq.items():
            F.fp8_amax(self.params[i], self._a(slot))
            F.fp8_quantize_tensor(self.params[i], F.E4M3, q, amax_in=self._a(slot),
                                  scale_out=self._s(slot))

    def _s(self, i):
        return self.scale[i:i + 1]

    def _a(self, i):
        return self.amax[i:i + 1]

    def forward(self, x: torch.Tensor, stream: torch.Tensor | None = None):
        """out [tokens, d] bf16 for the branch x and the stream it joins."""
        w1, w2, gain, b1 = self.params
        F.fp8_rmsnorm_quantize(x, gain, self.eps, F.E4M3, self.yq, residual=stream, sum_out=self.r,
                               scale=self._s(Y), amax_out=self._a(Y), inv_rms=self.inv)
        F.fp8_gemm_tensor_epilogue(self.yq, F.E4M3, self.w1q, F.E4M3, self._s(Y), self._s(K1), None,
                                   bias=b1, act=self.act, pre_out=self.z, q=self.aq, q_fmt=F.E4M3,
                                   q_scale=self._s(A), q_amax=self._a(A))
        F.fp8_gemm_tensor_epilogue(self.aq, F.E4M3, self.w2q, F.E4M3, self._s(A), self._s(K2),
                                   self.out, residual=self.r)
        return self.out

    def backward(self, dout: torch.Tensor, doutq=None, dout_scale=None):
        """dr [tokens, d] bf16, the gradient of x and of the stream.  doutq,
        dout_scale: E5M2 codes of dout where the block above has written them
        (its ``drq`` and ``drq_scale``)."""
        if (doutq is None) != (dout_scale is None):
            raise ValueError("doutq and dout_scale come together")
        E4, E5, MN = F.E4M3, F.E5M2, F.MN_MAJOR
        self.drq_scale.copy_(self._s(DR))  # what drq is written under below
        if doutq is None:
            doutq, dout_scale = self.doutq, self._s(DOUT)
            F.fp8_quantize_tensor(dout, E5, doutq, scale=dout_scale, amax_out=self._a(DOUT))
        dw1, dw2, dgain, db1 = self.grads
        F.fp8_gemm_tensor_act_backward(doutq, E5, self.w2q, E4, dout_scale, self._s(K2), self.z,
                                       self.act, q=self.dzq, q_fmt=E5, q_scale=self._s(DZ),
                                       q_amax=self._a(DZ), dbias=db1, workspace=self.act_ws,
                                       b_layout=MN)
        P = F.gemm_problem
        F.fp8_gemm_tensor_grouped([
            P(self.dzq, E5, self.w1q, E4, self._s(DZ), self._s(K1), self.dy, b_layout=MN),
            P(self.dzq, E5, self.yq, E4, self._s(DZ), self._s(Y), dw1, a_layout=MN, b_layout=MN),
            P(doutq, E5, self.aq, E4, dout_scale, self._s(A), dw2, a_layout=MN, b_layout=MN)])
        F.fp8_rmsnorm_backward(self.dy, self.r, self.inv, self.params[2], self.dr, d_residual=dout,
                               dw=dgain, q=self.drq, fmt=E5, scale=self._s(DR),
                               amax_out=self._a(DR), workspace=self.norm_ws)
        return self.dr

    def update(self):
        """The histories take this step's maxima (which fixes the next step's
        scales), then AdamW, which writes the weights' next codes under them."""
        F.fp8_delayed_state_update_multi([
            F.delayed_item(self.hist[i], self._s(i), self._a(i),
                           F.E5M2 if i in (DZ, DOUT, DR) else F.E4M3) for i in range(7)])
        F.fp8_adamw_multi(self.items, self.step_dev, **self.hp)

    def step(self, x, dout, stream=None, doutq=None, dout_scale=None):
        self.forward(x, stream)
        self.backward(dout, doutq, dout_scale)
        self.update()


class PreNormMLP:
    """Forward pass with fine-grained scales (sfmt: F.SCALE_F32 or SCALE_UE8M0):
    d and ffn multiples of 128."""

    def __init__(self, w1, b1, w2, gain, act: int = F.ACT_GELU_TANH, eps: float = 1e-5,
                 sfmt: int = F.SCALE_F32):
        ffn, d = w1.shape
        if d % 128 or ffn % 128 or w2.shape != (d, ffn):
            raise ValueError("w1 [ffn, d], w2 [d, ffn], both sizes multiples of 128")
        self.act, self.eps, self.sfmt, self.d, self.ffn = act, eps, sfmt, d, ffn
        self.gain, self.b1 = gain.contiguous(), b1.float().contiguous()
        self.st = torch.float32 if sfmt == F.SCALE_F32 else torch.uint8
        self.w = []
        for w in (w1, w2):
            n, k = w.shape
            q = torch.empty((n, k), dtype=torch.uint8, device=w.device)
            s = torch.empty(((n + 127) // 128, k // 128), dtype=self.st, device=w.device)
            F.fp8_quantize_block(w.contiguous(), F.E4M3, sfmt, q, s)
            self.w.append((q, s))

    def __call__(self, x: torch.Tensor, stream: torch.Tensor | None = None):
        """(out, r): out [M, d] bf16 = r + the block's output, r = x + stream."""
        m, dev, u8 = x.shape[0], x.device, torch.uint8
        r = torch.empty_like(x)
        yq, ys = torch.empty((m, self.d), dtype=u8, device=dev), \
            torch.empty((self.d // 128, m), dtype=self.st, device=dev)
        F.fp8_rmsnorm_quantize(x, self.gain, self.eps, F.E4M3, yq, residual=stream, sum_out=r,
                               scales=ys, sfmt=self.sfmt)
        a = torch.empty((m, self.ffn), dtype=torch.bfloat16, device=dev)
        F.fp8_gemm_group_epilogue(yq, ys, *self.w[0], self.sfmt, a, bias=self.b1, act=self.act)
        aq, as_ = torch.empty((m, self.ffn), dtype=u8, device=dev), \
            torch.empty((self.ffn // 128, m), dtype=self.st, device=dev)
        F.fp8_quantize_token_group(a, F.E4M3, self.sfmt, aq, as_)
        out = torch.empty((m, self.d), dtype=torch.bfloat16, device=dev)
        F.fp8_gemm_group_epilogue(aq, as_, *self.w[1], self.sfmt, out, residual=r)
        return out, r
