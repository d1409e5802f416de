"""The token mixer of a hybrid decoder's linear-attention layers, which stands before the expert layer (mx_layer.py) in three
layers of four, out of the operators without a context:

  x W_in^T -> moe_conv (q, k and v) -> moe_head_norm (q and k to unit length) -> moe_delta -> moe_head_norm (gated) -> W_out^T

Each sequence has its state in a slot: the last rows before the convolution, and a [v_dim, k_dim] matrix of each head.  A
batch holds prompts, pieces of prompts or single tokens, in any mixture (``moe.make_seqs``).  The three projections are
bf16 matrix products of torch; everything between them but the two gates' few values a token is the library's.

``python -m int4_expert_streaming_gb300.mx_layer`` times it with the expert layer behind it.
"""
from __future__ import annotations

import torch
import torch.nn.functional as F

import int4_expert_streaming_gb300 as moe


class DeltaMixer:
    """Of `heads` = (k_heads, v_heads, k_dim, v_dim), with C = 2 * k_heads * k_dim + v_heads * v_dim channels, bf16 CUDA
    tensors except where it says fp32:
      w_in     [C + v_heads * v_dim, hidden]: rows of q, k, v and then of the output's gate
      w_gates  [2 * v_heads, hidden]: rows of beta and then of the decay
      conv     [C, 2..4]
      a_log, dt_bias  fp32 [v_heads]: decay's logarithm g = -exp(a_log) * softplus(decay + dt_bias); beta = sigmoid(beta)
      norm     fp32 [v_dim]
      w_out    [hidden, v_heads * v_dim]
    slots states, zeros at first; max_tokens and max_seqs size the buffers.  One call at a time per object, all on one
    stream or ordered by the caller; a captured graph holds the object's buffers and states."""

    def __init__(self, w_in, w_gates, conv, a_log, dt_bias, norm, w_out, heads, slots: int, max_tokens: int,
                 max_seqs: int, eps: float = 1e-6):
        Hk, Hv, dk, dv = self.heads = heads
        self.hidden, self.channels = w_in.shape[1], 2 * Hk * dk + Hv * dv
        inner, C = Hv * dv, self.channels
        for name, t, shape, dtype in (
                ("w_in", w_in, (C + inner, self.hidden), torch.bfloat16), ("w_gates", w_gates, (2 * Hv, self.hidden), torch.bfloat16),
                ("conv", conv, (C, conv.shape[-1]), torch.bfloat16), ("a_log", a_log, (Hv,), torch.float32),
                ("dt_bias", dt_bias, (Hv,), torch.float32), ("norm", norm, (dv,), torch.float32),
                ("w_out", w_out, (self.hidden, inner), torch.bfloat16)):
            if tuple(t.shape) != shape or t.dtype is not dtype:
                raise ValueError(f"{name}: expected {shape} {dtype}, got {tuple(t.shape)} {t.dtype}")
        self.w_in, self.w_gates, self.conv, self.w_out = w_in, w_gates, conv.contiguous(), w_out
        self.rate, self.dt_bias, self.norm = a_log.exp(), dt_bias, norm.contiguous()
        self.unit = moe.make_head_norm_config(moe.MOE_NORM_L2, 1e-6)
        self.gated = moe.make_head_norm_config(moe.MOE_NORM_RMS, eps)
        self.max_tokens, self.max_seqs = max_tokens, max_seqs

        def bf16(*shape):
            return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        self.conv_state = bf16(slots, conv.shape[1] - 1, C)
        self.state = torch.zeros((slots, Hv, dv, dk), device="cuda")
        self.projected, self.mixed, self.o = bf16(max_tokens, C + inner), bf16(max_tokens, C), bf16(max_tokens, Hv, dv)
        self.workspace = torch.empty(moe.moe_delta_workspace(max_tokens, max_seqs, Hk, Hv, dk, dv), dtype=torch.uint8,
                                     device="cuda")

    def forward(self, x, seqs: moe.moe_seqs, y):
        """x [T, hidden] -> y [T, hidden], both bf16, on the current stream.  Rows of no sequence, or of one without a
        slot, get zeros (where x is finite)."""
        T, st = x.shape[0], torch.cuda.current_stream()
        Hk, Hv, dk, dv = self.heads
        if x.shape != (T, self.hidden) or y.shape != x.shape:
            raise ValueError(f"x {tuple(x.shape)} and y {tuple(y.shape)} are not of width {self.hidden}")
        if T > self.max_tokens or seqs.n > self.max_seqs:
            raise ValueError(f"{T} tokens of {seqs.n} sequences, room for {self.max_tokens} of {self.max_seqs}")
        if T == 0:
            return y
        p, m, o = self.projected[:T], self.mixed[:T], self.o[:T]
        torch.mm(x, self.w_in.T, out=p)
        beta, decay = (x @ self.w_gates.T).float().split(Hv, 1)
        g = -self.rate * F.softplus(decay + self.dt_bias)
        moe.moe_conv(p[:, :self.channels], self.conv, m, seqs=seqs, state=self.conv_state, stream=st)
        q, k, v = m.split([Hk * dk, Hk * dk, Hv * dv], 1)
        q, k, v = q.unflatten(1, (Hk, dk)), k.unflatten(1, (Hk, dk)), v.unflatten(1, (Hv, dv))
        moe.moe_head_norm(self.unit, q, q, x2=k, y2=k, stream=st)
        if seqs.offsets_dev or seqs.slot_dev:  # there may be rows that the delta rule leaves as an earlier call left them
            o.zero_()
        moe.moe_delta(q, k, v, g, beta.sigmoid(), self.state, o, dk ** -0.5, seqs, self.workspace, st)
        moe.moe_head_norm(self.gated, o, o, self.norm, p[:, self.channels:].unflatten(1, (Hv, dv)), stream=st)
        return torch.mm(o.flatten(1), self.w_out.T, out=y)
