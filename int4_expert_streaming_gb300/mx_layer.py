"""A routed expert layer in microscaled 4-bit floats, out of the operators without a context:

  logits -> moe_route -> moe_dispatch -> moe_mx_quantise (token rows, in expert order) -> moe_mx_product (gate and up)
         -> moe_mx_quantise (SwiGLU) -> moe_mx_product (down) -> moe_combine

``python -m int4_expert_streaming_gb300.mx_layer`` runs one layer of the 512-expert shapes on random weights and prints
its time, and then that of a decoder layer: the delta rule's mixer (delta_layer.py) and these experts; ``MxLayer`` is the same as a class, and an example of how the calls go together: what is laid out once, what
is sized by the largest batch, and what each call is given.

An e4m3 scale has a narrow range, 2^-9 to 448, so every e4m3 matrix takes a tensor scale beside it: without one, blocks
whose largest value is below 0.006 vanish and those above 2688 saturate.  The weights' are found when they are quantised.
The token rows' and the SwiGLU rows' are given as numbers found beforehand (``tensor_scale`` of the largest value that is
expected), or else measured from each batch.
"""
from __future__ import annotations

import math

import torch

import int4_expert_streaming_gb300 as moe


LARGEST = 6 * 448  # of an e4m3 matrix: the largest code times the largest scale


def tensor_scale(largest: float) -> float:
    """The tensor scale that lets values up to `largest` be written without saturation."""
    return largest / LARGEST


def quantise_weights(w, fmt: int):
    """w [groups, rows, cols] (fp32 or bf16, CUDA) -> (matrix, tensor scales [groups] or None): each group's largest
    weight is brought to the largest product of code and scale."""
    E, N, K = w.shape
    m = moe.make_mx(fmt, N, K, groups=E)
    t = (w.abs().amax((1, 2)).float() / LARGEST).clamp(min=1e-30) if fmt == moe.MOE_MX_E4M3 else None
    moe.moe_mx_quantise(m, w.reshape(E * N, K), tensor_scale=t, stream=torch.cuda.current_stream())
    return m, t


def power_of_two_scale(largest):
    """largest [1] fp32, on the GPU -> the power of two t with t * 1024 <= largest < t * 2048: never saturating, and no
    rounding depends on it, so rows of the same values get the same codes in any batch (as long as their blocks' largest
    values are above 1e-4 of the batch's)."""
    t = (largest * 2.0 ** -10).clamp(2.0 ** -100, 2.0 ** 100)
    return (t.view(torch.int32) & 0x7F800000).view(torch.float32)  # the exponent alone


def largest_of(v, live, parts: int = 1):
    """The largest magnitude of v [rows, parts * n] in each of its parts [parts], over the rows with live [rows, 1]; rows
    that are not finite (their results are not either) are left out."""
    a = torch.linalg.vector_norm(v.view(v.shape[0], parts, -1), math.inf, 2)
    return torch.where(live, a, 0).nan_to_num(0, 0, 0).amax(0).float()


class MxLayer:
    """gate_up [E, 2 * inter, hidden] (gate rows, then up rows of each expert), down [E, hidden, inter]; cfg as of
    make_route_config; max_tokens sizes the buffers.  One call at a time per object.  From hidden or inter of 3841 on a
    batch of few rows may sum its products in another order than a large one.

    x_scale, h_scale (e4m3 only): tensor scales of the token rows and of the SwiGLU rows.  One that is None is measured
    from each batch, over the rows that have an expert, by about ten small launches; the SwiGLU rows' from the bound
    |silu(gate) * up| <= max |gate| * max |up|.  A row then depends on its batch, though only in blocks below 1e-4 of the
    batch's largest value."""

    def __init__(self, gate_up, down, cfg: moe.moe_route_config, max_tokens: int, router_bias=None,
                 fmt: int = moe.MOE_MX_E4M3, x_scale: float | None = None, h_scale: float | None = None):
        E, two_inter, hidden = gate_up.shape
        if down.shape != (E, hidden, two_inter // 2) or cfg.n_experts != E:
            raise ValueError(f"gate_up {tuple(gate_up.shape)}, down {tuple(down.shape)} and {cfg.n_experts} experts do "
                             "not go together")
        self.cfg, self.fmt, self.max_tokens, self.bias = cfg, fmt, max_tokens, router_bias
        self.E, self.hidden, self.inter = E, hidden, two_inter // 2
        for t in (x_scale, h_scale):
            if t is not None and (fmt != moe.MOE_MX_E4M3 or not 1e-30 <= t <= 1e30):
                raise ValueError("x_scale and h_scale are numbers from 1e-30 to 1e30 and go with MOE_MX_E4M3")
        self.gate_up, self.alpha_up = quantise_weights(gate_up, fmt)
        self.down, self.alpha_down = quantise_weights(down, fmt)
        self.x_scale, self.h_scale = (None if t is None else torch.full((E,), t, device="cuda")
                                      for t in (x_scale, h_scale))
        # the products' factors, where the scales are known
        self.product_up, self.product_down = (
            a if a is None or t is None else a * t
            for a, t in ((self.alpha_up, self.x_scale), (self.alpha_down, self.h_scale)))
        pairs, k = max_tokens * cfg.top_k, cfg.top_k

        def i32(*shape):
            return torch.empty(shape, dtype=torch.int32, device="cuda")
        self.idx, self.w = i32(max_tokens, k), torch.empty((max_tokens, k), device="cuda")
        self.offsets, self.row_of_pair = i32(E + 1), i32(max_tokens, k)
        self.token_of_row, self.group_of_row = i32(pairs), i32(pairs)
        # a smaller batch needs no more CTAs than the largest one
        self.workspace = torch.empty(max(1, moe.moe_dispatch_workspace(max_tokens, k, E)), dtype=torch.uint8, device="cuda")
        self.x = moe.make_mx(fmt, pairs, hidden, groups=E, ragged=True)
        self.h = moe.make_mx(fmt, pairs, self.inter, groups=E, ragged=True)
        self.up = torch.empty((pairs, two_inter), dtype=torch.bfloat16, device="cuda")
        self.out = torch.empty((pairs, hidden), dtype=torch.bfloat16, device="cuda")

    def forward(self, x, logits, y):
        """x [T, hidden] and logits [T, E] (fp32 or bf16) -> y [T, hidden] (fp32 or bf16), on the current stream."""
        T, k, st = x.shape[0], self.cfg.top_k, torch.cuda.current_stream()
        n = T * k
        if tuple(x.shape) != (T, self.hidden) or tuple(logits.shape) != (T, self.E) or tuple(y.shape) != (T, self.hidden):
            raise ValueError(f"x {tuple(x.shape)}, logits {tuple(logits.shape)} and y {tuple(y.shape)} do not go together "
                             f"in a layer of {self.E} experts and width {self.hidden}")
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens, room for {self.max_tokens}")
        idx, w, rop = self.idx[:T], self.w[:T], self.row_of_pair[:T]
        tor, gor = self.token_of_row[:n], self.group_of_row[:n]
        moe.moe_route(self.cfg, logits, self.bias, idx, w, st)
        moe.moe_dispatch(idx, self.E, self.offsets, rop, tor, gor, self.workspace, st)
        mx, mh = self._batch(self.x, n), self._batch(self.h, n)
        tx, th, alpha_up, alpha_down = self.x_scale, self.h_scale, self.product_up, self.product_down
        if tx is None and alpha_up is not None and n:
            tx = power_of_two_scale(largest_of(x, idx[:, :1] >= 0)).expand(self.E).contiguous()
            alpha_up = alpha_up * tx
        moe.moe_mx_quantise(mx, x, src_row=tor, group_of_row=gor, offsets=self.offsets, tensor_scale=tx, stream=st)
        moe.moe_mx_product(mx, self.gate_up, self.up[:n], offsets=self.offsets, alpha=alpha_up, stream=st)
        if th is None and alpha_down is not None and n:
            th = power_of_two_scale(largest_of(self.up[:n], gor[:, None] >= 0, 2).prod(0, keepdim=True))
            th = th.expand(self.E).contiguous()
            alpha_down = alpha_down * th
        moe.moe_mx_quantise(mh, self.up[:n], act=moe.MOE_ACT_SWIGLU, group_of_row=gor, offsets=self.offsets,
                            tensor_scale=th, stream=st)
        moe.moe_mx_product(mh, self.down, self.out[:n], offsets=self.offsets, alpha=alpha_down, stream=st)
        moe.moe_combine(self.out[:n], rop, w, y, st)
        return y

    @staticmethod
    def _batch(m: moe.moe_mx, rows: int) -> moe.moe_mx:
        """The same data, for a batch of fewer rows."""
        b = moe.moe_mx(m.data_dev, rows, m.cols, m.groups, m.format, m.ragged)
        b.device = m.device
        return b


def time_of(call, iters: int = 50) -> float:
    """us of one call, in a CUDA graph."""
    for _ in range(3):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(iters):
        graph.replay()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) * 1000 / iters


class DecoderLayer:
    """x + mixer(rms norm of x), and on that the same with the experts, whose logits are the normed rows times router
    [E, hidden] bf16."""

    def __init__(self, mixer, experts: MxLayer, router):
        self.mixer, self.experts, self.router = mixer, experts, router
        self.mixed = torch.zeros((mixer.max_tokens, mixer.hidden), dtype=torch.bfloat16, device="cuda")
        self.expert_out = torch.zeros_like(self.mixed)

    def forward(self, x, seqs: moe.moe_seqs):
        """x [T, hidden] bf16 -> a new tensor like it, on the current stream."""
        T, width = x.shape
        x = x + self.mixer.forward(torch.rms_norm(x, (width,), eps=1e-6), seqs, self.mixed[:T])
        normed = torch.rms_norm(x, (width,), eps=1e-6)
        return x + self.experts.forward(normed, normed @ self.router.T, self.expert_out[:T])


def main() -> None:
    from .delta_layer import DeltaMixer

    E, k, hidden, inter = 512, 10, 2048, 512
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, sigma=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * sigma).to(torch.bfloat16)
    gate_up, down = normal(E, 2 * inter, hidden, sigma=0.02), normal(E, hidden, inter, sigma=0.02)
    given = {"x_scale": tensor_scale(8.0), "h_scale": tensor_scale(32.0)}  # room over what these inputs reach
    for T, scales in ((T, s) for s in (given, {}) for T in (1, 8, 64, 4096)):
        layer = MxLayer(gate_up, down, moe.make_route_config(E, k), max_tokens=T, **scales)
        x, logits = normal(T, hidden), normal(T, E).float()
        y = torch.empty((T, hidden), device="cuda")
        us = time_of(lambda: layer.forward(x, logits, y))
        how = "given" if scales else "measured from the batch"
        print(f"{T} tokens, activation scales {how}: {us:.1f} us a layer")

    Hk, Hv, d = 16, 32, 128
    C, inner = (2 * Hk + Hv) * d, Hv * d
    weights = (normal(C + inner, hidden, sigma=0.02), normal(2 * Hv, hidden, sigma=0.02), normal(C, 4, sigma=0.5),
               torch.zeros(Hv, device="cuda"), torch.zeros(Hv, device="cuda"), torch.ones(d, device="cuda"),
               normal(hidden, inner, sigma=0.02))
    router = normal(E, hidden, sigma=0.02)
    for T, n in ((1, 1), (8, 8), (64, 64), (4096, 1)):
        mixer = DeltaMixer(*weights, (Hk, Hv, d, d), n, T, n)
        layer = DecoderLayer(mixer, MxLayer(gate_up, down, moe.make_route_config(E, k), max_tokens=T, **given), router)
        offsets = None if n == T else torch.tensor([0, T], dtype=torch.int32, device="cuda")
        x, y, seqs = normal(T, hidden), torch.empty((T, hidden), dtype=torch.bfloat16, device="cuda"), moe.make_seqs(n, offsets)
        print(f"{T} tokens of {n} sequences: mixer {time_of(lambda: mixer.forward(x, seqs, y)):.1f} us, decoder layer "
              f"{time_of(lambda: layer.forward(x, seqs)):.1f} us")


if __name__ == "__main__":
    main()
