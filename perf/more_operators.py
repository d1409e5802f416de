"""Cases of the operators between two expert layers of a hybrid decoder: the short causal convolution over a layer's
channels, the norms of heads with the position rotation or a gate, and the gated delta rule (a linear attention whose
state is one matrix a head), each over batches of sequences whose states live in slots.

Each case can run in two ways: in a plain form (elementary torch operations in 32 bits) or, with ``own`` set, through the
library's calls.  Both take the same state.  4096 tokens is the library's own prefill size and 64 its largest decode
batch; heads, widths and dimensions are generic.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16}
CHUNK = 64  # tokens that the plain delta rule takes at a time


def listed():
    return [
        # a decode batch of 64 sequences, three of them padding: q, k and v of 16 and 32 heads of 128
        {"name": "conv decode 64x8192", "op": "conv", "tokens": 64, "sequences": 64, "padded": 3, "channels": 8192,
         "width": 4, "bias": False, "act": "silu", "type": "bfloat16"},
        # a prompt of 4096 tokens, same channels
        {"name": "conv prefill 4096x8192", "op": "conv", "tokens": 4096, "sequences": 1, "padded": 0, "channels": 8192,
         "width": 4, "bias": False, "act": "silu", "type": "bfloat16"},
        # prompts of many lengths together, in 32 bits, three taps with a bias and no activation
        {"name": "conv ragged 5003x1283 f32", "op": "conv", "tokens": 5003, "sequences": 24, "padded": 1,
         "channels": 1283, "width": 3, "bias": True, "act": "none", "type": "float32"},
        # one decoded token: 16 heads of queries and of keys to unit length
        {"name": "norm 1x16+16x128", "op": "norm", "tokens": 1, "heads": 16, "heads2": 16, "dim": 128, "norm": "l2",
         "weight": False, "gate": False, "rot": 0, "pairs": "halves", "far": 0, "type": "bfloat16"},
        # a prompt's queries and keys: weighted norm, a quarter of each head rotated
        {"name": "norm rotate 4096x16+2x256", "op": "norm", "tokens": 4096, "heads": 16, "heads2": 2, "dim": 256,
         "norm": "rms", "weight": True, "gate": False, "rot": 64, "pairs": "halves", "far": 0, "type": "bfloat16"},
        # a prompt's outputs of the delta rule: weighted norm and gate
        {"name": "norm gate 4096x32x128", "op": "norm", "tokens": 4096, "heads": 32, "heads2": 0, "dim": 128,
         "norm": "rms", "weight": True, "gate": True, "rot": 0, "pairs": "halves", "far": 0, "type": "bfloat16"},
        # a small batch a million tokens into its texts, heads of an odd size, in 32 bits, neighbours paired
        {"name": "norm rotate 77x20+5x80 far", "op": "norm", "tokens": 77, "heads": 20, "heads2": 5, "dim": 80,
         "norm": "rms", "weight": True, "gate": False, "rot": 80, "pairs": "adjacent", "far": 1 << 20,
         "type": "float32"},
        # one decoded token: latency
        {"name": "delta 1 token", "op": "delta", "tokens": 1, "sequences": 1, "padded": 0, "k_heads": 16, "v_heads": 32,
         "k_dim": 128, "v_dim": 128},
        # a decode batch of 64 sequences, three of them padding: the states' bytes
        {"name": "delta decode 64", "op": "delta", "tokens": 64, "sequences": 64, "padded": 3, "k_heads": 16,
         "v_heads": 32, "k_dim": 128, "v_dim": 128},
        # four drafted tokens for each of 16 sequences
        {"name": "delta 16 runs of 4", "op": "delta", "tokens": 64, "sequences": 16, "padded": 0, "k_heads": 16,
         "v_heads": 32, "k_dim": 128, "v_dim": 128},
        # a prompt of 4096 tokens
        {"name": "delta prefill 4096", "op": "delta", "tokens": 4096, "sequences": 1, "padded": 0, "k_heads": 16,
         "v_heads": 32, "k_dim": 128, "v_dim": 128},
        # prompts of many lengths together, smaller heads
        {"name": "delta ragged 9001", "op": "delta", "tokens": 9001, "sequences": 24, "padded": 1, "k_heads": 8,
         "v_heads": 16, "k_dim": 64, "v_dim": 96},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of its range; the large ones are odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v if v <= 64 or v % 2 or v == hi else v - 1


def draw(rng):
    op = rng.choice(["conv", "norm", "delta", "delta"])
    if op == "norm":
        dim = 8 * rng.randint(4, 32)
        rot = rng.choice([0, dim // 4 // 2 * 2, dim])
        heads = rng.choice([1, 2, 4, 8, 16, 32, rng.randint(3, 24)])
        return {"op": op, "tokens": min(_log(rng, 1, 4096), (1 << 24) // (heads * dim)), "heads": heads,
                "heads2": rng.choice([0, 1, heads, max(1, heads // 8)]), "dim": dim,
                "norm": rng.choice(["rms", "l2"]), "weight": rng.random() < 0.7, "gate": rng.random() < 0.3, "rot": rot,
                "pairs": rng.choice(["halves", "adjacent"]), "far": rng.choice([0, 0, _log(rng, 1 << 12, 1 << 21)]),
                "type": rng.choice(["float32", "bfloat16"])}
    sequences = rng.choice([1, 1, _log(rng, 2, 64)])
    tokens = sequences * rng.choice([1, rng.randint(2, 8), _log(rng, 16, 4096)])
    padded = rng.choice([0, sequences // 8])
    if op == "conv":
        channels = rng.choice([8 * _log(rng, 8, 1024), _log(rng, 64, 8192)])
        return {"op": op, "tokens": min(tokens, max(sequences, (1 << 25) // channels)), "sequences": sequences,
                "padded": padded, "channels": channels, "width": rng.randint(2, 4), "bias": rng.random() < 0.3,
                "act": rng.choice(["silu", "none"]), "type": rng.choice(["float32", "bfloat16"])}
    k_heads = rng.choice([1, 2, 4, 8, 16])
    v_heads = k_heads * rng.choice([1, 2, 2, 4]) if k_heads < 16 else rng.choice([16, 32])
    return {"op": op, "tokens": min(tokens, 4096 * 32 // v_heads, 8191), "sequences": sequences, "padded": padded,
            "k_heads": k_heads, "v_heads": v_heads, "k_dim": rng.choice([64, 128, 8 * rng.randint(4, 16)]),
            "v_dim": rng.choice([64, 128, 8 * rng.randint(4, 16)])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """Tokens of each sequence: all alike where they divide evenly, else shares of many sizes.  The same for every seed,
    so that the work of a case is known."""
    n, T = case["sequences"], case["tokens"]
    if T % n == 0 and T // n <= 8 or n == 1:
        return np.full(n, T // n, np.int64)
    rng = np.random.default_rng(T * 31 + n)
    share = np.exp(1.2 * rng.standard_normal(n))
    lens = np.floor(share / share.sum() * T).astype(np.int64)
    lens[np.argmax(lens)] += T - lens.sum()
    return lens


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    op, T, dt = case["op"], case["tokens"], TYPES.get(case.get("type"), torch.bfloat16)
    st = {"case": case, "op": op}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if op != "norm":
        n = case["sequences"]
        lens = _lengths(case)
        slots = n + 1
        slot = rng.permutation(slots)[:n].astype(np.int32)
        slot[n - case["padded"]:] = -1  # padding of a batch
        carry = (rng.random(n) < 0.75).astype(np.int32) if lens.max() > 1 else np.ones(n, np.int32)
        off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        st |= {"lens": lens.tolist(), "offsets": torch.from_numpy(off).cuda(), "slot": torch.from_numpy(slot).cuda(),
               "carry": torch.from_numpy(carry).cuda(), "most": int(lens.max())}
    if op == "conv":
        C, W = case["channels"], case["width"]
        st |= {"x": normal(T, C).to(dt), "w": 0.5 * normal(C, W).to(dt), "bias": 0.1 * normal(C) if case["bias"] else None,
               "state": normal(slots, W - 1, C).to(dt), "y": torch.zeros((T, C), dtype=dt, device="cuda")}
    elif op == "norm":
        H, H2, D, R = case["heads"], case["heads2"], case["dim"], case["rot"]
        spread = torch.exp(0.5 * normal(D))
        st |= {"x": (normal(T, H, D) * spread).to(dt), "y": torch.empty((T, H, D), dtype=dt, device="cuda"),
               "x2": (normal(T, H2, D) * spread).to(dt) if H2 else None,
               "y2": torch.empty((T, H2, D), dtype=dt, device="cuda") if H2 else None,
               "weight": 0.3 * normal(D) if case["weight"] else None,
               "weight2": 0.3 * normal(D) if case["weight"] and H2 else None,
               "gate": normal(T, H, D).to(dt) if case["gate"] else None, "pos": None, "inv_freq": None}
        if R:
            first = int(rng.integers(0, 1000)) + case["far"]
            st["pos"] = torch.arange(first, first + T, dtype=torch.int32, device="cuda")
            st["inv_freq"] = (1e6 ** (-torch.arange(R // 2, dtype=torch.float64, device="cuda") / (R // 2))).float()
    else:
        Hk, Hv, dk, dv = case["k_heads"], case["v_heads"], case["k_dim"], case["v_dim"]
        # queries, keys and values stand side by side, as the convolution before leaves them
        rows = torch.empty((T, 2 * Hk * dk + Hv * dv), dtype=torch.bfloat16, device="cuda")
        q, k, v = rows.split([Hk * dk, Hk * dk, Hv * dv], 1)
        for t in (q, k):
            a = normal(T, Hk, dk) + normal(Hk, dk)  # the keys of a head have something in common
            t.copy_((a / torch.sqrt((a * a).sum(2, keepdim=True))).flatten(1))
        v.copy_(normal(T, Hv * dv))
        rate = 16 * torch.rand(Hv, generator=gen, device="cuda") + 0.01
        st |= {"q": q.unflatten(1, (Hk, dk)), "k": k.unflatten(1, (Hk, dk)), "v": v.unflatten(1, (Hv, dv)),
               "g": -rate * torch.log1p(torch.exp(normal(T, Hv) - 4)), "beta": 1 / (1 + torch.exp(-normal(T, Hv))),
               "state": 0.3 * normal(slots, Hv, dv, dk), "scale": dk ** -0.5,
               "o": torch.zeros((T, Hv, dv), dtype=torch.bfloat16, device="cuda")}
    if own:  # descriptors only: the inputs are the same either way
        _plan(st, case)
    return st


def _plan(st, case):
    """What a program that calls the library keeps beside its tensors: descriptors and a workspace."""
    import int4_expert_streaming_gb300 as moe

    st["moe"] = moe
    if case["op"] == "norm":
        st["cfg"] = moe.make_head_norm_config(
            norm=moe.MOE_NORM_RMS if case["norm"] == "rms" else moe.MOE_NORM_L2, eps=1e-6, weight_offset=1.0,
            rot_dim=case["rot"], pairs=moe.MOE_ROT_HALVES if case["pairs"] == "halves" else moe.MOE_ROT_ADJACENT)
        return
    st["seqs"] = moe.make_seqs(case["sequences"], offsets=st["offsets"] if st["most"] > 1 else None, slot=st["slot"],
                               carry=st["carry"], max_len=st["most"])
    if case["op"] == "conv":
        st["act"] = moe.MOE_ACT_SILU if case["act"] == "silu" else moe.MOE_ACT_NONE
    else:
        need = moe.moe_delta_workspace(case["tokens"], case["sequences"], case["k_heads"], case["v_heads"],
                                       case["k_dim"], case["v_dim"], st["most"])
        st["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    moe, op = s["moe"], s["op"]
    if op == "conv":
        moe.moe_conv(s["x"], s["w"], s["y"], bias=s["bias"], act=s["act"], seqs=s["seqs"], state=s["state"])
        return {"y": s["y"], "state": s["state"]}
    if op == "norm":
        moe.moe_head_norm(s["cfg"], s["x"], s["y"], weight=s["weight"], gate=s["gate"], x2=s["x2"], y2=s["y2"],
                          weight2=s["weight2"], pos=s["pos"], inv_freq=s["inv_freq"])
        return {"y": s["y"], "y2": s["y2"]}
    moe.moe_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["o"], scale=s["scale"], seqs=s["seqs"],
                  workspace=s["workspace"])
    return {"o": s["o"], "state": s["state"]}


def _run_plain(s):
    return {"conv": _plain_conv, "norm": _plain_norm, "delta": _plain_delta}[s["op"]](s)


def _places(s):
    """For each token its sequence and its place there; for each sequence its first token, length and state slot."""
    first, lens = s["offsets"][:-1].long(), (s["offsets"][1:] - s["offsets"][:-1]).long()
    T = s["case"]["tokens"]
    seq = torch.searchsorted(s["offsets"].long(), torch.arange(T, device="cuda"), right=True) - 1
    return seq, torch.arange(T, device="cuda") - first[seq], first, lens, s["slot"].long()


def _plain_conv(s):
    x, W = s["x"].float(), s["case"]["width"]
    seq, place, first, lens, slot = _places(s)
    old = s["state"].float()[slot.clamp(min=0)] * s["carry"].bool()[:, None, None]
    # before every sequence the W - 1 rows of its state
    C, n = x.shape[1], len(slot)
    rows = torch.cat([old.flatten(0, 1), x])
    back = torch.arange(W, device="cuda") - (W - 1)
    at = place[:, None] + back
    at = torch.where(at >= 0, (first[seq][:, None] + at) + n * (W - 1), seq[:, None] * (W - 1) + at + W - 1)
    w = s["w"].float()
    y = (rows[at[:, 0]] * w[:, 0])
    for i in range(1, W):
        y += rows[at[:, i]] * w[:, i]
    if s["bias"] is not None:
        y += s["bias"]
    if s["case"]["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    there = slot >= 0
    s["y"].copy_(torch.where(there[seq][:, None], y, s["y"].float()).to(s["y"].dtype))
    last = lens[:, None] + torch.arange(W - 1, device="cuda") - (W - 1)
    own_rows = torch.arange(n, device="cuda")[:, None] * (W - 1)
    last = torch.where(last >= 0, first[:, None] + last + n * (W - 1), own_rows + last + W - 1)
    new = rows[last].to(s["state"].dtype)
    kept = there & (lens > 0)
    s["state"][slot[kept]] = new[kept]
    return {"y": s["y"], "state": s["state"]}


def _plain_heads(x, weight, gate, s):
    case, D, R = s["case"], s["case"]["dim"], s["case"]["rot"]
    x = x.float()
    total = (x * x).sum(2, keepdim=True)
    x = x / torch.sqrt((total / D if case["norm"] == "rms" else total) + 1e-6)
    if weight is not None:
        x = x * (1 + weight)
    if R:
        angle = s["pos"].double()[:, None] * s["inv_freq"].double()
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        if case["pairs"] == "halves":
            a, b = x[:, :, :R // 2], x[:, :, R // 2:R]
            x = torch.cat([a * cos - b * sin, b * cos + a * sin, x[:, :, R:]], 2)
        else:
            a, b = x[:, :, 0:R:2], x[:, :, 1:R:2]
            x = torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2), x[:, :, R:]], 2)
    if gate is not None:
        gate = gate.float()
        x = x * (gate / (1 + torch.exp(-gate)))
    return x


def _plain_norm(s):
    y = _plain_heads(s["x"], s["weight"], s["gate"], s).to(s["x"].dtype)
    y2 = None if s["x2"] is None else _plain_heads(s["x2"], s["weight2"], None, s).to(s["x2"].dtype)
    return {"y": y, "y2": y2}


def _plain_delta(s):
    """Chunks of tokens in lockstep over the sequences.  Within a chunk the updates u solve (1 + A) u = beta (v - decayed
    K S), A[i, j] = beta_i e^(G_i - G_j) k_i k_j for j < i, by substitution."""
    case = s["case"]
    n, Hk, Hv, dk, dv = case["sequences"], case["k_heads"], case["v_heads"], case["k_dim"], case["v_dim"]
    seq, place, first, lens, slot = _places(s)
    C = min(CHUNK, s["most"])
    chunks = -(-s["most"] // C)

    def spread(x):  # [T, H, ..] -> [chunks, n, H, C, ..], zeros where a sequence has ended
        z = x.new_zeros((n, chunks * C) + x.shape[1:], dtype=torch.float32)
        z[seq, place] = x.float()
        return z.unflatten(1, (chunks, C)).transpose(0, 1).transpose(2, 3).contiguous()

    share = Hv // Hk
    q, k = (spread(s[t].repeat_interleave(share, 1)) for t in ("q", "k"))
    v, g, beta = spread(s["v"]), spread(s["g"]), spread(s["beta"])
    G = g.double().cumsum(3)
    low = torch.ones((C, C), dtype=torch.bool, device="cuda").tril()
    decay = torch.where(low, torch.exp((G[..., :, None] - G[..., None, :]).clamp(max=0)), 0).float()
    A = (beta[..., None] * decay * (k @ k.transpose(3, 4))).tril(-1)
    P = decay * (q @ k.transpose(3, 4))
    inverse = torch.eye(C, device="cuda").expand(A.shape).contiguous()
    for i in range(1, C):
        inverse[..., i, :] -= (A[..., i, None, :i] @ inverse[..., :i, :]).squeeze(-2)
    inverse = inverse * beta[..., None, :]
    grown, left = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    S = s["state"][slot.clamp(min=0)] * s["carry"].bool()[:, None, None, None]  # [n, Hv, dv, dk]
    o = torch.empty_like(v)
    for c in range(chunks):
        u = inverse[c] @ (v[c] - grown[c] * (k[c] @ S.transpose(2, 3)))
        o[c] = s["scale"] * (grown[c] * (q[c] @ S.transpose(2, 3)) + P[c] @ u)
        S = grown[c][..., -1:, :] * S + u.transpose(2, 3) @ (left[c] * k[c])
    there = slot >= 0
    flat = o.transpose(0, 1).transpose(2, 3).reshape(n, chunks * C, Hv, dv)[seq, place]
    s["o"].copy_(torch.where(there[seq][:, None, None], flat, s["o"].float()).to(s["o"].dtype))
    kept = there & (lens > 0)
    s["state"][slot[kept]] = S[kept]
    return {"o": s["o"], "state": s["state"]}


# ---------------------------------------------------------------------------
# work and the results in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op, T = case["op"], case["tokens"]
    size = 2 if case.get("type", "bfloat16") == "bfloat16" else 4
    if op == "norm":
        rows = T * (case["heads"] + case["heads2"])
        gates = T * case["heads"] if case["gate"] else 0
        return {"bytes": (2 * rows + gates) * case["dim"] * size + (4 * T if case["rot"] else 0),
                "flops": 6 * rows * case["dim"]}
    lens = _lengths(case)
    live = lens[:len(lens) - case["padded"]]
    tokens, states = int(live.sum()), int((live > 0).sum())
    if op == "conv":
        C, W = case["channels"], case["width"]
        return {"bytes": (2 * tokens + 2 * states * (W - 1) + W) * C * size, "flops": 2 * W * tokens * C}
    Hk, Hv, dk, dv = case["k_heads"], case["v_heads"], case["k_dim"], case["v_dim"]
    row = 2 * (2 * Hk * dk + 2 * Hv * dv) + 8 * Hv
    return {"bytes": tokens * row + states * Hv * dk * dv * 8, "flops": 7 * tokens * Hv * dk * dv}


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "norm": _exact_norm, "delta": _exact_delta}[case["op"]](s, case)


def _exact_conv(s, case):
    W = case["width"]
    y, state = s["y"].double(), s["state"].double()
    slot, carry, at = s["slot"].tolist(), s["carry"].tolist(), 0
    for n, length in enumerate(s["lens"]):
        if slot[n] >= 0 and length:
            before = state[slot[n]] if carry[n] else torch.zeros_like(state[0])
            rows = torch.cat([before, s["x"][at:at + length].double()])
            r = (rows.unfold(0, W, 1) * s["w"].double()).sum(2)
            if s["bias"] is not None:
                r = r + s["bias"].double()
            y[at:at + length] = r * torch.sigmoid(r) if case["act"] == "silu" else r
            state[slot[n]] = rows[length:]
        at += length
    return {"y": y, "state": state}


def _exact_norm(s, case):
    D, R = case["dim"], case["rot"]

    def heads(x, weight, gate):
        if x is None:
            return None
        x = x.double()
        x = x * torch.rsqrt(x.square().mean(2, keepdim=True) * (1 if case["norm"] == "rms" else D) + 1e-6)
        if weight is not None:
            x = x + x * weight.double()
        if R:
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                               s["pos"].double()[:, None] * s["inv_freq"].double())[:, None]
            part = x[..., :R].unflatten(2, (2, -1)).transpose(2, 3) if case["pairs"] == "halves" \
                else x[..., :R].unflatten(2, (-1, 2))
            z = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
            x = torch.cat([(z.transpose(2, 3) if case["pairs"] == "halves" else z).flatten(2), x[..., R:]], 2)
        return x if gate is None else x * gate.double() * torch.sigmoid(gate.double())

    return {"y": heads(s["x"], s["weight"], s["gate"]), "y2": heads(s["x2"], s["weight2"], None)}


def _exact_delta(s, case):
    """Token by token: S <- e^g S; S <- S + beta (v - S k) k^T; o = scale S q."""
    share = case["v_heads"] // case["k_heads"]
    lens, slot = np.array(s["lens"]), s["slot"].cpu().numpy()
    first = np.concatenate([[0], np.cumsum(lens)])[:-1]
    order = np.argsort(-lens, kind="stable")
    order = order[(slot[order] >= 0) & (lens[order] > 0)]
    o, state = s["o"].double(), s["state"].double()
    if order.size == 0:
        return {"o": o, "state": state}
    where = torch.from_numpy(slot[order].astype(np.int64)).cuda()
    at = torch.from_numpy(first[order].astype(np.int64)).cuda()
    S = state[where] * s["carry"].double()[torch.from_numpy(order).cuda()][:, None, None, None]
    alive = [int((lens[order] > t).sum()) for t in range(int(lens[order].max()))]
    for t, m in enumerate(alive):
        r = at[:m] + t
        q, k = (s[x][r].double().repeat_interleave(share, 1).unsqueeze(3) for x in ("q", "k"))
        v, g, beta = s["v"][r].double().unsqueeze(3), s["g"][r].double(), s["beta"][r].double()
        M = S[:m] * torch.exp(g)[:, :, None, None]
        M += (beta[:, :, None, None] * (v - M @ k)) * k.transpose(2, 3)
        S[:m] = M
        o[r] = s["scale"] * (M @ q).squeeze(3)
    state[where] = S
    return {"o": o, "state": state}
