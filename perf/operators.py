"""Cases of the expert-layer operators in microscaled 4-bit floats: routing with groups and a balance bias, the sort of
the chosen (token, expert) pairs, quantisation, the grouped product and the weighted combine.

Each case can run in two ways: in a plain form (elementary torch operations in 32 bits) or, with ``own`` set, through the
library's calls.  Both take the same state.  Hidden 2048, expert width 512 (gate and up side by side: 1024) and 512
experts / 10 chosen or 256 / 8 are the library's own workload sizes; the others are generic.
"""
import functools
import math

import numpy as np
import torch

own = False

BLOCK = {"e8m0": 32, "e4m3": 16}  # columns that share a scale, by the scale's type
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16}
TILE_ROWS, TILE_COLS = 128, 256


def listed():
    return [
        # the router of one decoded token, 512 experts / 10 chosen: latency
        {"name": "route 1x512 softmax", "op": "route", "tokens": 1, "experts": 512, "top_k": 10, "groups": 1,
         "top_groups": 1, "score": "softmax", "bias": False, "type": "float32", "padded": 0},
        # a prefill's router with sigmoid scores, balance bias, 4 of 8 groups, and a few padding tokens
        {"name": "route 4001x256 groups", "op": "route", "tokens": 4001, "experts": 256, "top_k": 8, "groups": 8,
         "top_groups": 4, "score": "sigmoid", "bias": True, "type": "float32", "padded": 37},
        # a decode batch of 64 tokens sorted by expert
        {"name": "dispatch 64x8", "op": "dispatch", "tokens": 64, "experts": 256, "top_k": 8, "skew": 0.0, "padded": 0},
        # a prefill of 4096 tokens with skewed expert popularity
        {"name": "dispatch 4096x10", "op": "dispatch", "tokens": 4096, "experts": 512, "top_k": 10, "skew": 1.1,
         "padded": 0},
        # token rows of a decode batch gathered in expert order, then read back
        {"name": "quantise 64 rows e8m0", "op": "quantise", "tokens": 8, "experts": 256, "top_k": 8, "cols": 2048,
         "format": "e8m0", "type": "float32", "act": False, "skew": 0.0},
        # the experts' SwiGLU between the two products of a prefill, then read back
        {"name": "swiglu 40960x512 e4m3", "op": "quantise", "tokens": 4096, "experts": 512, "top_k": 10, "cols": 512,
         "format": "e4m3", "type": "bfloat16", "act": True, "skew": 1.1},
        # one token against a dense (shared) expert's gate and up rows: latency and weight bytes
        {"name": "product 1 row", "op": "product", "tokens": 1, "experts": 1, "top_k": 1, "rows": 1024, "cols": 2048,
         "format": "e4m3", "type": "bfloat16", "skew": 0.0},
        # a decode batch of 8 tokens: 64 rows spread over 256 experts, gate and up
        {"name": "product 8 tokens of 256", "op": "product", "tokens": 8, "experts": 256, "top_k": 8, "rows": 1024,
         "cols": 2048, "format": "e8m0", "type": "bfloat16", "skew": 0.0},
        # a prefill of 4096 tokens, skewed popularity, gate and up
        {"name": "product 4096 tokens of 512", "op": "product", "tokens": 4096, "experts": 512, "top_k": 10,
         "rows": 1024, "cols": 2048, "format": "e4m3", "type": "bfloat16", "skew": 1.1},
        # a dense projection of a long prefill: bound by the tensor cores
        {"name": "product dense 7937x8192x8192", "op": "product", "tokens": 7937, "experts": 1, "top_k": 1,
         "rows": 8192, "cols": 8192, "format": "e8m0", "type": "bfloat16", "skew": 0.0},
        # one decoded token's ten expert rows: latency
        {"name": "combine 1x10", "op": "combine", "tokens": 1, "top_k": 10, "cols": 2048, "type": "bfloat16",
         "padded": 0},
        # a prefill's combine: bound by memory
        {"name": "combine 4096x10", "op": "combine", "tokens": 4096, "top_k": 10, "cols": 2048, "type": "bfloat16",
         "padded": 5},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of its range; the large ones are odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v if v <= 2048 or v % 2 or v == hi else v - 1


def _width(rng, lo, hi):
    """A matrix side: a power of two as often as any other number."""
    return rng.choice([_log(rng, lo, hi), 1 << rng.randint(lo.bit_length(), hi.bit_length() - 1)])


def draw(rng):
    op = rng.choice(["route", "dispatch", "quantise", "product", "product", "combine"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        experts = groups * _log(rng, 4, max(5, 1024 // groups))
        top_groups = rng.randint(max(1, (groups + 3) // 4), groups)
        top_k = rng.randint(1, min(16, top_groups * (experts // groups)))
        tokens = min(_log(rng, 1, 8192), max(1, (1 << 22) // experts))
        return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "groups": groups,
                "top_groups": top_groups, "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5,
                "type": rng.choice(["float32", "bfloat16"]), "padded": rng.choice([0, tokens // 9])}
    if op == "dispatch":
        experts = _log(rng, 8, 1024)
        tokens = min(_log(rng, 1, 8192), (1 << 21) // experts)
        return {"op": op, "tokens": tokens, "experts": experts, "top_k": rng.randint(1, min(10, experts)),
                "skew": rng.choice([0.0, 0.6, 1.1]), "padded": rng.choice([0, tokens // 7])}
    if op == "quantise":
        experts = rng.choice([1, _log(rng, 8, 512)])
        return {"op": op, "tokens": _log(rng, 1, 4096), "experts": experts,
                "top_k": 1 if experts == 1 else rng.randint(1, min(10, experts)),
                "cols": _width(rng, 1, 2048 if experts > 1 else 4096),
                "format": rng.choice(["e8m0", "e4m3"]), "type": rng.choice(["float32", "bfloat16"]),
                "act": rng.random() < 0.4, "skew": rng.choice([0.0, 1.1])}
    if op == "product":
        experts = rng.choice([1, 1, _log(rng, 8, 512)])
        top_k = 1 if experts == 1 else rng.randint(1, min(10, experts))
        if experts == 1:
            rows, cols = _width(rng, 32, 8192), _width(rng, 32, 8192)
        else:
            rows = _width(rng, 64, 2048)
            cols = _width(rng, 64, (1 << 21) // rows if rows > 1024 else 2048)
        return {"op": op, "tokens": _log(rng, 1, 8000 if experts == 1 else 4096), "experts": experts, "top_k": top_k,
                "rows": rows, "cols": cols, "format": rng.choice(["e8m0", "e4m3"]),
                "type": rng.choice(["float32", "bfloat16"]), "skew": rng.choice([0.0, 1.1])}
    tokens = _log(rng, 1, 4096)
    return {"op": op, "tokens": tokens, "top_k": rng.randint(1, 10), "cols": _log(rng, 1, 4096),
            "type": rng.choice(["float32", "bfloat16"]), "padded": rng.choice([0, tokens // 9])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=32)
def _choices(tokens, experts, top_k, skew):
    """Experts of each token [tokens, top_k]: the largest of normal scores plus a Zipf popularity.  The same for every
    seed, so that the work of a case is known; a seed renames the experts."""
    rng = np.random.default_rng(tokens * 1031 + experts)
    score = rng.standard_normal((tokens, experts), np.float32) - skew * np.log1p(np.arange(experts, dtype=np.float32))
    return np.argsort(-score, axis=1, kind="stable")[:, :top_k].astype(np.int32)


def _groups(case, rng):
    """A sorted batch: offsets [E + 1], the token and the expert of each row."""
    E = case["experts"]
    names = rng.permutation(E).astype(np.int32)
    e = names[_choices(case["tokens"], E, case["top_k"], case["skew"])].reshape(-1)
    order = np.argsort(e, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(e, minlength=E))]).astype(np.int32)
    return offsets, (order // case["top_k"]).astype(np.int32), e[order]


def _separated(logits, bias, case):
    """Logits in which no selection hangs on a rounding: rows with two scores (of experts or of groups) that are
    nearer than 1e-5 of their size without being equal take the place of none; a clean row stands there instead."""
    if not case["bias"]:
        return logits  # the order is that of the logits themselves
    l = logits.double()
    c = (torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)) + bias.double()
    G, E = case["groups"], case["experts"]
    g = c.unflatten(1, (G, -1)).topk(2 if E > G else 1, 2).values.sum(2)
    kept = torch.zeros_like(g, dtype=torch.bool).scatter_(1, g.topk(case["top_groups"], 1).indices, True)
    kept = torch.where(kept.repeat_interleave(E // G, 1), c, -math.inf)

    def near(v):
        v = v.sort(dim=1).values
        d = v[:, 1:] - v[:, :-1]
        return ((d < 1e-5 * v[:, 1:].abs() + 1e-7) & (d > 0)).any(1)

    bad = near(kept.topk(min(E, case["top_k"] + 1), 1).values) | near(g)
    clean = (~bad).nonzero().flatten()
    if clean.numel() == 0:
        return (torch.arange(logits.shape[1], device=logits.device) * 37 % logits.shape[1]).to(logits.dtype).expand_as(
            logits).contiguous() / 32 - 8
    return logits[torch.where(bad, clean[torch.arange(bad.numel(), device=bad.device) % clean.numel()],
                              torch.arange(bad.numel(), device=bad.device))]


def _e2m1(a):
    """The code of the e2m1 value nearest to a >= 0, ties to the even code, saturating: 0 .5 1 1.5 2 3 4 6."""
    c = (a > 0.25).to(torch.uint8)
    c += a >= 0.75
    c += a > 1.25
    c += a >= 1.75
    c += a > 2.5
    c += a >= 3.5
    c += a > 5.0
    return c


def _quantised(x, fmt, g):
    """Codes (sign in bit 3) and scale bytes of x [..., cols] in 32 bits; cols are padded with zeros to 256.  g: the
    tensor scale, one for each index of the first dimension (e4m3 only)."""
    B, cols = BLOCK[fmt], x.shape[-1]
    x = torch.nn.functional.pad(x, (0, -cols % TILE_COLS)).unflatten(-1, (-1, B))
    amax = x.abs().amax(-1)
    if fmt == "e8m0":
        e = (torch.frexp(amax)[1] - 3).clamp(min=-127)
        e = torch.where(amax > 0, e, -127)
        byte, scale = (e + 127).to(torch.uint8), torch.ldexp(torch.ones_like(amax), e)
    else:
        g = g.view((-1,) + (1,) * (amax.dim() - 1))
        s = (amax / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
        byte, scale = s.view(torch.uint8), s.float() * g
    q = x / scale.unsqueeze(-1)
    codes = torch.where(scale.unsqueeze(-1) > 0, _e2m1(q.abs()), 0)
    codes += (x < 0).to(torch.uint8) * 8
    return codes.flatten(-2), byte


def _tiled(codes, scales, fmt):
    """The library's tiles of codes [P, cols] and scale bytes [P, cols / B], P a multiple of 128 rows, cols of 256."""
    P, C = codes.shape
    atoms = TILE_COLS // BLOCK[fmt] // 4
    b = (codes[:, 0::2] | codes[:, 1::2] << 4).view(P // 128, 128, C // 256, 8, 16)
    r, c = torch.arange(128, device=b.device)[:, None], torch.arange(8, device=b.device)[None]
    b = b.transpose(1, 2)[:, :, r, c ^ (r & 7)]
    s = scales.view(P // 128, 4, 32, C // 256, atoms, 4).permute(0, 3, 4, 2, 1, 5)
    return torch.cat([b.reshape(P // 128, C // 256, -1), s.reshape(P // 128, C // 256, -1)], 2).flatten()


def _untiled(tiles, cols, fmt):
    """Codes [P, cols] and scale bytes [P, blocks] out of tiles; the inverse of _tiled."""
    kt, atoms = -(-cols // 256), TILE_COLS // BLOCK[fmt] // 4
    t = tiles.view(-1, kt, 16384 + 512 * atoms)
    r, c = torch.arange(128, device=t.device)[:, None], torch.arange(8, device=t.device)[None]
    b = t[:, :, :16384].reshape(-1, kt, 128, 8, 16)[:, :, r, c ^ (r & 7)].transpose(1, 2).reshape(-1, kt * 128)
    s = t[:, :, 16384:].reshape(-1, kt, atoms, 32, 4, 4).permute(0, 4, 3, 1, 2, 5).reshape(b.shape[0], -1)
    return torch.stack([b & 15, b >> 4], 2).flatten(1), s


def _tile_rows(offsets, group_of_row):
    """Where each row of a ragged matrix stands in its tiles."""
    r = np.arange(group_of_row.size)
    o = offsets[:-1].astype(np.int64)
    return r - o[group_of_row] + 128 * (o[group_of_row] // 128 + group_of_row)


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    op, T, dt = case["op"], case["tokens"], TYPES.get(case.get("type"))
    st = {"case": case, "op": op}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if op == "route":
        E, k = case["experts"], case["top_k"]
        logits = (1.5 * normal(T, E)).to(dt)
        bias = 0.05 * normal(E) if case["bias"] else None
        logits = _separated(logits, bias, case).contiguous()
        if case["padded"]:
            logits[torch.randperm(T, generator=gen, device="cuda")[:case["padded"]]] = -math.inf
        st |= {"logits": logits, "bias": bias, "idx": torch.empty((T, k), dtype=torch.int32, device="cuda"),
               "w": torch.empty((T, k), device="cuda")}
    elif op == "dispatch":
        E, k = case["experts"], case["top_k"]
        idx = rng.permutation(E).astype(np.int32)[_choices(T, E, k, case["skew"])]
        idx[rng.permutation(T)[:case["padded"]]] = -1
        st["idx"] = _cuda(idx)
        n = T * k
        st |= {name: torch.empty(size, dtype=torch.int32, device="cuda") for name, size in
               (("offsets", E + 1), ("row_of_pair", (T, k)), ("token_of_row", n), ("group_of_row", n))}
    elif op == "quantise":
        offsets, token, group = _groups(case, rng)
        cols, width = case["cols"], case["cols"] * (2 if case["act"] else 1)
        rows = token.size if case["act"] else T  # the activation's input is in expert order already
        x = normal(rows, width) * torch.exp(0.5 * normal(width))
        st |= {"x": x.to(dt), "offsets": _cuda(offsets), "group_of_row": _cuda(group),
               "src_row": None if case["act"] else _cuda(token),
               "values": torch.empty((token.size, cols), dtype=torch.bfloat16, device="cuda")}
        st["data"] = _ragged_room(case, token.size, cols)
    elif op == "product":
        offsets, token, group = _groups(case, rng)
        E, N, K, R, fmt = case["experts"], case["rows"], case["cols"], token.size, case["format"]
        at = torch.from_numpy(_tile_rows(offsets, group)).cuda()
        x = normal(T, K) * torch.exp(0.5 * normal(K))
        xg = x.abs().max().view(1) / (6 * 448)
        codes, scales = _quantised(x, fmt, xg)
        tok = torch.from_numpy(token).cuda().long()
        P = 128 * (R // 128 + E)

        def spread(v):
            to = torch.zeros((P, v.shape[1]), dtype=torch.uint8, device="cuda")
            to[at] = v[tok]
            return to

        st["x_tiles"] = _tiled(spread(codes), spread(scales), fmt)
        w = 0.02 * normal(E, N, K)
        wg = w.abs().amax((1, 2)) / (6 * 448)
        codes, scales = _quantised(torch.nn.functional.pad(w, (0, 0, 0, -N % 128)), fmt, wg)
        del w
        st["w_tiles"] = _tiled(codes.flatten(0, 1), scales.flatten(0, 1), fmt)
        del codes, scales
        st |= {"alpha": (xg * wg) if fmt == "e4m3" else None, "at": at, "most": int(np.diff(offsets).max()),
               "offsets": _cuda(offsets) if E > 1 else None, "group_of_row": _cuda(group), "first": _cuda(offsets),
               "y": torch.empty((R, N), dtype=dt, device="cuda")}
    else:
        k, cols = case["top_k"], case["cols"]
        row = rng.permutation(T * k).astype(np.int32).reshape(T, k)
        row[rng.permutation(T)[:case["padded"]]] = -1
        w = torch.rand((T, k), generator=gen, device="cuda")
        st |= {"rows": normal(T * k, cols).to(dt), "row_of_pair": _cuda(row), "w": w / w.sum(1, keepdim=True),
               "y": torch.empty((T, cols), device="cuda")}
    if own:  # descriptors only: the inputs are the same either way
        _plan(st, case)
    return st


def _ragged_room(case, rows, cols):
    fmt = case["format"]
    tile = 16384 + 512 * (TILE_COLS // BLOCK[fmt] // 4)
    return torch.empty((rows // 128 + case["experts"]) * -(-cols // 256) * tile, dtype=torch.uint8, device="cuda")


def _plan(st, case):
    """What a program that calls the library keeps beside its tensors: descriptors and a workspace."""
    import int4_expert_streaming_gb300 as moe

    st["moe"] = moe
    op = case["op"]
    if "format" in case:
        fmt = moe.MOE_MX_E8M0 if case["format"] == "e8m0" else moe.MOE_MX_E4M3
    if op == "route":
        st["cfg"] = moe.make_route_config(
            case["experts"], case["top_k"], n_groups=case["groups"], top_groups=case["top_groups"],
            group_best=2 if case["bias"] and case["experts"] > case["groups"] else 1,
            score=moe.MOE_SCORE_SIGMOID if case["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX, renorm=True, scale=2.5)
    elif op == "dispatch":
        need = moe.moe_dispatch_workspace(case["tokens"], case["top_k"], case["experts"])
        st["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    elif op == "quantise":
        st["mx"] = moe.make_mx(fmt, st["values"].shape[0], case["cols"], groups=case["experts"], ragged=True,
                               data=st["data"])
        st["act"] = moe.MOE_ACT_SWIGLU if case["act"] else moe.MOE_ACT_NONE
    elif op == "product":
        grouped = case["experts"] > 1
        st["x"] = moe.make_mx(fmt, st["y"].shape[0], case["cols"], groups=case["experts"], ragged=grouped,
                              data=st["x_tiles"])
        st["weights"] = moe.make_mx(fmt, case["rows"], case["cols"], groups=case["experts"], data=st["w_tiles"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    moe, op = s["moe"], s["op"]
    if op == "route":
        moe.moe_route(s["cfg"], s["logits"], s["bias"], s["idx"], s["w"])
        return {"idx": s["idx"], "w": s["w"]}
    if op == "dispatch":
        moe.moe_dispatch(s["idx"], s["case"]["experts"], s["offsets"], s["row_of_pair"], s["token_of_row"],
                         s["group_of_row"], s["workspace"])
        return {n: s[n] for n in ("offsets", "row_of_pair", "token_of_row", "group_of_row")}
    if op == "quantise":
        moe.moe_mx_quantise(s["mx"], s["x"], act=s["act"], src_row=s["src_row"], group_of_row=s["group_of_row"],
                            offsets=s["offsets"])
        moe.moe_mx_dequantise(s["mx"], s["values"], group_of_row=s["group_of_row"], offsets=s["offsets"])
        return {"values": s["values"]}
    if op == "product":
        moe.moe_mx_product(s["x"], s["weights"], s["y"], offsets=s["offsets"], alpha=s["alpha"])
        return {"y": s["y"]}
    moe.moe_combine(s["rows"], s["row_of_pair"], s["w"], s["y"])
    return {"y": s["y"]}


def _run_plain(s):
    case, op = s["case"], s["op"]
    if op == "route":
        return _plain_route(s["logits"].float(), s["bias"], case)
    if op == "dispatch":
        return _plain_dispatch(s["idx"], case)
    if op == "quantise":
        x = s["x"].float()
        if case["act"]:
            gate, up = x[:, :case["cols"]], x[:, case["cols"]:]
            x = gate / (1 + torch.exp(-gate)) * up
        else:
            x = x[s["src_row"]]
        codes, byte = _quantised(x, case["format"], torch.ones(1, device=x.device))
        return {"values": _values(codes, byte, case["format"])[:, :case["cols"]].to(torch.bfloat16)}
    if op == "product":
        N, K, E, fmt = case["rows"], case["cols"], case["experts"], case["format"]
        w = _values(*_untiled(s["w_tiles"], K, fmt), fmt).view(E, -1, -(-K // 256) * 256)[:, :N]
        x = _values(*_untiled(s["x_tiles"], K, fmt), fmt)[s["at"]]
        if E == 1:
            y = x @ w[0].T
        else:
            group = s["group_of_row"].long()
            place = torch.arange(group.numel(), device=group.device) - s["first"].long()[group]
            xe = x.new_zeros((E, s["most"], x.shape[1]))
            xe[group, place] = x
            y = torch.bmm(xe, w.transpose(1, 2))[group, place]
        if s["alpha"] is not None:
            y = y * s["alpha"][s["group_of_row"].long()][:, None]
        return {"y": y.to(s["y"].dtype)}
    row = s["row_of_pair"].long()
    w = torch.where(row >= 0, s["w"], 0.0)
    return {"y": (s["rows"].float()[row.clamp(min=0)] * w[:, :, None]).sum(1)}


def _plain_route(l, bias, case):
    T, E = l.shape
    k, G = case["top_k"], case["groups"]
    there = l > -math.inf
    top = torch.where(there, l, -math.inf).amax(1, keepdim=True)
    if case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        e = torch.where(there, torch.exp(l - top), 0.0)
        s = e / e.sum(1, keepdim=True)
    c = l if bias is None else s + bias
    c = torch.where(there, c, -math.inf)
    if G > 1:
        best = 2 if bias is not None and E > G else 1
        score = c.view(T, G, -1).sort(dim=2, descending=True).values[:, :, :best].sum(2)
        kept = score.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        mask = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        c = torch.where(mask.repeat_interleave(E // G, 1), c, -math.inf)
    v, i = c.sort(dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    w = torch.where(v > -math.inf, s.gather(1, i), 0.0)
    total = w.sum(1, keepdim=True)
    w = torch.where(total > 0, w / total, 0.0) * 2.5
    return {"idx": torch.where(v > -math.inf, i, -1).to(torch.int32), "w": w}


def _plain_dispatch(idx, case):
    T, k = idx.shape
    e = idx.flatten().long()
    n = e.numel()
    key = torch.where(e >= 0, e, case["experts"])
    order = key.sort(dim=0, stable=True).indices
    count = torch.zeros(case["experts"] + 1, dtype=torch.long, device=e.device).index_add_(0, key, torch.ones_like(key))[:-1]
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    place = torch.empty_like(e)
    place[order] = torch.arange(n, device=e.device)
    real = torch.arange(n, device=e.device) < offsets[-1]
    return {"offsets": offsets.int(), "row_of_pair": torch.where(e >= 0, place, -1).view(T, k).int(),
            "token_of_row": torch.where(real, order // k, -1).int(), "group_of_row": torch.where(real, key[order], -1).int()}


def _values(codes, byte, fmt):
    """The numbers that codes [.., cols] with scale bytes [.., cols / B] stand for, in 32 bits."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    scale = torch.ldexp(torch.ones((), device=codes.device), byte.int() - 127) if fmt == "e8m0" \
        else byte.view(torch.float8_e4m3fn).float()
    return (table[codes.int()].unflatten(-1, (-1, BLOCK[fmt])) * scale.unsqueeze(-1)).flatten(-2)


# ---------------------------------------------------------------------------
# work and the results in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op, T = case["op"], case["tokens"]
    size = 2 if case.get("type") == "bfloat16" else 4
    if op == "route":
        E, k = case["experts"], case["top_k"]
        return {"bytes": T * E * size + T * k * 8 + (4 * E if case["bias"] else 0), "flops": 8 * T * E}
    if op == "dispatch":
        n = T * case["top_k"]
        return {"bytes": 16 * n + 4 * (case["experts"] + 1), "flops": n}
    if op == "combine":
        n = T * case["top_k"]
        return {"bytes": n * (case["cols"] * size + 8) + T * case["cols"] * 4, "flops": 2 * n * case["cols"]}
    R, K = T * case["top_k"], case["cols"]
    packed = 0.5 + 1 / BLOCK[case["format"]]
    if op == "quantise":
        # input rows once, codes and scales written and read back, the values in bf16
        read = R * 2 * K * size if case["act"] else T * K * size
        return {"bytes": read + R * K * (2 * packed + 2) + 8 * R, "flops": 8 * R * K}
    active = int(np.unique(_choices(T, case["experts"], case["top_k"], case["skew"])).size)
    N = case["rows"]
    return {"bytes": (R * K + active * N * K) * packed + R * N * size, "flops": 2 * R * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        return None
    if op == "route":
        return _exact_route(s["logits"].double().cpu().numpy(), None if s["bias"] is None else s["bias"].double().cpu().numpy(), case)
    if op == "combine":
        row, w, rows = s["row_of_pair"].long(), s["w"].double(), s["rows"].double()
        y = torch.zeros((row.shape[0], rows.shape[1]), dtype=torch.float64, device="cuda")
        for j in range(row.shape[1]):
            y += torch.where(row[:, j] >= 0, w[:, j], 0.0)[:, None] * rows[row[:, j].clamp(min=0)]
        return {"y": y}
    if op == "quantise":
        x = s["x"].double()
        if case["act"]:
            x = x[:, :case["cols"]] * torch.sigmoid(x[:, :case["cols"]]) * x[:, case["cols"]:]
        else:
            x = x[s["src_row"].long()]
        return {"values": _exact_quantised(x, case["format"])}
    fmt, E, N, K = case["format"], case["experts"], case["rows"], case["cols"]
    x = _exact_values(s["x_tiles"], K, fmt)
    wide = x.shape[1]
    x = x[s["at"]]
    per = s["w_tiles"].numel() // E
    first = s["first"].tolist()
    y = torch.zeros((x.shape[0], N), dtype=torch.float64, device="cuda")
    for e in range(E):
        if first[e + 1] > first[e]:
            w = _exact_values(s["w_tiles"][e * per:(e + 1) * per], K, fmt)[:N, :wide]
            y[first[e]:first[e + 1]] = x[first[e]:first[e + 1]] @ w.T
            if s["alpha"] is not None:
                y[first[e]:first[e + 1]] *= s["alpha"][e].double()
    return {"y": y}


def _exact_route(l, bias, case):
    T, E = l.shape
    k, G = case["top_k"], case["groups"]
    weights = np.zeros((T, k))
    for t in range(T):
        row = l[t]
        if not (row > -np.inf).any():
            continue
        if case["score"] == "sigmoid":
            s = 1 / (1 + np.exp(-row))
        else:
            s = np.exp(row - row.max())
            s /= s.sum()
        c = s if bias is None else s + bias
        best = 2 if bias is not None and E > G else 1
        score = np.sort(c.reshape(G, -1), 1)[:, ::-1][:, :best].sum(1)
        kept = np.argsort(-score, kind="stable")[:case["top_groups"]]
        allowed = np.isin(np.arange(E) // (E // G), kept)
        chosen = np.argsort(-np.where(allowed, c, -np.inf), kind="stable")[:k]
        weights[t] = 2.5 * s[chosen] / s[chosen].sum()
    return {"idx": None, "w": weights}


def _exact_quantised(x, fmt):
    """x [rows, cols] in 64 bits to the nearest values of the format, by the spacing of e2m1 at each magnitude."""
    B, cols = BLOCK[fmt], x.shape[1]
    x = torch.nn.functional.pad(x, (0, -cols % B)).view(x.shape[0], -1, B)
    amax = x.abs().amax(2, keepdim=True)
    if fmt == "e8m0":
        scale = torch.exp2(torch.floor(torch.log2(amax.clamp(min=1e-300))).clamp(min=-125) - 2)
    else:
        a = (amax / 6).clamp(max=448)
        step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
        scale = torch.round(a / step) * step
    q = (x.abs() / scale.clamp(min=1e-300)).clamp(max=6)
    step = torch.exp2(torch.floor(torch.log2(q.clamp(min=1.0))) - 1)
    q = torch.where(scale > 0, (torch.round(q / step) * step).clamp(max=6), 0)
    return (torch.copysign(q * scale, x)).flatten(1)[:, :cols]


def _exact_values(tiles, cols, fmt):
    """Tiles to numbers in 64 bits: sign, exponent and mantissa bits taken apart."""
    codes, byte = _untiled(tiles, cols, fmt)
    c = codes.double()
    sign = 1 - 2 * torch.floor(c / 8)
    m = c % 8
    e = torch.floor(m / 2)
    value = sign * torch.where(e > 0, (1 + (m % 2) / 2) * torch.exp2(e - 1), m / 2)
    b = byte.double()
    if fmt == "e8m0":
        scale = torch.exp2(b - 127)
    else:
        e = torch.floor(b / 8)
        scale = torch.where(e > 0, (1 + (b % 8) / 8) * torch.exp2(e - 7), (b % 8) / 8 * 2.0 ** -6)
    return (value.unflatten(1, (-1, BLOCK[fmt])) * scale[:, :, None]).flatten(1)
