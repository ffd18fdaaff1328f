"""The serving operators around the paged key/value cache, as measurable cases.

Four operators: the rotation of queries and keys by their positions (and its
backward), the append of new tokens to a paged cache with the rotation on the
way, the causal-window decode step over that cache, and the decode step of a
batch whose sequences share a long prefix.  ``run`` computes a case in its
plain form (elementary torch operations in 32 bits, angles in 64), or, where
``own`` is true, by the calls a user makes of the framework.
"""
import math

import numpy as np
import torch

own = False

HD = 64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------- cases --

def _rope(name, dtype, B, Hq, Hk, n, axes=1, rot=64, inter=False, back=False, start=0):
    return {"name": name, "op": "rope", "dtype": dtype, "B": B, "H": Hq, "Hkv": Hk, "n": n, "axes": axes,
            "rot": rot, "interleaved": inter, "back": back, "start": start}


def _append(name, dtype, B, H, Hkv, page, new, length, axes=1, rot=64, inter=False, start=0):
    return {"name": name, "op": "append", "dtype": dtype, "B": B, "H": H, "Hkv": Hkv, "page": page, "new": new,
            "length": length, "axes": axes, "rot": rot, "interleaved": inter, "start": start}


def _decode(name, dtype, B, H, Hkv, page, length, window, dilated=False, prefix=0):
    return {"name": name, "op": "decode", "dtype": dtype, "B": B, "H": H, "Hkv": Hkv, "page": page,
            "length": length, "window": window, "dilated": dilated, "prefix": prefix}


def listed():
    return [
        # one new token of a character model: the smallest call, all latency
        _rope("rope_one_token", "bf16", 1, 8, 8, 1, start=23039),
        # image or video patches (time, height, width), an odd count, a partial rotation, f32
        _rope("rope_patches_f32", "f32", 3, 12, 12, 1369, axes=3, rot=48),
        # gradients of queries and keys of the long-encoder shape
        _rope("rope_bwd_long", "bf16", 2, 16, 16, 16384, back=True),
        # a step of a few sequences of the character model
        _append("append_step", "bf16", 4, 8, 8, 64, 1, 23040),
        # a step of a large batch with grouped key/value heads, far positions
        _append("append_step_batch", "f16", 256, 32, 8, 16, 1, 600, inter=True, start=900000),
        # ragged prompts of the padded batch, lengths 2048 to 4096
        _append("append_prompts", "f16", 8, 12, 12, 32, 4096, 4096),
        # the character model's step: window 512, dilation 2 on two heads
        _decode("decode_window", "bf16", 1, 8, 8, 64, 23040, 512, dilated=True),
        # a batch with the base model's window over ragged lengths
        _decode("decode_window_batch", "f16", 64, 12, 12, 16, 4096, 256),
        # every earlier row, grouped heads, ragged lengths of the long shape
        _decode("decode_full_grouped", "bf16", 24, 16, 4, 32, 16384, -1),
        # a few sequences on a short instruction, f32, odd sizes
        _decode("prefix_small_f32", "f32", 5, 2, 2, 16, 77, 64, prefix=1001),
        # many questions about one base-length document: window over the own rows
        _decode("prefix_document", "bf16", 64, 12, 12, 64, 700, 256, prefix=4096),
        # a large batch with grouped heads on a long shared prefix, all own rows
        _decode("prefix_long_grouped", "bf16", 128, 16, 4, 128, 500, -1, prefix=16384),
    ]


MOST_WORK = 280e6  # bytes, or flops / 50: about the largest listed case
MOST_CACHE = 2e9   # bytes of the whole cache, of which a window reads a part


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges that the listed ones stand for."""
    while True:
        c = _draw(rng)
        w = work(c)
        cache = 0 if c["op"] == "rope" else 2 * c["B"] * c["length"] * c["Hkv"] * HD * BYTES[c["dtype"]]
        if max(w["bytes"], w["flops"] / 50) <= MOST_WORK and cache <= MOST_CACHE:
            return c


def _draw(rng):
    op = rng.choice(["rope", "append", "decode", "prefix"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    Hkv = rng.choice([1, 2, 3, 4, 8, 12, 16])
    H = Hkv * rng.choice([1, 1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    axes, rot = rng.choice([1, 1, 2, 3]), rng.choice([64, 64, 32, 48, 10])
    inter, start = rng.random() < 0.4, rng.choice([0, 0, 7, 4096, 1000003])
    if op == "rope":
        c = _rope("", dtype, _log(rng, 1, 16), H, Hkv, _log(rng, 1, 16384), axes, rot, inter, rng.random() < 0.5, start)
    elif op == "append":
        new = 1 if rng.random() < 0.5 else _log(rng, 2, 4096)
        c = _append("", dtype, _log(rng, 1, 256), H, Hkv, page, new, new + _log(rng, 1, 4000), axes, rot, inter, start)
    elif op == "decode":
        window = rng.choice([-1, 0, 5, 64, 256, 512])
        c = _decode("", dtype, _log(rng, 1, 128), H, Hkv, page, _log(rng, 1, 24000), window,
                    window > 0 and rng.random() < 0.4)
    else:
        window = rng.choice([-1, 64, 256, 512])
        c = _decode("", dtype, _log(rng, 1, 160), H, Hkv, page, _log(rng, 1, 1500), window,
                    window > 0 and rng.random() < 0.2, _log(rng, 50, 16384 if dtype != "f32" else 2048))
    del c["name"]
    return c


def _lengths(c):
    """Ragged lengths between half of the largest and the largest; they go by the case alone."""
    B, most = c["B"], c["length"]
    low = most // 2
    n = np.array([most - (b * 7919) % (most - low + 1) if b else most for b in range(B)])
    return np.maximum(n, 1)


def _new_counts(c):
    if c["new"] == 1:
        return np.ones(c["B"], dtype=np.int64)
    low = c["new"] // 2
    n = np.array([c["new"] - (b * 6151) % (c["new"] - low + 1) if b else c["new"] for b in range(c["B"])])
    return np.minimum(np.maximum(n, 1), _lengths(c))


def _dilation(c):
    return [2 if c["dilated"] and h < max(1, c["Hkv"] // 4) else 1 for h in range(c["Hkv"])]


def work(c):
    e = BYTES[c["dtype"]]
    if c["op"] == "rope":
        rows = c["B"] * c["n"] * (c["H"] + c["Hkv"])
        return {"bytes": 2 * rows * HD * e + 4 * c["axes"] * c["B"] * c["n"], "flops": 3 * rows * c["rot"]}
    if c["op"] == "append":
        T = int(_new_counts(c).sum())
        rows = T * (c["H"] + 2 * c["Hkv"])
        return {"bytes": 2 * rows * HD * e + 4 * c["axes"] * T, "flops": 3 * T * (c["H"] + c["Hkv"]) * c["rot"]}
    keys = 0
    for d in _dilation(c):
        L = _lengths(c)
        keys += int((L if c["window"] < 0 else np.minimum(c["window"], (L - 1) // d) + 1).sum())
    G = c["H"] // c["Hkv"]
    once = keys + c["prefix"] * c["Hkv"]
    pairs = G * keys + c["prefix"] * c["B"] * c["H"]
    return {"bytes": 2 * once * HD * e + 2 * c["B"] * c["H"] * HD * e + 4 * c["B"] * c["H"],
            "flops": 4 * HD * pairs}


# ------------------------------------------------------------------ inputs --

def _pair_axis(c):
    """The axis of each channel pair: sections in the order time, height, width."""
    pairs = c["rot"] // 2
    if c["axes"] == 1:
        return [0] * pairs
    first = max(1, pairs // 4)
    rest = pairs - first
    cut = first + (rest + 1) // 2
    return [0 if i < first else 1 if c["axes"] == 2 or i < cut else 2 for i in range(pairs)]


def _grid(index, axes, start):
    """Positions [axes, ...] of tokens that are numbered row by row, 24 a row and 16 rows a frame."""
    if axes == 1:
        return (index + start).unsqueeze(0).to(torch.int32)
    if axes == 2:
        return torch.stack([index // 24 + start, index % 24]).to(torch.int32)
    return torch.stack([index // 384 + start, index // 24 % 16, index % 24]).to(torch.int32)


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    s = {"case": c}
    B, H, Hkv = c["B"], c["H"], c["Hkv"]
    if c["op"] == "rope":
        s["q"], s["k"] = normal(B, H, c["n"], HD), normal(B, Hkv, c["n"], HD)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        at = torch.arange(c["n"], device="cuda").expand(B, c["n"]) + torch.arange(B, device="cuda")[:, None] * 3
        s["positions"] = _grid(at, c["axes"], c["start"]).contiguous()
        return s
    lengths = _lengths(c)
    page = c["page"]
    columns = -(-int(lengths.max()) // page) + 1
    prefix_pages = -(-c.get("prefix", 0) // page)
    pages = B * columns + prefix_pages + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    s["k_pages"], s["v_pages"] = normal(pages, Hkv, page, HD), normal(pages, Hkv, page, HD)
    s["table"] = order[:B * columns].view(B, columns).contiguous()
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if c["op"] == "append":
        counts = _new_counts(c)
        T = int(counts.sum())
        # the projections' layout: heads first, tokens of all sequences packed
        for name, heads in (("q", H), ("k", Hkv), ("v", Hkv)):
            s[name] = normal(heads, T, HD).transpose(0, 1)
        s["q_out"] = torch.empty(T, H, HD, dtype=dt, device="cuda")
        ends = np.cumsum(counts)
        s["cu"] = torch.tensor(np.concatenate([[0], ends]), dtype=torch.int32, device="cuda") if c["new"] > 1 else None
        row = np.arange(T) - np.repeat(ends - counts, counts) + np.repeat(lengths - counts, counts)
        s["positions"] = _grid(torch.tensor(row, device="cuda"), c["axes"], c["start"]).contiguous()
        return s
    s["q"] = normal(B, H, HD)
    s["prefix_table"] = order[B * columns:B * columns + prefix_pages].contiguous() if prefix_pages else None
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(B, H, dtype=torch.float32, device="cuda")
    return s


# -------------------------------------------------------------- plain form --

def _rotated(x, positions, c, sign):
    """x [..., HD] rotated by positions [axes, ...]; the angles in 64 bits, the rest in 32."""
    rot = c["rot"]
    pairs = rot // 2
    freq = 10000.0 ** (torch.arange(pairs, device=x.device, dtype=torch.float64) * (-2.0 / rot))
    axis = torch.tensor(_pair_axis(c), device=x.device)
    angle = positions.double().movedim(0, -1)[..., axis] * freq
    cos, sin = angle.cos().float(), (sign * angle.sin()).float()
    x = x.float()
    if c["interleaved"]:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
    else:
        u, v = x[..., :pairs], x[..., pairs:rot]
        turned = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _run_rope(s, c):
    sign = -1.0 if c["back"] else 1.0
    at = s["positions"][:, :, None, :]
    return {"q": _rotated(s["q"], at, c, sign).to(s["q"].dtype), "k": _rotated(s["k"], at, c, sign).to(s["k"].dtype)}


def _run_append(s, c):
    T = s["k"].shape[0]
    tokens = torch.arange(T, device="cuda")
    if s["cu"] is None:
        seq, row = tokens, s["lengths"].long() - 1
    else:
        cu = s["cu"].long()
        seq = torch.searchsorted(cu, tokens, right=True) - 1
        row = s["lengths"].long()[seq] - cu[seq + 1] + tokens
    at = s["positions"][:, :, None]
    q = _rotated(s["q"], at, c, 1.0).to(s["q"].dtype)
    k = _rotated(s["k"], at, c, 1.0).to(s["k"].dtype)
    page, slot = s["table"][seq, row // c["page"]].long(), row % c["page"]
    s["k_pages"][page, :, slot] = k
    s["v_pages"][page, :, slot] = s["v"]
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _run_decode(s, c):
    B, H, Hkv, page = c["B"], c["H"], c["Hkv"], c["page"]
    q = s["q"].float().view(B, Hkv, H // Hkv, HD) * (1.0 / math.sqrt(HD))
    last = s["lengths"].long()[:, None, None] - 1
    most = c["length"]
    if c["window"] < 0:
        row = torch.arange(most, device="cuda").expand(B, Hkv, most)
        valid = row <= last
    else:
        d = torch.tensor(_dilation(c), device="cuda")[None, :, None]
        row = last - torch.arange(min(c["window"] + 1, most), device="cuda") * d
        valid = row >= 0
    row = row.clamp(min=0)
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    at = s["table"].long()[torch.arange(B, device="cuda")[:, None, None], row // page]
    k, v = s["k_pages"][at, head, row % page].float(), s["v_pages"][at, head, row % page].float()
    scores = (q @ k.transpose(-1, -2)).masked_fill(~valid[:, :, None], -math.inf)
    if c["prefix"]:
        pk, pv = (s[n][s["prefix_table"].long()].float().transpose(0, 1).reshape(Hkv, -1, HD)[:, :c["prefix"]]
                  for n in ("k_pages", "v_pages"))
        scores = torch.cat([q.transpose(0, 1).reshape(Hkv, -1, HD).matmul(pk.transpose(-1, -2))
                            .view(Hkv, B, H // Hkv, -1).transpose(0, 1), scores], -1)
    top = scores.amax(-1, keepdim=True)
    p = (scores - top).exp()
    total = p.sum(-1, keepdim=True)
    p = p / total
    o = p[..., c["prefix"]:] @ v
    if c["prefix"]:
        o = o + (p[..., :c["prefix"]].transpose(0, 1).reshape(Hkv, -1, c["prefix"]) @ pv) \
            .view(Hkv, B, H // Hkv, HD).transpose(0, 1)
    lse = (top + total.log()).view(B, H)
    return {"o": o.reshape(B, H, HD).to(s["q"].dtype), "lse": lse}


# --------------------------------------------------------- the framework's --

def _own(s, c):
    from sparse_sliding_window_b200 import lf_attn as L
    plan = s.get("plan")
    if plan is None:  # what a program keeps: parameters and, for the cache, a workspace
        code = {"f32": L.LF_F32, "bf16": L.LF_BF16, "f16": L.LF_F16}[c["dtype"]]
        plan = s["plan"] = {}
        if c["op"] != "decode":
            plan["rope"] = L.make_rope_params(c["rot"], c["interleaved"], c["axes"], _pair_axis(c))
        if c["op"] != "rope":
            decode = c["op"] == "decode"
            plan["p"] = L.make_paged_params(
                c["B"], c["H"], c["Hkv"], c["page"], s["k_pages"].shape[0], s["table"].shape[1],
                window=c["window"] if decode else -1, dilation=_dilation(c) if decode else None, dtype=code,
                prefix_len=c["prefix"] if decode else 0)
            plan["ws"] = L.paged_workspace(plan["p"])
    if c["op"] == "rope":
        call = L.lf_rope_bwd if c["back"] else L.lf_rope_fwd
        call(plan["rope"], [s["q"], s["k"]], [s["q_out"], s["k_out"]], s["positions"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "append":
        L.lf_cache_append(plan["p"], plan["rope"], s["q"], s["k"], s["v"], s["lengths"], s["table"], s["q_out"],
                          s["k_pages"], s["v_pages"], plan["ws"], cu_new=s["cu"], positions=s["positions"])
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    L.lf_paged_decode(plan["p"], s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["o"], s["lse"],
                      plan["ws"], prefix_table=s["prefix_table"])
    return {"o": s["o"], "lse": s["lse"]}


def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    return {"rope": _run_rope, "append": _run_append, "decode": _run_decode}[c["op"]](s, c)


# ------------------------------------------------------------------- exact --

def _turn(x, pos, c, sign):
    """One tensor rotated pair by pair from the definition: x float64 [..., HD], pos a list of [...] per axis."""
    y = x.clone()
    pairs = c["rot"] // 2
    for p, a in enumerate(_pair_axis(c)):
        u, v = (2 * p, 2 * p + 1) if c["interleaved"] else (p, p + pairs)
        angle = pos[a].double() * math.pow(10000.0, -2.0 * p / c["rot"])
        co, si = torch.cos(angle), sign * torch.sin(angle)
        y[..., u] = co * x[..., u] - si * x[..., v]
        y[..., v] = si * x[..., u] + co * x[..., v]
    return y


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        sign = -1.0 if c["back"] else 1.0
        return {n: torch.stack([_turn(s[n][b].double(), [a[b] for a in s["positions"]], c, sign)
                                for b in range(c["B"])]) for n in ("q", "k")}
    page = c["page"]
    table, lengths = s["table"].tolist(), s["lengths"].tolist()
    if c["op"] == "append":
        pos = [a[:, None] for a in s["positions"]]
        k = _turn(s["k"].double(), pos, c, 1.0)
        out = {"q": _turn(s["q"].double(), pos, c, 1.0), "k_pages": s["k_pages"].double(), "v_pages": s["v_pages"].double()}
        t = 0
        for b, count in enumerate(_new_counts(c).tolist()):
            rows = torch.arange(lengths[b] - count, lengths[b])
            where = torch.tensor(table[b])[rows // page].cuda(), (rows % page).cuda()
            out["k_pages"][where[0], :, where[1]] = k[t:t + count]
            out["v_pages"][where[0], :, where[1]] = s["v"][t:t + count].double()
            t += count
        return out
    B, H, Hkv = c["B"], c["H"], c["Hkv"]
    o = torch.zeros(B, H, HD, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, H, dtype=torch.float64, device="cuda")
    pages = s["prefix_table"].tolist() if c["prefix"] else []
    shared = [torch.cat([s[n][i] for i in pages], 1)[:, :c["prefix"]].double() if pages else
              torch.zeros(Hkv, 0, HD, dtype=torch.float64, device="cuda") for n in ("k_pages", "v_pages")]
    for b in range(B):
        L = lengths[b]
        used = torch.tensor(table[b][:-(-L // page)], device="cuda")
        k, v = (s[n][used].transpose(0, 1).reshape(Hkv, -1, HD)[:, :L] for n in ("k_pages", "v_pages"))
        for h, d in enumerate(_dilation(c)):
            keep = slice(None) if c["window"] < 0 else [j for j in range(L - 1, -1, -d)][:c["window"] + 1]
            kk, vv = torch.cat([shared[0][h], k[h][keep].double()]), torch.cat([shared[1][h], v[h][keep].double()])
            heads = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
            x = s["q"][b, heads].double() @ kk.T / math.sqrt(HD)
            lse[b, heads] = torch.logsumexp(x, -1)
            o[b, heads] = torch.softmax(x, -1) @ vv
    return {"o": o, "lse": lse}
