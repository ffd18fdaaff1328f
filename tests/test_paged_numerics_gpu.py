"""GPU tests of the paged decode's arithmetic where its kernels differ: how
probabilities enter the product with V, infinite values, far scores.  Every
case runs on each kernel of its type (PATHS names shapes that reach them)."""
import math

import numpy as np
import pytest

from sparse_sliding_window_b200 import lf_attn as L
from tests import paged_ref as R
from tests.test_paged_gpu import Cache, _reference

pytestmark = pytest.mark.gpu

# B, H, Hkv, prefix, length of the own rows
PATHS = {
    "cluster": (2, 4, 2, 0, 220),
    "cluster, wide group": (2, 40, 2, 0, 220),
    "runs": (40, 4, 2, 0, 220),
    "runs, wide group": (80, 20, 1, 0, 220),
    "direct prefix": (2, 2, 1, 200, 20),
    "prefix, few rows": (20, 2, 2, 220, 7),
    "prefix, 32 rows": (26, 26, 26, 220, 7),
    "prefix, 40 rows": (20, 4, 2, 220, 7),
    "prefix, many rows": (40, 40, 40, 220, 3),
    "prefix, many rows in two blocks": (70, 40, 20, 220, 3),
}


def _fill(c, rows_of, channel, values, which):
    """values[i] into a channel (or all: slice) of K or V at the i-th row of every sequence and of the prefix."""
    import torch
    pool = c.k if which == "k" else c.v
    val = torch.as_tensor(np.asarray(values, np.float32), device="cuda").to(pool.dtype)
    tables = [(c.table[b], int(n)) for b, n in enumerate(c.lengths)] + [(c.prefix_table, c.prefix)]
    for table, n in tables:
        if n == 0:
            continue
        at = torch.as_tensor(table[np.arange(n) // c.page].astype(np.int64), device="cuda")
        slot = torch.arange(n, device="cuda") % c.page
        x = val[rows_of(n)]
        if isinstance(channel, int):
            pool[at, :, slot, channel] = x[:, None].expand(n, c.Hkv)
        else:
            pool[at, :, slot] = x[:, None, None].expand(n, c.Hkv, 64)


def _decode(c, q, H, window=-1, scale=0.0):
    import torch
    o = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    p = c.params(H, window, None, scale)
    ws = L.paged_workspace(p)
    L.lf_paged_decode(p, q, c.k, c.v, c.t_table, c.t_lengths, o, lse, ws, prefix_table=c.t_prefix)
    L.lf_attn_status(ws)
    return o, lse


def _one_channel_query(B, H, dtype):
    import torch
    q = torch.zeros(B, H, 64, dtype=R.torch_dtype(dtype), device="cuda")
    q[..., 0] = 1
    return q


def _worst_probability(dtype):
    """A key x (score -x/8 against a query of 1) whose exp(-x/8) lies as far
    between two 16-bit numbers as any of a grid, and that probability."""
    import torch
    best = (0.0, None, None)
    for i in range(32, 64):
        x = i / 16
        p = math.exp(-x / 8)
        off = abs(float(torch.tensor(p, dtype=torch.float64).to(R.torch_dtype(dtype)).double()) - p) / p
        best = max(best, (off, x, p))
    return best


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("path", PATHS)
def test_probabilities_are_not_rounded_to_16_bits(path, dtype):
    """Two groups of keys, probability 1 and value +1, probability p and value
    -1, whose sums nearly cancel: a rounding of p to 16 bits would stand in the
    output alone, far above the output's own rounding.  Two 16-bit numbers hold
    p to within the square of a step (twice half a step each)."""
    B, H, Hkv, prefix, n = PATHS[path]
    off, x, p = _worst_probability(dtype)
    c = Cache(901, dtype, B, Hkv, 16, [n] * B, prefix)
    plus = round(32 * p / (1 + p))                       # of every 32 keys, spread over them
    first = [(i * plus) % 32 < plus for i in range(32)]
    assert sum(first) == plus
    _fill(c, lambda m: np.arange(m) % 32, 0, [0.0 if f else -x for f in first], "k")
    _fill(c, lambda m: np.arange(m) % 32, None, [1.0 if f else -1.0 for f in first], "v")
    q = _one_channel_query(B, H, dtype)
    o, lse = _decode(c, q, H)
    half = R.half_step(dtype)
    ref, rl, to, tl = _reference(c, q, H, -1, None, 0.125, (2 * half) ** 2)
    # what is to be seen: p rounded to 16 bits moves the output by about half of that rounding
    assert 0.45 * off > 1.2 * (to.max() + half * np.abs(ref).max())
    R.check("o", R.f64(o), ref, to + half * (np.abs(ref) + to))
    R.check("lse", R.f64(lse), rl, tl)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("path", PATHS)
def test_infinite_values_of_attended_keys(path, dtype):
    """An infinity among the attended values is the output's infinity, whatever
    the key's probability is (1 for a sequence of one key); infinities of both
    signs are NaN; the other channels are what they are without them."""
    import torch
    B, H, Hkv, prefix, n = PATHS[path]
    c = Cache(902, dtype, B, Hkv, 16, [1] + [n] * (B - 1), prefix)
    q = _one_channel_query(B, H, dtype)
    q += _normal_like(c, q) / 4
    tables = [(c.table[b], int(m)) for b, m in enumerate(c.lengths)] + [(c.prefix_table, prefix)]
    where = [(3, 0, math.inf), (4, 1, -math.inf), (5, 0, math.inf), (5, 1, -math.inf)]
    for table, m in tables:
        for ch, row, x in where:
            if row < m:
                c.v[table[row // 16], :, row % 16, ch] = x
    o, lse = _decode(c, q, H)
    assert (o[..., 3] == math.inf).all()
    two = o[1:] if not prefix else o
    assert (two[..., 4] == -math.inf).all() and torch.isnan(two[..., 5]).all()
    if not prefix:
        assert (o[0, :, 5] == math.inf).all() and torch.isfinite(o[0, :, 4]).all()
    clean = torch.where(torch.isinf(c.v), torch.zeros_like(c.v), c.v)
    o0, lse0 = _decode(_with(c, v=clean), q, H)
    rest = [ch for ch in range(64) if ch not in (3, 4, 5)]
    assert torch.equal(o[..., rest], o0[..., rest]) and torch.equal(lse, lse0)


def _normal_like(c, q):
    import torch
    return torch.from_numpy(c.rng.standard_normal(tuple(q.shape)).astype(np.float32)).to("cuda", q.dtype)


def _with(c, **kw):
    import copy
    d = copy.copy(c)
    d.__dict__.update(kw)
    return d


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("path", PATHS)
def test_many_small_probabilities_add_up(path, dtype):
    """Every 16th key has score 0 and value 0, the others probability 2^-26 of
    it and value 64: the output is what the small ones add up to."""
    B, H, Hkv, prefix, n = PATHS[path]
    c = Cache(903, dtype, B, Hkv, 16, [n] * B, prefix)
    x = 26 * math.log(2) * 8                      # 144.2: rounded by the type, the reference takes it as it is then
    _fill(c, lambda m: np.arange(m) % 16, 0, [0.0] + [-x] * 15, "k")
    _fill(c, lambda m: np.arange(m) % 16, None, [0.0] + [64.0] * 15, "v")
    q = _one_channel_query(B, H, dtype)
    o, lse = _decode(c, q, H)
    half = R.half_step(dtype)
    ref, rl, to, tl = _reference(c, q, H, -1, None, 0.125, (2 * half) ** 2 if dtype != "f32" else 0.0)
    # f16: a probability is held to 2^-31 of the largest one (of which there is one in sixteen keys), the
    # output's own spacing below the smallest normal number is 2^-24
    floor = 16 * 64 * 2.0 ** -31 + 2.0 ** -25 if dtype == "f16" else 0.0
    assert np.abs(ref).min() > 16 * floor
    R.check("o", R.f64(o), ref, to + floor + half * (np.abs(ref) + to))
    R.check("lse", R.f64(lse), rl, tl)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("path", PATHS)
def test_far_scores_stay_finite(path, dtype, sign):
    """Scores of 2^34 (f16) and 2^80: one key, row 1 of every sequence, is above
    all others by more than the scores' roundings and takes the whole
    probability."""
    B, H, Hkv, prefix, n = PATHS[path]
    c = Cache(904, dtype, B, Hkv, 16, [n] * B, prefix)
    top = 2.0 ** 14 if dtype == "f16" else 2.0 ** 40
    # multiples of top that the types hold and whose products need rounding; row 1 of a sequence outweighs the rest
    values = [1.0 + (i % 7) / 8 for i in range(32)]
    values = [top * (a if sign > 0 else a + 1) for a in values]
    for ch in range(64):
        _fill(c, lambda m: np.arange(m) % 32, ch, values, "k")
    win = top * (2.5 if sign > 0 else 0.625)
    for b in range(B):
        c.k[c.table[b, 0], :, 1] = win
    q = _one_channel_query(B, H, dtype)
    q[:] = sign * 1.1 * top
    o, lse = _decode(c, q, H)
    half = R.half_step(dtype)
    v = R.f64(c.v)
    s = float(q[0, 0, 0].double()) * win * 64 * 0.125
    for b in range(B):
        want = np.repeat(v[c.table[b, 0], :, 1], H // Hkv, axis=0)
        R.check("o", R.f64(o[b]), want, 2 * half * np.abs(want))
        # a float32 sum of 64 equal products and two scalings
        R.check("lse", R.f64(lse[b]), np.full(H, s), 70 * 2.0 ** -24 * abs(s))


@pytest.mark.parametrize("rise", [40, 44, 45.5, 60, 200])
@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("shape", [(40, 40, 40, 1500), (64, 64, 32, 1300), (20, 20, 20, 900)])
def test_prefix_scores_that_rise(shape, dtype, rise):
    """Scores that rise every 192 keys by about 8 in base 2 (44.4 in this
    channel), by less and by more, for some queries at half the rate, falling,
    or not at all: what a kernel has added up so far is scaled down, or may
    stay, and every chunk of the prefix has its own reference."""
    import torch
    B, H, Hkv, prefix = shape
    c = Cache(905, dtype, B, Hkv, 32, [3] * B, prefix)
    step = np.arange(prefix) // 192
    for j in range(prefix):
        c.k[int(c.prefix_table[j // 32]), :, j % 32, 0] = float(rise * (step[j] % 4))
    q = _normal_like(c, torch.zeros(B, H, 64)).to(R.torch_dtype(dtype))
    q[..., 0] = torch.from_numpy(c.rng.choice([1.0, 1.0, 0.5, 0.0, -1.0], (B, H))).to("cuda", q.dtype)
    if rise >= 60:
        # from a tile of 64 keys to the third after it, in the first head of a query that follows the rise: the
        # channel's 10.8 or 36 in base 2, more or less the difference of the other channels' maxima (below 10)
        b = int(np.flatnonzero(R.f64(q[:, 0, 0]) == 1)[0])
        top = (R.cache_rows(R.f64(c.k), c.prefix_table, prefix, 0) @ R.f64(q[b, 0]) / 8 * np.log2(np.e))[:768].reshape(12, 64).max(1)
        assert (top[3:] - top[:-3]).max() > 8 and (rise < 200 or (top[3:] - top[:-3]).min() > 8)
    o, lse = _decode(c, q, H)
    half = R.half_step(dtype)
    some = sorted(c.rng.choice(B, 12, replace=False).tolist())
    d = _with(c, lengths=c.lengths[some], table=c.table[some])
    ref, rl, to, tl = _reference(d, q[some], H, -1, None, 0.125, (2 * half) ** 2 if dtype != "f32" else 0.0)
    floor = 64 * 8 * 2.0 ** -31 if dtype == "f16" else 0.0
    R.check("o", R.f64(o[some]), ref, to + floor + half * (np.abs(ref) + to))
    R.check("lse", R.f64(lse[some]), rl, tl)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("B,H,Hkv,prefix", [(3, 4, 2, 100), (20, 4, 4, 300), (40, 4, 2, 300), (30, 40, 2, 200)])
def test_dilated_window_behind_a_prefix(B, H, Hkv, prefix, dtype):
    c = Cache(906, dtype, B, Hkv, 16, [(b * 37) % 150 for b in range(B)], prefix)
    q = _normal_like(c, _one_channel_query(B, H, dtype))
    dil = [1 + 2 * (h % 2) for h in range(Hkv)]
    o, lse = _decode_dilated(c, q, H, 20, dil)
    half = R.half_step(dtype)
    ref, rl, to, tl = _reference(c, q, H, 20, dil, 0.125, (2 * half) ** 2 if dtype != "f32" else 0.0)
    R.check("o", R.f64(o), ref, to + 2.0 ** -25 + half * (np.abs(ref) + to))
    R.check("lse", R.f64(lse), rl, tl)


def _decode_dilated(c, q, H, window, dil):
    import torch
    o, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device="cuda")
    p = c.params(H, window, dil)
    ws = L.paged_workspace(p)
    L.lf_paged_decode(p, q, c.k, c.v, c.t_table, c.t_lengths, o, lse, ws, prefix_table=c.t_prefix)
    L.lf_attn_status(ws)
    return o, lse


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("B,H,Hkv,prefix", [(1100, 2, 1, 150), (1100, 20, 1, 70), (300, 128, 128, 0)])
def test_batches_larger_than_the_run_list(B, H, Hkv, prefix, dtype):
    """More than 1024 sequences, behind a prefix, and more than 32768 (sequence, head) units."""
    c = Cache(907, dtype, B, Hkv, 16, [b % 24 for b in range(B)], prefix)
    q = _normal_like(c, _one_channel_query(B, H, dtype))
    o, lse = _decode(c, q, H)
    half = R.half_step(dtype)
    some = list(range(0, B, max(1, B * H // 2200)))
    d = _with(c, lengths=c.lengths[some], table=c.table[some])
    ref, rl, to, tl = _reference(d, q[some], H, -1, None, 0.125, (2 * half) ** 2 if dtype != "f32" else 0.0)
    R.check("o", R.f64(o[some]), ref, to + 2.0 ** -25 + half * (np.abs(ref) + to))
    R.check("lse", R.f64(lse[some]), rl, tl)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("B,H,Hkv,prefix", [(40, 4, 2, 300), (20, 4, 4, 300), (12, 2, 2, 200), (60, 4, 2, 0)])
def test_captured_steps_follow_what_kernels_write(B, H, Hkv, prefix, dtype):
    """Steps in one graph, each of which changes the lengths, the queries and
    the newest rows by kernels right before the call that reads them, are those
    of calls that wait for one another."""
    import torch
    steps = 6
    c = Cache(908, dtype, B, Hkv, 16, [40 + b % 3 for b in range(B)], prefix)
    p, rope = c.params(H, 30), L.make_rope_params()
    ws = L.paged_workspace(p)
    new = [_normal_like(c, torch.zeros(steps, B, h, 64)).to(c.k.dtype) for h in (H, Hkv, Hkv)]
    q, qo = torch.empty_like(new[0][0]), torch.empty_like(new[0][0])
    outs = torch.zeros(steps, B, H, 64, dtype=c.k.dtype, device="cuda"), torch.zeros(steps, B, H, device="cuda")
    start = c.t_lengths.clone()

    def run(kp, vp, lengths, o, lse, wait):
        lengths.copy_(start - steps)
        for s in range(steps):
            lengths.add_(1)
            q.copy_(new[0][s])
            L.lf_cache_append(p, rope, q, new[1][s], new[2][s], lengths, c.t_table, qo, kp, vp, ws)
            if wait:
                torch.cuda.synchronize()
            L.lf_paged_decode(p, qo, kp, vp, c.t_table, lengths, o[s], lse[s], ws, prefix_table=c.t_prefix)
            if wait:
                torch.cuda.synchronize()

    kp, vp, lengths = c.k.clone(), c.v.clone(), c.t_lengths.clone()
    want = torch.empty_like(outs[0]), torch.empty_like(outs[1])
    run(kp, vp, lengths, *want, True)
    L.lf_attn_status(ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(c.k, c.v, c.t_lengths, *outs, False)
    base = [x.clone() for x in (c.k, c.v)]
    for _ in range(20):
        c.k.copy_(base[0])
        c.v.copy_(base[1])
        outs[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in ((c.k, kp), (c.v, vp)))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("window", [384, 511, 512, 639, 640, 768])
@pytest.mark.parametrize("B,H,Hkv", [(20, 8, 4), (26, 40, 2)])
def test_units_of_a_few_tiles(B, H, Hkv, window, dtype):
    """Windows around the number of tiles up to which a unit stays in one block."""
    c = Cache(909, dtype, B, Hkv, 32, [(700 + 61 * b) % 900 for b in range(B)])
    q = _normal_like(c, _one_channel_query(B, H, dtype))
    o, lse = _decode(c, q, H, window)
    half = R.half_step(dtype)
    ref, rl, to, tl = _reference(c, q, H, window, None, 0.125, (2 * half) ** 2)
    R.check("o", R.f64(o), ref, to + 2.0 ** -25 + half * (np.abs(ref) + to))
    R.check("lse", R.f64(lse), rl, tl)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("path", PATHS)
def test_keys_of_probability_zero_weigh_nothing(path, dtype):
    """Every other key has score -inf and the type's largest value: the output
    is that of the same rows with values of 0 there, to the bit."""
    import torch
    B, H, Hkv, prefix, n = PATHS[path]
    c = Cache(910, dtype, B, Hkv, 16, [n] * B, prefix)
    q = _normal_like(c, _one_channel_query(B, H, dtype))
    q[..., 0] = 1
    dead = [(table[j // 16], j % 16) for table, m in [(c.table[b], n) for b in range(B)] + [(c.prefix_table, prefix)]
            for j in range(1, m, 2)]
    page, slot = (torch.tensor(x, device="cuda") for x in zip(*[(int(p), s) for p, s in dead]))
    c.k[page, :, slot, 0] = -math.inf
    c.v[page, :, slot] = 0
    want, wl = _decode(c, q, H)
    c.v[page, :, slot] = torch.finfo(c.v.dtype).max
    o, lse = _decode(c, q, H)
    assert torch.equal(o, want) and torch.equal(lse, wl) and torch.isfinite(o).all()
