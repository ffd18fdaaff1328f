"""GPU parity of the paged cache append and the paged decode against float64
numpy, and a run of rotation, prompt, append and decode together."""
import math

import numpy as np
import pytest

from sparse_sliding_window_b200 import lf_attn as L
from tests import paged_ref as R

pytestmark = pytest.mark.gpu

CODE = {"f32": L.LF_F32, "bf16": L.LF_BF16, "f16": L.LF_F16}


def _normal(rng, shape, dtype):
    import torch
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to("cuda", R.torch_dtype(dtype))


class Cache:
    """A pool whose rows that no call may read hold NaN and infinities, tables
    whose entries behind the lengths hold no pages."""

    def __init__(self, seed, dtype, B, Hkv, page, lengths, prefix=0, extra=3):
        import torch
        rng = self.rng = np.random.default_rng(seed)
        self.dtype, self.page, self.Hkv = dtype, page, Hkv
        self.lengths = np.asarray(lengths, np.int32)
        cols = max(1, -(-int(max(self.lengths.max(), 1)) // page)) + 1
        npre = -(-prefix // page)
        self.num = B * cols + npre + extra
        order = rng.permutation(self.num).astype(np.int32)
        self.table = order[:B * cols].reshape(B, cols).copy()
        self.prefix_table = order[B * cols:B * cols + npre].copy()
        self.prefix = prefix
        live = np.zeros((self.num, page), bool)
        for b, n in enumerate(self.lengths):
            used = -(-max(int(n), 0) // page)
            for c in range(cols):
                if c < used:
                    live[self.table[b, c], :min(page, n - c * page)] = True
                else:
                    self.table[b, c] = (-1, 2 ** 31 - 1, -2 ** 31)[c % 3]
        for c in range(npre):
            live[self.prefix_table[c], :min(page, prefix - c * page)] = True
        junk = np.where(rng.random((self.num, 1, page, 1)) < 0.5, np.nan, np.inf)
        k, v = (np.where(live[:, None, :, None], rng.standard_normal((self.num, Hkv, page, 64)), junk) for _ in range(2))
        self.live = live
        dt = R.torch_dtype(dtype)
        self.k, self.v = (torch.from_numpy(x.astype(np.float32)).to("cuda", dt) for x in (k, v))
        self.t_table, self.t_lengths = torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lengths).cuda()
        self.t_prefix = torch.from_numpy(self.prefix_table).cuda() if npre else None

    def params(self, H, window=-1, dil=None, scale=0.0):
        return L.make_paged_params(len(self.lengths), H, self.Hkv, self.page, self.num, self.table.shape[1], window, dil,
                                   scale, CODE[self.dtype], self.prefix)


def _reference(c, q, H, window, dil, scale, half_p):
    """o, lse and their allowances in float64."""
    B, G = len(c.lengths), H // c.Hkv
    k, v, qq = R.f64(c.k), R.f64(c.v), R.f64(q)
    o, lse = np.zeros((B, H, 64)), np.zeros((B, H))
    to, tl = np.zeros((B, H, 64)), np.zeros((B, H))
    for h in range(c.Hkv):
        pk, pv = (R.cache_rows(x, c.prefix_table, c.prefix, h) for x in (k, v))
        for b, n in enumerate(c.lengths.tolist()):
            own = R.attended(n, window, dil[h] if dil else 1)
            kk = np.concatenate([pk, R.cache_rows(k, c.table[b], n, h)[own]])
            vv = np.concatenate([pv, R.cache_rows(v, c.table[b], n, h)[own]])
            for g in range(h * G, (h + 1) * G):
                o[b, g], lse[b, g], to[b, g], tl[b, g] = R.softmax_row(qq[b, g], kk, vv, scale, half_p)
    return o, lse, to, tl


def _decode_and_check(c, H, window, dil=None, scale=0.0, q=None):
    import torch
    B = len(c.lengths)
    q = _normal(c.rng, (B, H, 64), c.dtype) if q is None else q
    o = torch.full((B, H, 64), float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full((B, H), float("nan"), device="cuda")
    p = c.params(H, window, dil, scale)
    ws = L.paged_workspace(p)
    L.lf_paged_decode(p, q, c.k, c.v, c.t_table, c.t_lengths, o, lse, ws, prefix_table=c.t_prefix)
    L.lf_attn_status(ws)
    half = R.half_step(c.dtype)
    ref, rl, to, tl = _reference(c, q, H, window, dil, scale or 1 / math.sqrt(64), half if c.dtype != "f32" else 0.0)
    # 2^-25: a 16-bit probability below the smallest normal number is off by that
    floor = 2.0 ** -25 * 8 if c.dtype == "f16" else 1e-30
    R.check("o", R.f64(o), ref, to + floor + (half + 2.0 ** -23) * (np.abs(ref) + to))
    R.check("lse", R.f64(lse), rl, tl)
    return p, ws, q, o, lse


DECODE = [
    # H, Hkv, page, lengths, window, dilation
    (1, 1, 16, [1], -1, None),
    (2, 2, 16, [0, 1, 16, 17], -1, None),
    (3, 3, 32, [300, 5], 64, [1, 2, 3]),
    (2, 1, 64, [257, 0, 64], 0, None),
    (6, 2, 16, [100, 33, 31, 1, 160], -1, None),
    (4, 1, 128, [700, 129], 256, None),
    (8, 1, 16, [513, 48], 511, [2]),
    (16, 2, 1024, [1500, 1025], -1, None),
    (5, 1, 16, [90], 33, None),
    (8, 8, 64, [2600], 512, [2, 2, 1, 1, 1, 1, 1, 1]),
    (12, 12, 16, [40 + 7 * b for b in range(70)], 64, None),
    (2, 2, 16, [50, 50], 2 ** 31 - 1, [2 ** 31 - 1, 7]),
    # many sequences: units cut between blocks, one much longer than the rest
    (4, 2, 16, [(b * 37) % 130 for b in range(60)] + [2000], -1, None),
    (4, 4, 32, [(b * 53) % 400 for b in range(30)], 100, [1, 2, 3, 1]),
    (20, 1, 16, [(b * 11) % 90 for b in range(80)], -1, None),
    (40, 1, 64, [b % 70 for b in range(80)], 30, None),
    (96, 1, 16, [b % 40 for b in range(41)], -1, None),
    (1, 1, 16, [b % 19 for b in range(1100)], -1, None),
    # units on both sides of the choice between the kernels, short and long windows
    (5, 5, 16, [(b * 97) % 600 for b in range(14)], 511, [1, 2, 3, 1, 1]),
    (10, 5, 16, [(b * 97) % 600 for b in range(15)], 511, [1, 2, 3, 1, 1]),
    (5, 5, 16, [(b * 97) % 600 for b in range(14)], 512, [1, 2, 3, 1, 1]),
    (16, 4, 64, [(b * 41) % 300 for b in range(18)], 256, None),
    (37, 37, 32, [700, 513], 40, None),
    (37, 37, 32, [700], -1, None),
    (38, 38, 32, [700], -1, None),
]


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode_matches_float64(case, dtype):
    H, Hkv, page, lengths, window, dil = DECODE[case]
    _decode_and_check(Cache(200 + case, dtype, len(lengths), Hkv, page, lengths), H, window, dil)


PREFIX = [
    # H, Hkv, page, lengths, window, prefix
    (1, 1, 16, [1], -1, 1),
    (1, 1, 16, [0], -1, 63),
    (2, 2, 16, [5, 0, 40], 8, 64),
    (2, 1, 32, [5, 17, 33, 64, 100], -1, 65),
    (4, 2, 64, [10] * 9, 4, 129),
    (3, 1, 16, list(range(11)), -1, 1000),
    (8, 1, 128, [30] * 8, 16, 300),
    (12, 12, 64, [b % 50 for b in range(70)], 16, 515),
    (8, 2, 16, [b % 5 for b in range(40)], -1, 200),
    (16, 2, 1024, [3] * 33, -1, 1100),
    (4, 2, 16, [(b * 37) % 130 for b in range(60)] + [1500], -1, 90),
    (24, 1, 32, [b % 40 for b in range(80)], 10, 200),
    (48, 1, 16, [b % 20 for b in range(80)], -1, 33),
    # few rows, but too many or too long for every sequence to read the prefix itself
    (2, 2, 16, [b % 9 for b in range(20)], -1, 300),
    (3, 3, 32, [b % 40 for b in range(13)], 12, 700),
    (1, 1, 32, [5, 0, 90], -1, 9000),
    (24, 2, 16, [7], 3, 8300),
    # several tiles a block, with a row block that is full, half full, or has a few rows too many
    (40, 40, 64, [b % 3 for b in range(40)], 4, 1500),
    (38, 19, 16, [b % 5 for b in range(64)], 4, 1301),
    (26, 26, 128, [b % 4 for b in range(97)], -1, 1152),
    (12, 12, 64, [300 + b for b in range(64)], 64, 4096),
]


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("case", range(len(PREFIX)))
def test_decode_with_shared_prefix_matches_float64(case, dtype):
    H, Hkv, page, lengths, window, prefix = PREFIX[case]
    _decode_and_check(Cache(300 + case, dtype, len(lengths), Hkv, page, lengths, prefix), H, window)


@pytest.mark.parametrize("dtype", R.DTYPES)
def test_decode_large_scores_and_scale(dtype):
    """Scores far apart: one key carries everything, the rest underflow."""
    c = Cache(31, dtype, 3, 1, 16, [70, 1, 33], prefix=100)
    q = _normal(c.rng, (3, 2, 64), dtype) * 30
    _decode_and_check(c, 2, -1, q=q)
    _decode_and_check(c, 2, -1, scale=2.5)


def test_decode_strided_query_and_no_lse():
    import torch
    c = Cache(41, "bf16", 3, 2, 16, [40, 0, 9], prefix=70)
    p, ws, q, o, lse = _decode_and_check(c, 4, -1)
    wide = torch.zeros(4, 3, 128, dtype=q.dtype, device="cuda")    # heads first, padded rows
    view = wide.transpose(0, 1)[..., 64:]
    view.copy_(q)
    o2 = torch.empty_like(o)
    L.lf_paged_decode(p, view, c.k, c.v, c.t_table, c.t_lengths, o2, None, ws, prefix_table=c.t_prefix)
    assert torch.equal(o, o2)
    same = q[:1, :1].expand(3, 4, 64)                              # a broadcast query
    L.lf_paged_decode(p, same, c.k, c.v, c.t_table, c.t_lengths, o2, None, ws, prefix_table=c.t_prefix)
    L.lf_paged_decode(p, same.contiguous(), c.k, c.v, c.t_table, c.t_lengths, o, None, ws, prefix_table=c.t_prefix)
    assert torch.equal(o, o2)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("prefix", [0, 100])
def test_decode_leaves_out_bad_pages_and_lengths(dtype, prefix):
    import torch
    lengths = [60, 33, 5]
    c = Cache(51, dtype, 3, 2, 16, lengths, prefix)
    H = 4
    p = c.params(H)
    ws = L.paged_workspace(p)
    q = _normal(c.rng, (3, H, 64), dtype)
    o = torch.full((3, H, 64), float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.zeros(3, H, device="cuda")

    def call(table, lens, pre, detail):
        L.lf_paged_decode(p, q, c.k, c.v, table, lens, o, lse, ws, prefix_table=pre)
        with pytest.raises(L.LfError) as e:
            L.lf_attn_status(ws)
        assert e.value.code == L.LF_ERR_DEVICE_INPUT and detail in str(e.value)
        L.lf_attn_status(ws)   # cleared
        return o.clone(), lse.clone()

    # a bad page: its rows are left out, as if the sequence did not have them
    for bad in (-1, c.num, 2 ** 31 - 1):
        table = c.t_table.clone()
        table[0, 1] = bad
        got, gl = call(table, c.t_lengths, c.t_prefix, "sequence 0")
        k, v, qq = R.f64(c.k), R.f64(c.v), R.f64(q)
        for h in range(H):
            rows = [j for j in range(60) if j // 16 != 1]
            kk, vv = (np.concatenate([R.cache_rows(x, c.prefix_table, prefix, h // 2),
                                      R.cache_rows(x, c.table[0], 60, h // 2)[rows]]) for x in (k, v))
            ro, rl, to, tl = R.softmax_row(qq[0, h], kk, vv, 0.125, R.half_step(dtype))
            R.check("o", R.f64(got[0, h]), ro, to + 2.0 ** -22 + R.half_step(dtype) * (np.abs(ro) + to))
            R.check("lse", R.f64(gl[0, h]), rl, tl)
    # a bad length: nothing for that sequence, the others as they were
    L.lf_paged_decode(p, q, c.k, c.v, c.t_table, c.t_lengths, o, lse, ws, prefix_table=c.t_prefix)
    L.lf_attn_status(ws)
    good = o.clone()
    for bad in (-1, c.table.shape[1] * 16 + 1, 2 ** 31 - 1, -2 ** 31):
        lens = c.t_lengths.clone()
        lens[1] = bad
        got, gl = call(c.t_table, lens, c.t_prefix, "sequence 1")
        assert torch.all(got[1] == 0) and torch.all(gl[1] == -math.inf)
        assert torch.equal(got[[0, 2]], good[[0, 2]])
    if prefix:
        pre = c.t_prefix.clone()
        pre[:] = c.num
        got, gl = call(c.t_table, c.t_lengths, pre, "prefix table")
        none = Cache(51, dtype, 3, 2, 16, lengths, prefix)
        none.prefix, none.prefix_table = 0, none.prefix_table[:0]
        # 16-bit probabilities enter the product with V rounded: sum_j p_j (1 + e_j) v_j with |e_j| <= half a
        # step is off by at most half_step * sum_j p_j |v_j|, the last argument's part of the allowance
        ro, rl, to, tl = _reference(none, q, H, -1, None, 0.125, R.half_step(dtype) if dtype != "f32" else 0.0)
        R.check("o", R.f64(got), ro, to + 2.0 ** -22 + R.half_step(dtype) * (np.abs(ro) + to))


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("B,Hkv,prefix", [(2, 1, 0), (2, 1, 200), (40, 2, 200), (80, 1, 0)])
def test_decode_scores_of_minus_infinity_weigh_nothing(dtype, B, Hkv, prefix):
    """Keys whose score is -inf (the newest ones, whole batches and tiles of
    them) have probability 0: the rest is the softmax over the other keys."""
    import torch
    gone, n = 150, 260
    c = Cache(77, dtype, B, Hkv, 16, [n] * B, prefix)
    q = _normal(c.rng, (B, 2 * Hkv, 64), dtype)
    q[..., 0] = q[..., 0].abs() + 0.5
    for b in range(B):
        for j in range(n - gone, n):
            c.k[c.table[b, j // 16], :, j % 16, 0] = -math.inf
    for j in range(0, prefix, 2):
        c.k[c.prefix_table[j // 16], :, j % 16, 0] = -math.inf
    p = c.params(2 * Hkv)
    ws = L.paged_workspace(p)
    o, lse = torch.empty_like(q), torch.empty(B, 2 * Hkv, device="cuda")
    L.lf_paged_decode(p, q, c.k, c.v, c.t_table, c.t_lengths, o, lse, ws, prefix_table=c.t_prefix)
    L.lf_attn_status(ws)
    k, v, qq = R.f64(c.k), R.f64(c.v), R.f64(q)
    for b in (0, B - 1):
        for h in range(2 * Hkv):
            kk, vv = (np.concatenate([R.cache_rows(x, c.prefix_table, prefix, h // 2)[1::2],
                                      R.cache_rows(x, c.table[b], n, h // 2)[:n - gone]]) for x in (k, v))
            ro, rl, to, tl = R.softmax_row(qq[b, h], kk, vv, 0.125, R.half_step(dtype))
            R.check("o", R.f64(o[b, h]), ro, to + 2.0 ** -22 + R.half_step(dtype) * (np.abs(ro) + to))
            R.check("lse", R.f64(lse[b, h]), rl, tl)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("B,Hkv,prefix", [(2, 1, 200), (40, 2, 0), (20, 2, 900), (40, 2, 200), (70, 20, 1500)])
def test_decode_low_scores_beside_scores_of_minus_infinity(dtype, B, Hkv, prefix):
    """Whole tiles of scores of -inf, before and between scores of about -300
    (exp of which is 0 in float32): the softmax over the latter."""
    import torch
    n = 400
    c = Cache(78, dtype, B, Hkv, 16, [n] * B, prefix)
    q = _normal(c.rng, (B, 2 * Hkv, 64), dtype)
    q[..., 0] = q[..., 0].abs() + 0.5
    q[..., 1] = 4
    gone = [j for j in range(n) if (n - 1 - j) // 128 % 2 == 0]
    pgone = [j for j in range(prefix) if j // 64 % 2 == 0]
    c.k[..., 1] = -600
    for b in range(B):
        for j in gone:
            c.k[c.table[b, j // 16], :, j % 16, 0] = -math.inf
    for j in pgone:
        c.k[c.prefix_table[j // 16], :, j % 16, 0] = -math.inf
    p = c.params(2 * Hkv)
    ws = L.paged_workspace(p)
    o, lse = torch.empty_like(q), torch.empty(B, 2 * Hkv, device="cuda")
    L.lf_paged_decode(p, q, c.k, c.v, c.t_table, c.t_lengths, o, lse, ws, prefix_table=c.t_prefix)
    L.lf_attn_status(ws)
    k, v, qq = R.f64(c.k), R.f64(c.v), R.f64(q)
    rows, prows = np.setdiff1d(np.arange(n), gone), np.setdiff1d(np.arange(prefix), pgone)
    for b in (0, B - 1):
        for h in range(2 * Hkv):
            kk, vv = (np.concatenate([R.cache_rows(x, c.prefix_table, prefix, h // 2)[prows],
                                      R.cache_rows(x, c.table[b], n, h // 2)[rows]]) for x in (k, v))
            ro, rl, to, tl = R.softmax_row(qq[b, h], kk, vv, 0.125, R.half_step(dtype))
            R.check("o", R.f64(o[b, h]), ro, to + 2.0 ** -22 + R.half_step(dtype) * (np.abs(ro) + to))
            R.check("lse", R.f64(lse[b, h]), rl, tl)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("B,Hkv,prefix", [(3, 1, 0), (3, 1, 150), (20, 2, 900), (40, 2, 200), (80, 1, 0), (80, 1, 40)])
def test_decode_nan_query_stays_nan_and_its_own(dtype, B, Hkv, prefix):
    """A NaN in a query makes its output and lse NaN; the other queries' bits
    stay, and so does the zero of a query without keys."""
    import torch
    c = Cache(79, dtype, B, Hkv, 16, [0] + [200] * (B - 1), prefix)
    q = _normal(c.rng, (B, 4 * Hkv, 64), dtype)
    p = c.params(4 * Hkv)
    ws = L.paged_workspace(p)
    out = []
    for bad in (False, True):
        if bad:
            q[1, 2, 5] = math.nan
        o, lse = torch.empty_like(q), torch.empty(B, 4 * Hkv, device="cuda")
        L.lf_paged_decode(p, q, c.k, c.v, c.t_table, c.t_lengths, o, lse, ws, prefix_table=c.t_prefix)
        L.lf_attn_status(ws)
        out.append((o, lse))
    assert out[1][0][1, 2].isnan().all() and out[1][1][1, 2].isnan()
    for x, y in zip(out[0], out[1]):
        assert not x.isnan().any()
        y = y.clone()
        y[1, 2] = x[1, 2]
        assert torch.equal(x, y)
    if not prefix:
        assert (out[0][0][0] == 0).all() and (out[0][1][0] == -math.inf).all()


@pytest.mark.parametrize("B,prefix", [(2, 0), (40, 0), (80, 0), (40, 150), (1, 9000)])
def test_pools_beyond_2_31_elements(B, prefix):
    """Pages at the end of pools of more than 2^31 elements: append, then decode
    by each of the kernels, against the same rows in a small pool."""
    import torch
    page, cols, num = 1024, 2, 2 ** 21 // 64 + 2 * 40 + 20
    small = B * cols + 12
    far = num - small                       # the big pool's last pages are the small pool's
    big = [torch.empty(num, 1, page, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert big[0].numel() > 2 ** 31 and far * page * 64 > 2 ** 31 - 2 ** 23
    rng = np.random.default_rng(13)
    pools = [_normal(rng, (small, 1, page, 64), "bf16") for _ in range(2)]
    for x, y in zip(big, pools):
        x[far:] = y
    table = torch.from_numpy(rng.permutation(small)[:B * cols].reshape(B, cols).astype(np.int32)).cuda()
    pre = torch.arange(small - 9, small, dtype=torch.int32, device="cuda")[:-(-prefix // page)] if prefix else None
    lengths = torch.full((B,), 1500, dtype=torch.int32, device="cuda")
    q, k, v = (_normal(rng, (B, h, 64), "bf16") for h in (2, 1, 1))
    out = []
    for n, (kp, vp), off in ((small, pools, 0), (num, big, far)):
        p = L.make_paged_params(B, 2, 1, page, n, cols, 300, None, 0.0, L.LF_BF16, prefix)
        ws = L.paged_workspace(p)
        qo, o, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(B, 2, device="cuda")
        t = table + off
        L.lf_cache_append(p, L.make_rope_params(), q, k, v, lengths, t, qo, kp, vp, ws)
        L.lf_paged_decode(p, qo, kp, vp, t, lengths, o, lse, ws, prefix_table=None if pre is None else pre + off)
        L.lf_attn_status(ws)
        out.append((o, lse))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    assert all(torch.equal(x[far:], y) for x, y in zip(big, pools))     # the appended rows, and no other


def test_decode_captured_and_two_graphs_share_a_workspace():
    """Replays follow the lengths and tables of the moment; two graphs with one
    workspace, replayed one after the other, do not disturb each other."""
    import torch
    c = Cache(61, "bf16", 6, 2, 16, [90, 17, 64, 3, 0, 33], prefix=333)
    p = c.params(4, 20)
    ws = L.paged_workspace(p)
    qs = [_normal(c.rng, (6, 4, 64), "bf16") for _ in range(2)]
    outs = [(torch.empty_like(q), torch.empty(6, 4, device="cuda")) for q in qs]
    args = lambda q, o: (p, q, c.k, c.v, c.t_table, c.t_lengths, o[0], o[1], ws, c.t_prefix)  # noqa: E731
    for q, o in zip(qs, outs):
        L.lf_paged_decode(*args(q, o))
    graphs = []
    for q, o in zip(qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.lf_paged_decode(*args(q, o))
        graphs.append(g)
    for lens in ([90, 17, 64, 3, 0, 33], [1, 0, 20, 3, 0, 30]):
        c.t_lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        want = []
        for q in qs:
            o = torch.empty_like(q), torch.empty(6, 4, device="cuda")
            L.lf_paged_decode(*args(q, o))
            want.append(o)
        for o in outs:
            o[0].zero_()
        for _ in range(3):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    L.lf_attn_status(ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs[0][0].zero_()
    side.wait_stream(torch.cuda.current_stream())
    L.lf_paged_decode(*args(qs[0], outs[0]), stream=side)
    side.synchronize()
    assert torch.equal(outs[0][0], want[0][0])


def test_decode_calls_with_other_params_share_a_workspace():
    """One zeroed workspace for calls of different batches and heads, each
    repeated: the same bits every time, and those of a fresh workspace."""
    import torch
    runs = []
    for k, (H, Hkv, lengths, prefix) in enumerate([(4, 2, [(b * 29) % 300 for b in range(64)], 0), (12, 3, [900] * 30, 50),
                                                   (2, 2, [5, 700], 130), (40, 1, [77] * 90, 0)]):
        c = Cache(510 + k, "bf16", len(lengths), Hkv, 16, lengths, prefix)
        runs.append((c, c.params(H), _normal(c.rng, (len(lengths), H, 64), "bf16")))
    ws = torch.zeros(max(L.lf_paged_workspace_size(p) for _, p, _ in runs), dtype=torch.uint8, device="cuda")

    def once(c, p, q, w):
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        L.lf_paged_decode(p, q, c.k, c.v, c.t_table, c.t_lengths, o, lse, w, prefix_table=c.t_prefix)
        return o, lse

    want = [once(*r, L.paged_workspace(r[1])) for r in runs]
    for _ in range(3):
        for r, w in zip(runs, want):
            got = once(*r, ws)
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    L.lf_attn_status(ws)


# ------------------------------------------------------------------- append --

APPEND = [
    # H, Hkv, page, lengths, new tokens (None: one each), rot, interleaved, axes, positions given, prefix
    (1, 1, 16, [1], None, 64, False, 1, False, 0),
    (8, 8, 64, [70, 0, 64, 65], None, 64, False, 1, False, 100),
    (6, 2, 16, [33, 16, 500], None, 64, True, 1, True, 0),
    (4, 4, 32, [40, 100, 7, 0, 33], [40, 1, 7, 0, 32], 64, False, 1, False, 7),
    (12, 3, 16, [200, 17], [199, 17], 48, False, 3, True, 0),
    (2, 2, 128, [129, 5, 300], [128, 0, 3], 10, False, 1, False, 0),
    (2, 1, 16, [31, 90], [1, 90], 0, False, 1, False, 0),      # no rotation
    (4, 1, 16, [b % 9 for b in range(300)], [min(b % 9, b % 4) for b in range(300)], 32, True, 2, True, 0),
]


def _positions(rng, axes, T):
    return rng.integers(0, 2 ** 30, (axes, T)).astype(np.int32)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_matches_float64(case, dtype):
    import torch
    H, Hkv, page, lengths, new, rot, inter, axes, given, prefix = APPEND[case]
    B = len(lengths)
    c = Cache(400 + case, dtype, B, Hkv, page, lengths)
    c.prefix = prefix
    counts = [1] * B if new is None else new
    tail = 0 if new is None else 3                    # tokens behind the last sequence
    T = sum(counts) + tail
    q, k, v = (_normal(c.rng, (h, T, 64), dtype).transpose(0, 1) for h in (H, Hkv, Hkv))
    cu = None if new is None else torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    pair_axis = [p % axes for p in range(rot // 2)] if axes > 1 else None
    rope = L.make_rope_params(rot, inter, axes, pair_axis) if rot else None
    pos = _positions(c.rng, axes, T) if given else None
    p = c.params(H)
    ws = L.paged_workspace(p)
    before = [x.clone() for x in (c.k, c.v)]
    qo = torch.full((T, H, 64), 7.0, dtype=q.dtype, device="cuda")
    L.lf_cache_append(p, rope, q, k, v, c.t_lengths, c.t_table, qo, c.k, c.v, ws, cu_new=cu,
                      positions=None if pos is None else torch.from_numpy(pos).cuda())
    L.lf_attn_status(ws)
    half = R.half_step(dtype)
    ek, ev, eq = (R.f64(x) for x in (*before, torch.full_like(qo, 7.0)))
    tk, tq = np.zeros(ek.shape), np.zeros(eq.shape)
    t = 0
    for b, cnt in enumerate(counts):
        if new is None and lengths[b] == 0:
            t += 1
            continue
        for i in range(cnt):
            row = lengths[b] - cnt + i
            at = (np.array([[prefix + row]]) if pos is None else pos[:, t:t + 1])
            for x, e, tol, idx in ((q, eq, tq, (t, slice(None))), (k, ek, tk, (c.table[b, row // page], slice(None), row % page))):
                y, allow = R.rope(R.f64(x[t]), at, rot, inter, pair_axis)
                e[idx], tol[idx] = y, allow + half * np.abs(y) if rot else 0.0
            ev[c.table[b, row // page], :, row % page] = R.f64(v[t])
            t += 1
    same = lambda x: np.nan_to_num(x, nan=1e9, posinf=2e9)  # noqa: E731  the untouched rows hold NaN and infinities
    R.check("q", R.f64(qo), eq, tq)
    R.check("k", same(R.f64(c.k)), same(ek), tk)
    R.check("v", same(R.f64(c.v)), same(ev), 0.0)


def test_append_without_query_and_in_place():
    import torch
    c = Cache(71, "bf16", 3, 2, 16, [5, 20, 16])
    d = Cache(71, "bf16", 3, 2, 16, [5, 20, 16])
    p, rope = c.params(4), L.make_rope_params()
    ws = L.paged_workspace(p)
    q, k, v = (_normal(c.rng, (3, h, 64), "bf16") for h in (4, 2, 2))
    qo = torch.empty_like(q)
    L.lf_cache_append(p, rope, q, k, v, c.t_lengths, c.t_table, qo, c.k, c.v, ws)
    L.lf_cache_append(p, rope, None, k, v, d.t_lengths, d.t_table, None, d.k, d.v, ws)
    L.lf_cache_append(p, rope, q, k, v, d.t_lengths, d.t_table, q, d.k, d.v, ws)      # q in place
    L.lf_attn_status(ws)
    assert torch.equal(q, qo)
    assert torch.equal(torch.nan_to_num(c.k.float()), torch.nan_to_num(d.k.float()))
    assert torch.equal(torch.nan_to_num(c.v.float()), torch.nan_to_num(d.v.float()))


def test_append_skips_bad_tables_and_lengths():
    import torch
    c = Cache(81, "f32", 4, 1, 16, [20, 30, 5, 1])
    p = c.params(1)
    ws = L.paged_workspace(p)
    k = torch.ones(4, 1, 64, device="cuda")
    rows = [20, 30, 5, 1]

    def call(table, lens, cu, x, detail):
        pools = torch.zeros_like(c.k), torch.zeros_like(c.v)
        L.lf_cache_append(p, None, None, x, x, lens, table, None, *pools, ws, cu_new=cu)
        with pytest.raises(L.LfError) as e:
            L.lf_attn_status(ws)
        assert e.value.code == L.LF_ERR_DEVICE_INPUT and detail in str(e.value)
        return pools

    def expect(pools, seqs):
        want = torch.zeros_like(c.k)
        for b in seqs:
            want[c.table[b, (rows[b] - 1) // 16], :, (rows[b] - 1) % 16] = 1
        assert torch.equal(pools[0], want) and torch.equal(pools[1], want)

    for bad in (-1, c.num, 2 ** 31 - 1, -2 ** 31):
        table = c.t_table.clone()
        table[1, 1] = bad
        expect(call(table, c.t_lengths, None, k, "sequence 1"), [0, 2, 3])
    for bad in (-1, c.table.shape[1] * 16 + 1, 2 ** 31 - 1, -2 ** 31):
        lens = c.t_lengths.clone()
        lens[2] = bad
        expect(call(c.t_table, lens, None, k, "sequence 2"), [0, 1, 3])
    # more tokens than the sequence is long, and offsets that do not ascend
    cu = torch.tensor([0, 1, 2, 3, 5], dtype=torch.int32, device="cuda")
    expect(call(c.t_table, c.t_lengths, cu, torch.ones(5, 1, 64, device="cuda"), "sequence 3"), [0, 1, 2, 3])
    cu = torch.tensor([2, 1, 0, -5, 4], dtype=torch.int32, device="cuda")
    pools = call(c.t_table, c.t_lengths, cu, k, "cu_new")
    assert int((pools[0] != 0).sum()) <= 4 * 64


def test_append_captured_follows_the_lengths():
    import torch
    c = Cache(91, "bf16", 2, 2, 16, [64, 64])
    p, rope = c.params(2), L.make_rope_params(interleaved=True)
    ws = L.paged_workspace(p)
    q, k, v = (_normal(c.rng, (2, 2, 64), "bf16") for _ in range(3))
    qo, qe = torch.empty_like(q), torch.empty_like(q)
    lens = torch.tensor([1, 40], dtype=torch.int32, device="cuda")
    L.lf_cache_append(p, rope, q, k, v, lens, c.t_table, qo, c.k, c.v, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.lf_cache_append(p, rope, q, k, v, lens, c.t_table, qo, c.k, c.v, ws)
        lens.add_(1)
    ek, ev = c.k.clone(), c.v.clone()
    for step in range(3):
        now = lens.clone()
        g.replay()
        L.lf_cache_append(p, rope, q, k, v, now, c.t_table, qe, ek, ev, ws)
        torch.cuda.synchronize()
        # bit for bit (the untouched rows hold NaN)
        assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in ((qo, qe), (c.k, ek), (c.v, ev)))
    L.lf_attn_status(ws)
    assert lens.tolist() == [4, 43]


def test_paged_python_refusals():
    import torch
    c = Cache(95, "bf16", 2, 2, 16, [5, 6], prefix=20)
    p, rope = c.params(4), L.make_rope_params()
    ws = L.paged_workspace(p)
    q, k, v = (_normal(c.rng, (2, h, 64), "bf16") for h in (4, 2, 2))
    o, lse = torch.empty_like(q), torch.empty(2, 4, device="cuda")
    good = dict(q=q, k_pages=c.k, v_pages=c.v, block_table=c.t_table, lengths=c.t_lengths, o=o, lse=lse, ws=ws,
                prefix_table=c.t_prefix)
    L.lf_paged_decode(p, **good)
    for kw in (dict(q=q[:1]), dict(q=q.float()), dict(q=q.cpu()), dict(k_pages=c.k[:-1]), dict(v_pages=c.v.transpose(1, 2)),
               dict(block_table=c.t_table[:, :1]), dict(block_table=c.t_table.long()), dict(lengths=c.t_lengths[:1]),
               dict(lengths=c.t_lengths.cpu()), dict(o=o.float()), dict(o=o.transpose(0, 1).contiguous().transpose(0, 1)),
               dict(lse=lse.half()), dict(lse=lse[:1]), dict(ws=ws[:256]), dict(ws=ws[16:]), dict(ws=ws.float()),
               dict(prefix_table=None), dict(prefix_table=c.t_prefix[:1]), dict(k_pages=c.k.cpu()),
               dict(q=torch.zeros(2, 4, 66, dtype=q.dtype, device="cuda")[..., 1:65])):
        with pytest.raises(L.LfError) as e:
            L.lf_paged_decode(p, **{**good, **kw})
        assert e.value.code == L.LF_ERR_INVALID, kw
    good = dict(q=q, k=k, v=v, lengths=c.t_lengths, block_table=c.t_table, q_out=o, k_pages=c.k, v_pages=c.v, ws=ws)
    L.lf_cache_append(p, rope, **good)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    for kw in (dict(q=None), dict(q_out=None), dict(k=k[:1]), dict(v=v.half()), dict(q_out=o[:1]), dict(cu_new=cu[:2]),
               dict(cu_new=cu.long()), dict(positions=cu), dict(positions=cu[None, :1]), dict(k=torch.cat([k, k])[:3], v=v),
               dict(k=torch.cat([k, k])[:3], v=torch.cat([k, k])[:3], q=torch.cat([q, q])[:3], q_out=torch.cat([q, q])[:3])):
        with pytest.raises(L.LfError) as e:
            L.lf_cache_append(p, rope, **{**good, **kw})
        assert e.value.code == L.LF_ERR_INVALID, kw
    with pytest.raises(L.LfError):
        L.lf_cache_append(p, L.make_rope_params(n_axes=2), **good)
    L.lf_attn_status(ws)


# ----------------------------------------------------------------- together --

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_append_and_steps_match_the_causal_forward(dtype):
    """A prompt through rotation and the causal forward, its rotated rows
    appended to the cache, then steps of append and decode: every step's output
    is the causal forward's row, and the contiguous decode step's."""
    import torch
    B, H, n, steps, page, r, dil = 2, 4, 150, 6, 16, 40, [1, 2, 1, 3]
    rng = np.random.default_rng(17)
    lens = [150, 97]                                     # of the prompts
    q, k, v = (_normal(rng, (B, H, n + steps, 64), dtype) for _ in range(3))
    rope = L.make_rope_params()
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    L.lf_rope_fwd(rope, [q, k], [qr, kr])
    total = n + steps
    pf = L.make_params(B, H, total, r, dil, True, 0.0, CODE[dtype], 0)
    ws_f = L.workspace(pf)
    mask = torch.ones(B, total, dtype=torch.int32, device="cuda")
    o_full, lse_full = torch.empty_like(q), torch.empty(B, H, total, device="cuda")
    L.lf_attn_fwd(pf, qr, kr, v, qr, kr, v, mask, o_full, lse_full, ws_f)
    L.lf_attn_status(ws_f)

    cols = -(-total // page)
    pages = B * cols + 2
    table = torch.from_numpy(rng.permutation(pages)[:B * cols].reshape(B, cols).astype(np.int32)).cuda()
    kp, vp = (torch.full((pages, H, page, 64), float("nan"), dtype=q.dtype, device="cuda") for _ in range(2))
    p = L.make_paged_params(B, H, H, page, pages, cols, r, dil, 0.0, CODE[dtype])
    ws = L.paged_workspace(p)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
    pack = lambda x: torch.cat([x[b, :, :lens[b]] for b in range(B)], 1).transpose(0, 1)  # noqa: E731
    qo = torch.empty(sum(lens), H, 64, dtype=q.dtype, device="cuda")
    L.lf_cache_append(p, rope, pack(q), pack(k), pack(v), lengths, table, qo, kp, vp, ws, cu_new=cu)
    assert torch.equal(qo, pack(qr).contiguous())        # the append turns as the rotation does
    u = R.half_step(dtype)
    for s in range(steps):
        lengths += 1
        now = [lens[b] + s for b in range(B)]
        at = lambda x: torch.stack([x[b, :, now[b]] for b in range(B)])  # noqa: E731
        qs = torch.empty(B, H, 64, dtype=q.dtype, device="cuda")
        L.lf_cache_append(p, rope, at(q), at(k), at(v), lengths, table, qs, kp, vp, ws)
        o, lse = torch.empty_like(qs), torch.empty(B, H, device="cuda")
        L.lf_paged_decode(p, qs, kp, vp, table, lengths, o, lse, ws)
        o1, lse1 = torch.empty_like(o), torch.empty_like(lse)
        L.lf_attn_decode(pf, qs, kr, v, lengths, o1, lse1)
        L.lf_attn_status(ws)
        assert torch.equal(qs, at(qr))
        # at most 41 keys of |v| < 6: roundings of P (16-bit forward) and of the two outputs
        for other, ol in ((at(o_full), at(lse_full[..., None])[..., 0]), (o1, lse1)):
            assert float((o.double() - other.double()).abs().max()) <= 6 * (3 * u + 2.0 ** -15)
            assert float((lse.double() - ol.double()).abs().max()) <= 2.0 ** -15 * (1 + float(lse.abs().max()))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_shared_prefix_is_the_same_as_a_copy_per_sequence(dtype):
    """A batch behind a shared prefix gives what each sequence gives with the
    prefix's rows copied into its own pages."""
    import torch
    B, H, Hkv, page, prefix = 5, 4, 2, 16, 96            # whole pages, so the copies are table entries
    lens = [1, 20, 33, 16, 50]
    c = Cache(97, dtype, B, Hkv, page, lens, prefix)
    q = _normal(c.rng, (B, H, 64), dtype)
    p = c.params(H)
    ws = L.paged_workspace(p)
    o, lse = torch.empty_like(q), torch.empty(B, H, device="cuda")
    L.lf_paged_decode(p, q, c.k, c.v, c.t_table, c.t_lengths, o, lse, ws, prefix_table=c.t_prefix)
    table = torch.cat([c.t_prefix.expand(B, prefix // page), c.t_table], 1).contiguous()
    p1 = L.make_paged_params(B, H, Hkv, page, c.num, table.shape[1], -1, None, 0.0, CODE[dtype])
    o1, lse1 = torch.empty_like(o), torch.empty_like(lse)
    L.lf_paged_decode(p1, q, c.k, c.v, table, c.t_lengths + prefix, o1, lse1, ws)
    L.lf_attn_status(ws)
    u = R.half_step(dtype)
    assert float((o.double() - o1.double()).abs().max()) <= 6 * (3 * u + 2.0 ** -15)
    assert float((lse - lse1).abs().max()) <= 2.0 ** -15 * (1 + float(lse.abs().max()))
