"""The paged cache without a GPU: the exports and host checks of
include/lf_paged.h, and the index arithmetic that every kernel takes its
addresses from (csrc/lf_pages.cuh, compiled here as host C++), good tables and
bad ones."""
import ctypes
import os
import random
import re
import subprocess

import numpy as np
import pytest

from sparse_sliding_window_b200 import build as lfbuild
from sparse_sliding_window_b200 import lf_attn as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    lfbuild.build()
    return L.load()


# --------------------------------------------------------- index arithmetic --

SHIM = """
#include "lf_pages.cuh"
extern "C" int pool_row(const int32_t *t, int c, int n, int s, int hkv, int h, int r) { return lf_pool_row(t, c, n, s, hkv, h, r); }
extern "C" int window_keys(int len, int w, int d) { return lf_window_keys(len, w, d); }
extern "C" int token_seq(const int32_t *cu, int B, int t) { return lf_token_seq(cu, B, t); }
extern "C" int new_row(int len, int cnt, int i, int c, int s, int ragged) { return lf_new_row(len, cnt, i, c, s, ragged != 0); }
extern "C" int len_ok(int len, int c, int s) { return lf_len_ok(len, c, s); }
"""


@pytest.fixture(scope="module")
def pages(tmp_path_factory):
    d = tmp_path_factory.mktemp("pages")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.check_call(["g++", "-O1", "-shared", "-fPIC", "-I", os.path.join(ROOT, "sparse_sliding_window_b200", "csrc"),
                           "-o", str(so), str(src)])
    return ctypes.CDLL(str(so))


def _i32(values):
    return (ctypes.c_int32 * len(values))(*values)


def test_pool_rows_stay_inside_the_pool(pages):
    num, hkv, shift, cols = 7, 3, 4, 4
    table = [6, 0, 3, 5]
    seen = set()
    for h in range(hkv):
        for row in range(cols << shift):
            at = pages.pool_row(_i32(table), cols, num, shift, hkv, h, row)
            assert at == (table[row >> shift] * hkv + h) * 16 + row % 16
            assert 0 <= at < num * hkv * 16
            seen.add(at)
    assert len(seen) == hkv * (cols << shift)   # no two rows share a place


@pytest.mark.parametrize("page", [-1, -2 ** 31, 7, 8, 2 ** 31 - 1])
def test_bad_pages_and_rows_have_no_address(pages, page):
    table = _i32([page, 2])
    for row in (0, 15):
        assert pages.pool_row(table, 2, 7, 4, 3, 2, row) == -2
    assert pages.pool_row(table, 2, 7, 4, 3, 2, 16) == (2 * 3 + 2) * 16
    for row in (-1, -2 ** 31, 32, 33, 2 ** 31 - 1):   # outside the table: it is not read
        assert pages.pool_row(table, 2, 7, 4, 3, 2, row) == -1


def test_largest_pool_row_is_below_2_31(pages):
    # num_pages * Hkv * page_size < 2^31 is what the host lets through
    num, hkv, shift = 2 ** 20 - 1, 2, 10
    at = pages.pool_row(_i32([num - 1]), 1, num, shift, hkv, hkv - 1, 1023)
    assert at == ((num - 1) * hkv + hkv - 1) * 1024 + 1023 and at < 2 ** 31


def test_window_keys(pages):
    for length in (-5, 0, 1, 2, 17, 300):
        for window in (-1, 0, 1, 5, 299, 2 ** 31 - 1):
            for d in (1, 2, 3, 400, 2 ** 31 - 1):
                if window < 0 and d > 1:
                    continue
                want = [j for j in range(length) if window < 0 or ((length - 1 - j) % d == 0 and (length - 1 - j) // d <= window)]
                assert pages.window_keys(length, window, d) == len(want)
                if want:   # the last key is a row
                    assert length - 1 - (len(want) - 1) * (1 if window < 0 else d) == want[0]


def test_token_sequences(pages):
    rng = random.Random(3)
    for _ in range(50):
        B = rng.randint(1, 40)
        counts = [rng.choice([0, 0, 1, 2, 7]) for _ in range(B)]
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(int).tolist()
        for t in range(cu[-1]):
            b = pages.token_seq(_i32(cu), B, t)
            assert cu[b] <= t < cu[b + 1]
        assert 0 <= pages.token_seq(_i32(cu), B, cu[-1] + 3) < B
        junk = [rng.randint(-2 ** 31, 2 ** 31 - 1) for _ in range(B + 1)]
        for t in (0, 5, 2 ** 31 - 1):
            assert 0 <= pages.token_seq(_i32(junk), B, t) < B


def test_new_rows(pages):
    assert [pages.new_row(10, 3, i, 2, 4, 1) for i in range(3)] == [7, 8, 9]
    assert pages.new_row(0, 1, 0, 2, 4, 0) == -1            # idle
    assert pages.new_row(0, 1, 0, 2, 4, 1) == -2            # a token for an empty cache
    assert pages.new_row(2, 3, 0, 2, 4, 1) == -2 and pages.new_row(2, 3, 1, 2, 4, 1) == 0
    assert pages.new_row(32, 1, 0, 2, 4, 0) == 31
    for length in (33, -1, -2 ** 31, 2 ** 31 - 1):
        assert pages.new_row(length, 1, 0, 2, 4, 0) == -2 and not pages.len_ok(length, 2, 4)


# ---------------------------------------------------------------- host checks --

def test_exports(lib):
    text = open(os.path.join(ROOT, "include", "lf_paged.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(lf_(?:rope|paged|cache)_\w+)\s*\(", text)))
    assert names == sorted(L.PAGED_EXPORTS)
    for name in names:
        assert hasattr(lib, name), name


GOOD = dict(B=2, H=4, Hkv=2, page_size=16, num_pages=9, max_pages=4, window=5, dtype=L.LF_BF16)


def test_workspace_sizes(lib):
    small = L.lf_paged_workspace_size(L.make_paged_params(**GOOD))
    assert small > 0 and small % 256 == 0
    more = L.lf_paged_workspace_size(L.make_paged_params(**{**GOOD, "B": 200, "prefix_len": 1000}))
    assert more >= small + 200 * 4 * (64 + 2) * 4 and more % 256 == 0   # a part of every query at least
    for bad in (dict(B=0), dict(H=0), dict(Hkv=0), dict(Hkv=3), dict(H=256, Hkv=2), dict(page_size=8), dict(page_size=24),
                dict(page_size=2048), dict(num_pages=0), dict(max_pages=0), dict(dtype=3), dict(prefix_len=-1),
                dict(prefix_len=2 ** 30 + 1), dict(head_dim=128), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(dilation=[1, 0]), dict(window=-1, dilation=[1, 2]), dict(B=1000000), dict(B=999999, H=6, prefix_len=10),
                dict(num_pages=2 ** 27), dict(max_pages=2 ** 26 + 1)):
        assert L.lf_paged_workspace_size(L.make_paged_params(**{**GOOD, **bad})) == 0, bad
        assert lib.lf_attn_last_error(), bad
    assert lib.lf_paged_workspace_size(None) == 0


def _buf(n=8192):
    buf = (ctypes.c_char * n)()
    return buf, (ctypes.addressof(buf) + 255) & ~255


def test_decode_and_append_refusals(lib):
    keep, a = _buf()
    p = L.make_paged_params(**GOOD)
    pp = ctypes.byref(p)

    def decode(par=pp, q=a, st=None, kp=a, vp=a, table=a, lens=a, pre=None, o=a, lse=None, ws=a, n=1 << 30):
        return lib.lf_paged_decode(par, q, st, kp, vp, table, lens, pre, o, lse, ws, n, None)

    for kw in (dict(par=None), dict(q=None), dict(q=a + 2), dict(kp=None), dict(vp=a + 8), dict(table=None), dict(table=a + 1),
               dict(lens=None), dict(o=None), dict(o=a + 4), dict(lse=a + 2), dict(ws=None), dict(ws=a + 16), dict(n=16),
               dict(st=(ctypes.c_int64 * 2)(-64, 64)), dict(st=(ctypes.c_int64 * 2)(256, 65))):
        assert decode(**kw) == L.LF_ERR_INVALID, kw
    pre = L.make_paged_params(**{**GOOD, "prefix_len": 100})
    assert decode(par=ctypes.byref(pre)) == L.LF_ERR_INVALID and b"prefix_table" in lib.lf_attn_last_error()
    wide = L.make_paged_params(**{**GOOD, "head_dim": 128})
    assert decode(par=ctypes.byref(wide)) == L.LF_ERR_UNSUPPORTED

    def append(par=pp, rope=None, T=2, q=a, k=a, v=a, st=None, cu=None, lens=a, pos=None, table=a, qo=a, kp=a, vp=a, ws=a, n=1 << 30):
        return lib.lf_cache_append(par, rope, T, q, k, v, st, cu, lens, pos, table, qo, kp, vp, ws, n, None)

    two = ctypes.byref(L.make_rope_params(n_axes=2, pair_axis=[0, 1] * 16))
    for kw in (dict(par=None), dict(T=-1), dict(T=3), dict(q=None), dict(qo=None), dict(k=None), dict(v=a + 2), dict(kp=None),
               dict(vp=None), dict(lens=None), dict(lens=a + 2), dict(cu=a + 3), dict(pos=a + 1), dict(table=None), dict(ws=None),
               dict(n=0), dict(rope=two), dict(st=(ctypes.c_int64 * 6)(512, 64, 128, 64, 128, 64)),
               dict(q=a + 512, st=(ctypes.c_int64 * 6)(256, 60, 128, 64, 128, 64))):
        assert append(**kw) == L.LF_ERR_INVALID, kw
    assert append(T=0, cu=a) == L.LF_OK      # nothing to do: no launch


def test_rope_refusals(lib):
    keep, a = _buf()
    good = L.make_rope_params()

    def call(r=good, B=2, n=5, dtype=L.LF_BF16, heads=3, x=a, out=a, xs=(960, 320, 64), os=(960, 320, 64), nt=1, pos=None, fn=None):
        t = L.lf_rope_tensor()
        t.x, t.out, t.heads = x, out, heads
        t.x_stride[:], t.out_stride[:] = xs, os
        return (fn or lib.lf_rope_fwd)(r if r is None else ctypes.byref(r), B, n, dtype, nt, ctypes.byref(t), pos, None)

    for kw in (dict(r=None), dict(B=0), dict(n=0), dict(dtype=5), dict(heads=0), dict(heads=129), dict(x=None), dict(out=a + 8),
               dict(nt=0), dict(nt=9), dict(pos=a + 2), dict(xs=(960, 320, 60)), dict(xs=(-960, 320, 64)), dict(os=(960, 0, 64)),
               dict(out=a + 4096, os=(960, 320, 56)), dict(out=a + 4096, os=(256, 320, 64)), dict(xs=(1920, 320, 64)),
               dict(r=L.make_rope_params(rot_dim=7, pair_axis=None)), dict(r=L.make_rope_params(rot_dim=66)),
               dict(r=L.make_rope_params(n_axes=0)), dict(r=L.make_rope_params(n_axes=5)), dict(r=L.make_rope_params(n_axes=2)),
               dict(r=L.make_rope_params(pair_axis=[0] * 31 + [1])), dict(r=L.make_rope_params(base=-1.0)),
               dict(r=L.make_rope_params(base=float("nan"))), dict(r=L.make_rope_params(freqs=[float("inf")] * 32))):
        assert call(**kw) == L.LF_ERR_INVALID, kw
        assert call(fn=lib.lf_rope_bwd, **kw) == L.LF_ERR_INVALID, kw


def test_python_binding_refuses_cpu_tensors_and_bad_lists(lib):
    import torch
    x = torch.zeros(1, 1, 4, 64)
    with pytest.raises(L.LfError):
        L.lf_rope_fwd(L.make_rope_params(), [x], [x])
    with pytest.raises(L.LfError):
        L.lf_rope_fwd(L.make_rope_params(), [], [])
    with pytest.raises(L.LfError):
        L.make_rope_params(rot_dim=32, pair_axis=[0] * 32)
    with pytest.raises(L.LfError):
        L.make_paged_params(**{**GOOD, "dilation": [1]})
    p = L.make_paged_params(**GOOD)
    pool = torch.zeros(9, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(L.LfError):
        L.lf_paged_decode(p, pool, pool, pool, pool, pool, pool, None, pool)
