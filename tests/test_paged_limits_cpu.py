"""Host checks of include/lf_paged.h at the limits that it states, without a GPU."""
import ctypes

import pytest

from sparse_sliding_window_b200 import build as lfbuild
from sparse_sliding_window_b200 import lf_attn as L


@pytest.fixture(scope="module")
def lib():
    lfbuild.build()
    return L.load()


def _rope(lib, r, heads=1):
    """lf_rope_fwd with a NULL tensor: what is refused before that is refused by the params."""
    t = L.lf_rope_tensor()
    t.x, t.out, t.heads = None, None, heads
    code = lib.lf_rope_fwd(ctypes.byref(r), 1, 1, L.LF_F32, 1, ctypes.byref(t), None, None)
    return code, lib.lf_attn_last_error().decode()


def _c_params(base):
    r = L.lf_rope_params()
    r.rot_dim, r.n_axes, r.base = 64, 1, base
    return r


@pytest.mark.parametrize("base", [1e-8, 1e-300])
def test_a_base_too_small_is_named(lib, base):
    for r in (_c_params(base), L.make_rope_params(base=base)):
        code, text = _rope(lib, r)
        assert code == L.LF_ERR_INVALID and "base" in text and "freqs" not in text


def test_frequency_and_head_limits(lib):
    assert "x is NULL" in _rope(lib, _c_params(1e-6))[1]            # 1e-6^(-62/64) = 6.5e5
    assert "x is NULL" in _rope(lib, L.make_rope_params(freqs=[1e6, -1e6] * 16))[1]
    code, text = _rope(lib, L.make_rope_params(freqs=[1.0] * 31 + [1.0001e6]))
    assert code == L.LF_ERR_INVALID and "freqs[31]" in text
    assert "x is NULL" in _rope(lib, L.make_rope_params(), 128)[1]
    assert "heads" in _rope(lib, L.make_rope_params(), 129)[1]


PAGED = dict(B=2, H=4, Hkv=2, page_size=16, num_pages=9, max_pages=4, window=5, dtype=L.LF_BF16)


def test_scale_that_overflows_in_base_2(lib):
    """Scores are kept in base 2: scale * log2 e must be finite, too."""
    for scale, fine in ((2.3e38, True), (2.4e38, False), (3.4e38, False)):
        assert (L.lf_paged_workspace_size(L.make_paged_params(scale=scale, **PAGED)) > 0) == fine, scale
