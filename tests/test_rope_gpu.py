"""GPU parity of the rotation (lf_rope_fwd / lf_rope_bwd) against float64."""
import numpy as np
import pytest

from sparse_sliding_window_b200 import lf_attn as L
from tests import paged_ref as R

pytestmark = pytest.mark.gpu


def _axes(n_axes, pairs):
    return [p * n_axes // pairs for p in range(pairs)] if n_axes > 1 else None


def _grid(rng, n_axes, B, n, kind):
    if kind == "far":
        return rng.integers(-2 ** 31, 2 ** 31, (n_axes, B, n)).astype(np.int32)
    return rng.integers(0, 5000, (n_axes, B, n)).astype(np.int32)


def _normal(rng, shape, dtype):
    import torch
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to("cuda", R.torch_dtype(dtype))


CASES = [
    # B, heads of the tensors, n, rot, interleaved, axes, positions
    (1, [1], 1, 64, False, 1, None),
    (2, [3, 1], 5, 64, False, 1, "near"),
    (1, [12, 12, 12, 12], 130, 64, True, 1, "far"),
    (3, [8, 2], 33, 48, False, 3, "near"),
    (2, [5], 65, 48, True, 3, "far"),
    (2, [2, 7], 19, 10, False, 2, "far"),
    (1, [4, 4], 257, 2, False, 1, None),
    (1, [3], 40, 10, True, 4, "near"),
    (1, [1, 2, 3, 4, 5, 6, 7, 8], 3, 32, False, 2, "near"),
]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_rope_matches_float64(case, dtype, back):
    import torch
    B, heads, n, rot, inter, n_axes, kind = CASES[case]
    rng = np.random.default_rng(100 + case)
    xs = [_normal(rng, (B, h, n, 64), dtype) for h in heads]
    outs = [torch.full_like(x, float("nan")) for x in xs]
    pos = None if kind is None else _grid(rng, n_axes, B, n, kind)
    axes = _axes(n_axes, rot // 2)
    r = L.make_rope_params(rot, inter, n_axes, axes)
    (L.lf_rope_bwd if back else L.lf_rope_fwd)(r, xs, outs, None if pos is None else torch.from_numpy(pos).cuda())
    at = np.broadcast_to(np.arange(n), (1, B, n)) if pos is None else pos
    for x, out in zip(xs, outs):
        ref, tol = R.rope(R.f64(x), at[:, :, None, :], rot, inter, axes, sign=-1.0 if back else 1.0)
        R.check("rope", R.f64(out), ref, tol + R.half_step(dtype) * np.abs(ref))
        assert torch.equal(out[..., rot:], x[..., rot:])   # channels that do not turn are copied


def test_rope_frequencies_of_the_caller():
    import torch
    rng = np.random.default_rng(7)
    x = _normal(rng, (1, 2, 50, 64), "f32")
    freqs = list(rng.uniform(-3, 3, 32))
    out = torch.empty_like(x)
    L.lf_rope_fwd(L.make_rope_params(freqs=freqs), [x], [out])
    ref, tol = R.rope(R.f64(x), np.arange(50)[None, None, None], 64, False, freqs=freqs)
    R.check("rope", R.f64(out), ref, tol + 2.0 ** -24 * np.abs(ref))


def test_rope_backward_is_the_gradient():
    """<g, d rope(x)/dx h> against central differences of the forward: the map
    is linear, so a step of any size gives the derivative up to roundings."""
    import torch
    rng = np.random.default_rng(11)
    B, H, n = 2, 3, 21
    x, h, g = (_normal(rng, (B, H, n, 64), "f32") for _ in range(3))
    pos = torch.from_numpy(_grid(rng, 1, B, n, "near")).cuda()
    r = L.make_rope_params(48)
    gx, up, dn = (torch.empty_like(x) for _ in range(3))
    L.lf_rope_bwd(r, [g], [gx], pos)
    L.lf_rope_fwd(r, [x + h], [up], pos)
    L.lf_rope_fwd(r, [x - h], [dn], pos)
    want = float((g.double() * (up.double() - dn.double()) / 2).sum())
    got = float((gx.double() * h.double()).sum())
    # each of the three results is off by at most 2^-21 (|x_u| + |x_v|) per element
    allow = 2.0 ** -20 * float((g.abs() * (x.abs() + h.abs()) * 2).sum() + (g.abs() * h.abs() * 2).sum())
    assert abs(got - want) <= allow


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rot,inter", [(64, False), (64, True), (10, False)])
def test_rope_strided_and_in_place(dtype, rot, inter):
    import torch
    rng = np.random.default_rng(5)
    B, H, n = 2, 3, 37
    packed = _normal(rng, (B, n, 2 * H, 64), dtype)          # q and k heads side by side, tokens first
    before = packed.clone()
    q, k = packed[:, :, :H].transpose(1, 2), packed[:, :, H:].transpose(1, 2)
    r = L.make_rope_params(rot, inter)
    qo = torch.empty(B, H, n, 64, dtype=packed.dtype, device="cuda")
    L.lf_rope_fwd(r, [q, k], [qo, k])                        # k in place
    for x, got in ((before[:, :, :H].transpose(1, 2), qo), (before[:, :, H:].transpose(1, 2), k)):
        ref, tol = R.rope(R.f64(x), np.arange(n)[None, None, None], rot, inter)
        R.check("rope", R.f64(got), ref, tol + R.half_step(dtype) * np.abs(ref))
    assert torch.equal(packed[:, :, :H], before[:, :, :H])   # q itself untouched
    # a broadcast input: every head the same tensor
    one = before[:, :, :1].transpose(1, 2).expand(B, H, n, 64)
    L.lf_rope_fwd(r, [one], [qo])
    assert all(torch.equal(qo[:, 0], qo[:, h]) for h in range(H))


def test_rope_keeps_infinities_and_nan_in_their_pairs():
    import torch
    for rot, inter in ((48, False), (10, True), (10, False)):
        x = torch.ones(1, 1, 4, 64, device="cuda")
        x[0, 0, 1, 60], x[0, 0, 2, 63] = float("inf"), float("nan")
        out = torch.empty_like(x)
        L.lf_rope_fwd(L.make_rope_params(rot, inter), [x], [out])
        assert torch.isinf(out[0, 0, 1, 60]) and torch.isnan(out[0, 0, 2, 63])
        assert int(torch.isfinite(out).sum()) == out.numel() - 2


def test_rope_captured_and_on_another_stream():
    import torch
    rng = np.random.default_rng(9)
    x = _normal(rng, (2, 4, 64, 64), "bf16")
    out, eager = torch.empty_like(x), torch.empty_like(x)
    pos = torch.zeros(1, 2, 64, dtype=torch.int32, device="cuda")
    r = L.make_rope_params()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    L.lf_rope_fwd(r, [x], [out], pos, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lf_rope_fwd(r, [x], [out], pos)
        L.lf_rope_fwd(r, [out], [out], pos)                  # in place, behind the first
    for k in (1, 77):
        pos.fill_(k)
        graph.replay()
        L.lf_rope_fwd(r, [x], [eager], pos)
        L.lf_rope_fwd(r, [eager], [eager], pos)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_rope_python_refusals():
    import torch
    x = torch.zeros(2, 3, 5, 64, device="cuda")
    r = L.make_rope_params()
    for xs, outs, pos in (([x], [x[:, :2]], None), ([x], [x.double()], None), ([x], [x, x], None), ([x[0]], [x[0]], None),
                          ([x], [torch.zeros(2, 3, 5, 64)], None), ([x[..., :32]], [x[..., :32]], None),
                          ([x], [x], torch.zeros(1, 2, 4, dtype=torch.int32, device="cuda")),
                          ([x], [x], torch.zeros(1, 2, 5, device="cuda")),
                          ([x], [x], torch.zeros(1, 2, 5, dtype=torch.int32)),
                          ([x.transpose(2, 3).contiguous().transpose(2, 3)], [x], None),
                          ([x.double()], [x.double()], None), ([x], [x[:, :1].expand(2, 3, 5, 64)], None)):
        with pytest.raises(L.LfError) as e:
            L.lf_rope_fwd(r, xs, outs, pos)
        assert e.value.code == L.LF_ERR_INVALID
