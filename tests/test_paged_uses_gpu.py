"""GPU tests of uses of the paged cache that the other files leave out: calls at
once, on streams and host threads, strided queries in every kernel, the widest
head group, pages that several tables hold, nothing to append."""
import threading

import numpy as np
import pytest

from sparse_sliding_window_b200 import lf_attn as L
from tests import paged_ref as R
from tests.test_paged_gpu import Cache, _decode_and_check, _normal
from tests.test_paged_numerics_gpu import PATHS

pytestmark = pytest.mark.gpu


def _setup(seed, path, dtype):
    import torch
    B, H, Hkv, prefix, n = PATHS[path]
    c = Cache(seed, dtype, B, Hkv, 16, [max(0, n - (b * 7) % (n + 1)) for b in range(B)], prefix)
    p = c.params(H)
    q = _normal(c.rng, (B, H, 64), dtype)
    return c, p, q, L.paged_workspace(p), (torch.empty_like(q), torch.empty(B, H, device="cuda"))


def _call(s, stream=None):
    c, p, q, ws, (o, lse) = s
    L.lf_paged_decode(p, q, c.k, c.v, c.t_table, c.t_lengths, o, lse, ws, prefix_table=c.t_prefix, stream=stream)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_calls_at_once_on_streams_and_threads(dtype):
    """Every kernel on a stream of its own, from one host thread and from several, again and again."""
    import torch
    runs = [_setup(920 + i, path, dtype) for i, path in enumerate(PATHS)]
    want = []
    for s in runs:
        _call(s)
        torch.cuda.synchronize()
        want.append([x.clone() for x in s[4]])
    streams = [torch.cuda.Stream() for _ in runs]

    def check():
        torch.cuda.synchronize()
        for s, w in zip(runs, want):
            assert torch.equal(s[4][0], w[0]) and torch.equal(s[4][1], w[1])
            for x in s[4]:
                x.zero_()
        torch.cuda.synchronize()

    for s in runs:
        for x in s[4]:
            x.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for s, stream in zip(runs, streams):
            _call(s, stream)
    check()
    failed = []

    def work(s, stream):
        try:
            for _ in range(20):
                _call(s, stream)
        except Exception as e:  # noqa: BLE001  seen by the test's thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(runs, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    check()
    for s in runs:
        L.lf_attn_status(s[3])


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("path", PATHS)
def test_strided_and_broadcast_queries(path, dtype):
    """Heads first with padded rows, and one query for all: the bits of contiguous ones."""
    import torch
    c, p, q, ws, (o, lse) = s = _setup(940, path, dtype)
    _call(s)
    B, H = q.shape[:2]
    wide = torch.full((H, B, 96), float("nan"), dtype=q.dtype, device="cuda")
    view = wide.transpose(0, 1)[..., 32:]
    view.copy_(q)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    _call((c, p, view, ws, (o2, lse2)))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    one = q[:1, :1].expand(B, H, 64)
    _call((c, p, one, ws, (o, lse)))
    _call((c, p, one.contiguous(), ws, (o2, lse2)))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("B,prefix,window", [(1, 0, -1), (2, 70, 9), (50, 0, 20), (40, 150, -1)])
def test_one_group_of_all_heads(B, prefix, window, dtype):
    _decode_and_check(Cache(950, dtype, B, 1, 32, [(b * 31) % 90 + 1 for b in range(B)], prefix), 128, window)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("B,Hkv,prefix", [(3, 2, 64), (40, 2, 96), (24, 2, 96), (40, 2, 0)])
def test_pages_in_several_tables(B, Hkv, prefix, dtype):
    """Sequences that hold the same pages, a table with one page twice, and the prefix's page in a sequence's table."""
    import torch
    c = Cache(960, dtype, B, Hkv, 16, [70] * B, prefix)
    c.table[1::2] = c.table[0]                    # half of the batch shares one sequence's pages
    c.table[2, 1] = c.table[2, 0]
    if prefix:
        c.table[2, 3] = c.prefix_table[1]
        c.prefix_table[0] = c.prefix_table[2]
        c.t_prefix = torch.from_numpy(c.prefix_table).cuda()
    c.t_table = torch.from_numpy(c.table).cuda()
    _decode_and_check(c, 2 * Hkv, -1)


def test_append_of_nothing_and_of_one_token_to_a_page_border():
    import torch
    c = Cache(970, "bf16", 3, 2, 16, [17, 16, 0])
    p, rope = c.params(4), L.make_rope_params()
    ws = L.paged_workspace(p)
    before = c.k.clone(), c.v.clone()
    empty = [torch.empty(0, h, 64, dtype=c.k.dtype, device="cuda") for h in (4, 2, 2)]
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    L.lf_cache_append(p, rope, *empty, c.t_lengths, c.t_table, empty[0].clone(), c.k, c.v, ws, cu_new=cu)
    L.lf_attn_status(ws)
    assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip((c.k, c.v), before))
    one = [torch.ones(2, h, 64, dtype=c.k.dtype, device="cuda") for h in (4, 2, 2)]
    cu.copy_(torch.tensor([0, 1, 2, 2], dtype=torch.int32))
    L.lf_cache_append(p, None, *one, c.t_lengths, c.t_table, one[0].clone(), c.k, c.v, ws, cu_new=cu)
    L.lf_attn_status(ws)
    changed = (c.v.view(torch.int16) != before[1].view(torch.int16)).any(-1).any(1).nonzero().tolist()
    assert sorted(map(tuple, changed)) == sorted([(int(c.table[0, 1]), 0), (int(c.table[1, 0]), 15)])


def _in_a_new_thread(f):
    """f() in a host thread that has made no CUDA call."""
    import torch
    torch.cuda.synchronize()
    failed = []

    def work():
        try:
            f()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed


@pytest.mark.parametrize("path", PATHS)
def test_first_call_of_a_host_thread(path):
    import torch
    s = _setup(980, path, "bf16")
    stream = torch.cuda.current_stream()
    _call(s, stream)
    want = [x.clone() for x in s[4]]
    for x in s[4]:
        x.zero_()
    _in_a_new_thread(lambda: _call(s, stream))
    assert all(torch.equal(x, y) for x, y in zip(s[4], want))


def test_first_call_of_a_host_thread_of_the_other_operators():
    """The projections, the forward and the cross-attention encode tensor maps before anything else, too."""
    import torch
    B, n, H, dt = 1, 256, 4, torch.bfloat16
    stream = torch.cuda.current_stream()
    x = torch.randn(B, n, H * 64, device="cuda").to(dt)
    w, b = torch.randn(H * 64, H * 64, device="cuda").to(dt), torch.zeros(H * 64, device="cuda", dtype=dt)
    p = L.make_proj_params(B, n, H)
    ws = L.proj_workspace(p)
    outs = [torch.zeros(B, H, n, 64, dtype=dt, device="cuda") for _ in range(2)]
    y = [torch.zeros(B, n, H * 64, dtype=dt, device="cuda") for _ in range(2)]
    q = torch.randn(B, H, n, 64, device="cuda").to(dt)
    pa = L.make_params(B, H, n, 16, None, False, 0.0, L.LF_BF16, 0)
    wf, wb = L.workspace(pa), L.workspace(pa, True)
    mask = torch.ones(B, n, dtype=torch.int32, device="cuda")
    o, lse = [torch.zeros_like(q) for _ in range(2)], [torch.zeros(B, H, n, device="cuda") for _ in range(2)]
    grads = [[torch.zeros_like(q) for _ in range(6)] for _ in range(2)]
    pc = L.make_cross_params(B, H, n, n, L.LF_BF16)
    wc, oc = L.cross_workspace(pc), [torch.zeros_like(q) for _ in range(2)]
    calls = [
        lambda i: L.lf_attn_cross_fwd(pc, q, q, q, None, oc[i], None, wc, stream),
        lambda i: L.lf_proj_in(p, x, w, b, [outs[i]], ws, stream=stream),
        lambda i: L.lf_proj_out(p, q, w, b, y[i], ws, stream=stream),
        lambda i: L.lf_attn_fwd(pa, q, q, q, q, q, q, mask, o[i], lse[i], wf, stream),
        lambda i: L.lf_attn_bwd(pa, q, q, q, q, q, q, mask, o[0], lse[0], q, *grads[i], wb, stream),
    ]
    for f in calls:
        f(0)
        _in_a_new_thread(lambda: f(1))
    for a, c in [outs, y, o, lse, oc] + [list(z) for z in zip(*grads)]:
        assert torch.equal(a, c) and bool((a != 0).any() | (c == 0).all())
