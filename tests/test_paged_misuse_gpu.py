"""GPU tests of what the calls of the paged cache record about their inputs."""
import numpy as np
import pytest

from sparse_sliding_window_b200 import lf_attn as L
from tests.test_paged_gpu import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu,tokens,where", [
    ([0, 5, 3, 8], 8, "sequence 1"),          # sequence 1 ends before it begins; every token lies in one of the others
    ([0, 2, 3, 9], 5, "sequence 2"),          # ends behind the tokens that there are
    ([1, 2, 3, 5], 5, "sequence 0"),          # begins behind the first token
    ([0, 4, 4, 2 ** 31 - 1], 5, "sequence 2"),
    ([-3, 2, 3, 5], 5, "sequence 0"),
])
def test_append_records_offsets_that_are_none(cu, tokens, where):
    import torch
    c = Cache(93, "f32", 3, 1, 16, [20, 30, 25])
    p = c.params(1)
    ws = L.paged_workspace(p)
    k = torch.ones(tokens, 1, 64, device="cuda")
    pools = torch.zeros_like(c.k), torch.zeros_like(c.v)
    t_cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    L.lf_cache_append(p, None, None, k, k, c.t_lengths, c.t_table, None, *pools, ws, cu_new=t_cu)
    with pytest.raises(L.LfError) as e:
        L.lf_attn_status(ws)
    assert e.value.code == L.LF_ERR_DEVICE_INPUT and "cu_new" in str(e.value) and where in str(e.value)
    # nothing but rows of the sequences, and not more rows than tokens
    rows = torch.zeros(c.num, 16, dtype=torch.bool, device="cuda")
    for b, n in enumerate(c.lengths):
        for j in range(int(n)):
            rows[int(c.table[b, j // 16]), j % 16] = True
    for x in pools:
        written = (x != 0).any(-1)[:, 0]
        assert not (written & ~rows).any() and int(written.sum()) <= tokens
    # offsets that are right leave no word, with empty sequences and tokens behind the last one
    for good in ([0, 2, 2, 5], [0, 0, 0, 0], [0, 1, 2, 3]):
        t_cu.copy_(torch.tensor(good, dtype=torch.int32))
        L.lf_cache_append(p, None, None, k, k, c.t_lengths, c.t_table, None, *pools, ws, cu_new=t_cu)
    L.lf_attn_status(ws)


def test_append_records_offsets_of_many_idle_sequences():
    """More sequences than a block has threads, one token, the offsets wrong far behind it."""
    import torch
    B = 3000
    c = Cache(94, "f32", B, 1, 16, [1] + [0] * (B - 1))
    p = c.params(1)
    ws = L.paged_workspace(p)
    k = torch.ones(1, 1, 64, device="cuda")
    cu = torch.ones(B + 1, dtype=torch.int32, device="cuda")
    cu[0] = 0
    L.lf_cache_append(p, None, None, k, k, c.t_lengths, c.t_table, None, c.k, c.v, ws, cu_new=cu)
    L.lf_attn_status(ws)
    cu[2900] = 0
    L.lf_cache_append(p, None, None, k, k, c.t_lengths, c.t_table, None, c.k, c.v, ws, cu_new=cu)
    with pytest.raises(L.LfError) as e:
        L.lf_attn_status(ws)
    assert "sequence 2899" in str(e.value)


def test_mask_errors_of_large_batches_keep_their_text():
    """The status details of the paged calls do not overlap those of the mask pass, whatever the batch."""
    import torch
    B = 2000001
    p = L.make_params(B, 1, 2, 0, None, False, 0.0, L.LF_BF16, 1)
    ws = L.workspace(p)
    mask = torch.ones(B, 2, dtype=torch.int32, device="cuda")
    mask[B - 1] = 2                                     # two global tokens, and one is allowed
    counts = torch.empty(B, 1, dtype=torch.int64, device="cuda")
    L.lf_attn_count_pairs(p, mask, counts, ws)
    with pytest.raises(L.LfError) as e:
        L.lf_attn_status(ws)
    assert "sequence %d has more global tokens" % (B - 1) in str(e.value)


def test_too_many_selected_rows_are_reported_as_that():
    import torch
    B, n, H = 2, 8, 4
    p = L.make_proj_params(B, n, H)
    ws = L.proj_workspace(p, 2)
    dt = torch.bfloat16
    x, w, b = (torch.zeros(*s, dtype=dt, device="cuda") for s in ((B, n, H * 64), (H * 64, H * 64), (H * 64,)))
    mask = torch.ones(B, n, dtype=torch.int32, device="cuda")
    mask[1, :3] = 2
    L.lf_proj_in(p, x, w, b, [torch.zeros(B, H, n, 64, dtype=dt, device="cuda")], ws, rows_mask=mask, rows_code=2, max_rows=2)
    with pytest.raises(L.LfError) as e:
        L.lf_attn_status(ws)
    assert e.value.code == L.LF_ERR_DEVICE_INPUT and "sequence 1 has more selected rows" in str(e.value)
