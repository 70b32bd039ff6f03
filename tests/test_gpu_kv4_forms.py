"""Attention over the 4-bit cache, each kernel that a call can take by name: the plan is asked for and asserted, so that a
case cannot drift to another kernel when a rule moves. Bounds: the head of test_gpu_kv4.py."""

import numpy as np
import pytest
import torch

import compressed_sparse_kv_dsv4_b200 as dsv4
from compressed_sparse_kv_dsv4_b200 import _abi as A
from tests.parity import require_gpu
from tests.test_gpu_kv4 import ROOMY, check_attention, cu_of, fill_cache, i32, make_cache, rand_rows, roomy

pytestmark = pytest.mark.gpu


def plan_of(q, cu, start, c, max_new):
    return dsv4.kv4_attention_plan(dsv4.kv4_attention_args(q, cu, start, c, max_new=max_new))


SIXTEEN = [  # dim, query heads, key heads, new tokens, first positions, pages that the table has more
    (64, 4, 1, [5, 5], [0, 700], 1000),                       # twenty rows: a whole tile of sixteen and a quarter of one
    (64, 12, 2, [3, 0, 2], [62, 5, 900], 900),                # eighteen rows and twelve; a sequence that brings none
    (64, 24, 6, [5, 1, 3, 4, 2] * 2, [3, 64, 127, 128, 1000, 63, 0, 255, 256, 257], 50),
    (64, 20, 4, [8, 1], [20000, 9], 500),                     # forty rows, split over the card
    (64, 40, 4, [1] * 20, [i * 61 % 900 for i in range(20)], 80),
    (128, 4, 1, [4, 4], [0, 700], 1300),
    (128, 4, 1, [3, 4, 0, 2], [61, 125, 9, 509], 900),
    (128, 16, 1, [1, 1], [40000, 3], 1900),                   # sixteen heads to a key head, split over the card
    (128, 16, 4, [5] * 20, [i * 37 % 700 for i in range(20)], 60),
    (128, 12, 4, [3] * 20, [i * 61 % 900 for i in range(20)], 60),
    (128, 40, 4, [1] * 20, [i * 131 % 2000 for i in range(20)], 80),  # forty heads' ten to a key head
]


@pytest.mark.parametrize("case", SIXTEEN, ids=lambda c: f"D{c[0]}-{c[1]}over{c[2]}-{len(c[3])}x{max(c[3])}-{max(c[4])}")
@pytest.mark.parametrize("fill", [0xFF, 0xC8])
def test_tiles_of_sixteen_rows(case, fill):
    require_gpu()
    D, Hq, Hk, lens, starts, extra = case
    rng = np.random.default_rng(sum(starts) + Hq)
    c = make_cache(rng, lens, starts, Hk, D, fill=fill, extra_blocks=extra)
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, sum(lens), Hq, D, torch.bfloat16, 2)
    cu, start = cu_of(lens), i32(starts)
    plan = plan_of(q, cu, start, c, max(lens))
    assert (plan.form, plan.rows) == (A.KV4_STEP, 16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((sum(lens) + 5, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    out_, lse = dsv4.kv4_attention(q, cu, start, c, max_new=max(lens), out=out[:sum(lens)], with_lse=True, d_status=st)
    assert st.item() == 0 and torch.all(out[sum(lens):] == 3)
    check_attention(c, q, lens, starts, out_, lse)
    again = dsv4.kv4_attention(q, cu, start, c, max_new=max(lens), with_lse=True)
    assert torch.equal(out_, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("D,Hq,Hk,lens,starts,extra", [(64, 4, 1, [5, 5], [600, 130], 1000), (128, 4, 1, [4, 4], [600, 130], 1300)])
def test_tiles_of_sixteen_rows_keep_nan_and_bad_pages_apart(D, Hq, Hk, lens, starts, extra):
    require_gpu()
    rng = np.random.default_rng(51)
    c = make_cache(rng, lens, starts, Hk, D, extra_blocks=extra)
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, sum(lens), Hq, D, torch.bfloat16)
    cu, start, n = cu_of(lens), i32(starts), lens[0]
    plan = plan_of(q, cu, start, c, max(lens))
    assert (plan.form, plan.rows) == (A.KV4_STEP, 16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    run = lambda x=q, cache=c: dsv4.kv4_attention(x, cu, start, cache, max_new=max(lens), with_lse=True, d_status=st)
    clean, lse0 = run()
    for where in (5, 600, 602, 600 + n - 1):
        page, row = c.block_table[0, where // 256].item(), where % 256
        sees = torch.zeros(sum(lens), dtype=torch.bool, device="cuda")
        sees[:n] = torch.arange(n, device="cuda") + 600 >= where
        for scales, blk, cols in ((c.v_scales, 1, slice(32, 64)), (c.k_scales, 0, slice(None))):
            old = scales[page, 0, row, blk].clone()
            scales[page, 0, row, blk] = 255
            out, lse = run()
            scales[page, 0, row, blk] = old
            want = torch.zeros_like(out, dtype=torch.bool)
            want[:, :, cols] = sees[:, None, None]
            assert torch.equal(out.isnan(), want) and torch.equal(out[~want], clean[~want])
            assert torch.equal(lse.isnan(), want[..., 0] if scales is c.k_scales else torch.zeros_like(lse, dtype=torch.bool))
    for x in (float("nan"), float("inf"), float("-inf")):
        bad = q.clone()
        bad[2, 1, 7] = x
        out, lse = run(bad)
        assert out[2, 1].isnan().all() and lse[2, 1].isnan()
        out[2, 1], lse[2, 1] = clean[2, 1], lse0[2, 1]
        assert torch.equal(out, clean) and torch.equal(lse, lse0)
    assert st.item() == 0
    # a page of the first sequence that does not exist: its positions are left out, the second sequence is as it was
    table = c.block_table.clone()
    table[0, 1] = c.k_codes.shape[0]
    out, lse = run(q, dsv4.DeviceKv4Cache(c.k_codes, c.v_codes, c.k_scales, c.v_scales, table))
    assert st.item() == A.DEV_BAD_PAGE and torch.equal(out[n:], clean[n:]) and torch.equal(lse[n:], lse0[n:])
    # the same sequence without those positions, page 1's place taken by page 2
    short = dsv4.DeviceKv4Cache(c.k_codes, c.v_codes, c.k_scales, c.v_scales, c.block_table[:1][:, [0, 2]].contiguous())
    check_attention(short, q[:n], [n], [600 - 256], out[:n], lse[:n])
    gone = dsv4.DeviceKv4Cache(c.k_codes, c.v_codes, c.k_scales, c.v_scales, torch.full_like(table, -1))
    out, lse = run(bad, gone)
    assert torch.all(out == 0) and torch.all(lse == -np.inf)


@pytest.mark.parametrize("extra,splits", [(0, 2), (30, 8)])
def test_a_prompts_partial_wave_at_128_channels(extra, splits):
    """More blocks than SMs: the keys of the last, partial wave's blocks are shared out."""
    require_gpu()
    if torch.cuda.get_device_properties(0).multi_processor_count != 148:
        pytest.skip("the wave is counted for 148 SMs")
    rng = np.random.default_rng(52)
    lens, starts = [300, 280], [2100, 0]
    c = make_cache(rng, lens, starts, 20, 128, fill=0xFF, extra_blocks=extra)
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, sum(lens), 80, 128, torch.bfloat16)
    cu, start = cu_of(lens), i32(starts)
    plan = plan_of(q, cu, start, c, 300)
    assert (plan.form, plan.rows, plan.units, plan.shared, plan.splits) == (A.KV4_PROMPT, 256, 200, 52, splits)
    for max_new in (300, 100):
        out, lse = dsv4.kv4_attention(q, cu, start, c, max_new=max_new, with_lse=True)
        check_attention(c, q, lens, starts, out, lse, sample=8, ctx=f"max_new {max_new}")


def test_the_wide_tables_cases_take_tensor_scores():
    """The cases of test_gpu_kv4.py that are there for the form with scores on the tensor cores do reach it (one hint of one of them
    is a prompt's), and codes 16 bytes off a multiple of 32 do not."""
    require_gpu()
    for Hq, Hk, lens, starts in ROOMY:
        c = roomy(np.random.default_rng(1), lens, starts, Hk)
        q = torch.zeros((sum(lens), Hq, 128), dtype=torch.bfloat16, device="cuda")
        for max_new in {1, max(lens)} - {6}:
            plan = plan_of(q, cu_of(lens), i32(starts), c, max_new)
            assert (plan.form, plan.rows) == (A.KV4_STEP_TENSOR, 8), (Hq, Hk, max_new)
    raw = torch.zeros(c.k_codes.numel() + 64, dtype=torch.uint8, device="cuda")
    at = (16 - raw.data_ptr()) % 32
    c = dsv4.DeviceKv4Cache(raw[at:at + c.k_codes.numel()].view(c.k_codes.shape), c.v_codes, c.k_scales, c.v_scales, c.block_table)
    assert plan_of(q, cu_of(lens), i32(starts), c, 1).form == A.KV4_STEP


def test_one_batch_in_every_form():
    """The same tokens over the same cache through each kernel, by the width of the table and the hint alone."""
    require_gpu()
    rng = np.random.default_rng(53)
    lens, starts = [4, 3], [600, 130]
    c = make_cache(rng, lens, starts, 1, 128, extra_blocks=1300)
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, sum(lens), 4, 128, torch.bfloat16)
    cu, start = cu_of(lens), i32(starts)
    seen = set()
    for blocks, max_new in ((5, 1), (5, 4), (1303, 1), (1303, 4), (1303, 500)):
        x = dsv4.DeviceKv4Cache(c.k_codes, c.v_codes, c.k_scales, c.v_scales, c.block_table[:, :blocks].contiguous())
        plan = plan_of(q, cu, start, x, max_new)
        seen.add((plan.form, plan.rows))
        out, lse = dsv4.kv4_attention(q, cu, start, x, max_new=max_new, with_lse=True)
        check_attention(x, q, lens, starts, out, lse)
    assert {(A.KV4_STEP, 8), (A.KV4_STEP, 16), (A.KV4_STEP_TENSOR, 8)} <= seen


def test_one_workspace_serves_calls_of_all_sizes():
    """Sized once for the largest, it is enough for smaller calls that split more, and gives the bits that a call's own does."""
    require_gpu()
    rng = np.random.default_rng(54)
    lens, starts = [700, 4, 1], [2000, 600, 9000]
    c = make_cache(rng, lens, starts, 2, 128, extra_blocks=20)
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, sum(lens), 8, 128, torch.bfloat16)
    ws = dsv4.kv4_attention_workspace(q, cu_of(lens), c, max_new=700, smaller=True)
    one = lambda s: dsv4.DeviceKv4Cache(c.k_codes, c.v_codes, c.k_scales, c.v_scales, c.block_table[s:s + 1])
    at = np.concatenate([[0], np.cumsum(lens)])
    forms = set()
    for s, n in ((0, 700), (0, 40), (1, 4), (2, 1)):
        a, cu, start = q[at[s]:at[s] + n], cu_of([n]), i32([starts[s]])
        forms.add(plan_of(a, cu, start, one(s), n).form)
        want = dsv4.kv4_attention(a, cu, start, one(s), max_new=n, with_lse=True)
        got = dsv4.kv4_attention(a, cu, start, one(s), max_new=n, with_lse=True, workspace=ws)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert forms == {A.KV4_STEP, A.KV4_PROMPT}
    dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=700, workspace=ws)
