"""The 4-bit key/value cache's calls beside the library's others, and at their edges.

Bounds are those at the head of test_gpu_kv4.py where a test does not derive its own.
"""

import numpy as np
import pytest
import torch

import compressed_sparse_kv_dsv4_b200 as dsv4
import oracle.kv4_oracle as K
import perf.operators as operators
import synthetic as W
from tests.parity import require_gpu
from tests.test_gpu_kv4 import (BF16, cu_of, dev, fill_cache, i32, make_cache, pair_bound, positions, rand_rows)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- the next call on the stream

def decode_case(B):
    """A dense layer's attention step over B sequences: (layer, queries' shape, arguments)."""
    spec = W.C128_SPEC
    la = W.make_layer(spec, B, 20, 5)
    dl = dsv4.DeviceLayer.from_arrays(la)
    pos = i32([128 * 18 + 7 * s for s in range(B)])
    args = dict(q_dtype="bf16", out_dtype="bf16", n_entries=i32([18] * B), rope_dims=spec.rope_dims)
    return dl, pos, spec.H, spec.D, args


def test_norms_feed_the_next_call():
    """The attention's first kernel takes the queries before it waits for the kernel before it: the norm's last rows,
    of many, must be there when the next call begins."""
    require_gpu()
    B, T = 4, 4096
    dl, pos, H, D, args = decode_case(B)
    q = torch.randn((T, H, D), device="cuda", generator=torch.Generator("cuda").manual_seed(3)).bfloat16()
    g = torch.ones(D, device="cuda")
    out = torch.empty_like(q)
    cu, start = cu_of([T]), i32([0])
    dsv4.qk_norm_rope(q, None, cu, start, gamma_q=g, q_out=out)
    torch.cuda.synchronize()
    want = dsv4.sparse_mqa_decode(out[-B:], pos, dl.cache, dl.ring, **args)
    torch.cuda.synchronize()
    for _ in range(10):
        out.zero_()
        torch.cuda.synchronize()
        dsv4.qk_norm_rope(q, None, cu, start, gamma_q=g, q_out=out)
        got = dsv4.sparse_mqa_decode(out[-B:], pos, dl.cache, dl.ring, **args)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("new,D", [(1, 64), (1, 128), (300, 128)])
def test_a_workspace_passes_to_the_next_call(new, D):
    """The attention's first kernel writes its workspace before it waits: the call before has read its parts."""
    require_gpu()
    rng = np.random.default_rng(41)
    B = 4
    dl, pos, H, Dq, args = decode_case(B)
    lens, starts = [new] * 2, [30000, 20000]
    c = make_cache(rng, lens, starts, 4, D)
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, 2 * new, 16, D, torch.bfloat16)
    dq = torch.randn((B, H, Dq), device="cuda").bfloat16()
    cu, start = cu_of(lens), i32(starts)
    want, lse0 = dsv4.kv4_attention(q, cu, start, c, max_new=new, with_lse=True)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(want), torch.empty_like(lse0)
    step = dsv4.sparse_mqa_decode(dq, pos, dl.cache, dl.ring, workspace=ws, **args)
    torch.cuda.synchronize()
    for _ in range(10):
        dsv4.kv4_attention(q, cu, start, c, max_new=new, out=out, lse=lse, workspace=ws)
        got = dsv4.sparse_mqa_decode(dq, pos, dl.cache, dl.ring, workspace=ws, **args)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, lse0) and torch.equal(got, step)


# ---------------------------------------------------------------- the append's queries

@pytest.mark.parametrize("din", ["f32", "bf16"])
@pytest.mark.parametrize("dout", ["f32", "bf16"])
@pytest.mark.parametrize("D,Hq,Hk,rope,extra", [(64, 7, 1, 64, 0), (128, 12, 4, 44, 4)])
def test_append_queries_in_both_types(D, Hq, Hk, rope, extra, din, dout):
    require_gpu()
    rng = np.random.default_rng(D + Hq)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}
    lens, starts = [33, 0, 5], [250, 9, 100003]
    c = make_cache(rng, lens, starts, Hk, D)
    T = sum(lens)
    q, qv = rand_rows(rng, T, Hq, D, dt[din], extra)
    k, _ = rand_rows(rng, T, Hk, D, dt[din], extra)
    g = 1 + 0.3 * rng.standard_normal(D).astype(np.float32)
    for gamma in (g, None):
        out = torch.full((T + 3, Hq, D), 7.0, dtype=dt[dout], device="cuda")
        got, ks, _ = dsv4.kv4_append(k, k, cu_of(lens), i32(starts), c, q=q, gamma_q=None if gamma is None else dev(g),
                                     q_out=out[:T], rope_dims=rope, with_stored=True)
        assert got.data_ptr() == out.data_ptr() and torch.all(out[T:] == 7) and ks.dtype == torch.bfloat16
        want = K.norm_rotate(qv, gamma, 1e-6, positions(lens, starts), rope, 10000.0)
        limit = pair_bound(want, rope) + (BF16 * np.abs(want) if dout == "bf16" else 0) + 1e-30
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= limit)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_measured_append_returns_what_its_plain_form_does(dtype, monkeypatch):
    """perf/operators.py counts the queries' bytes in their own type: its calls ask for that type."""
    require_gpu()
    case = dict(op="append", batch=3, new=9, ctx=300, ragged=True, heads=4, kv_heads=2, dim=64, rope=32, dtype=dtype)
    kinds = []
    for own in (False, True):
        monkeypatch.setattr(operators, "own", own)
        got = operators.run(operators.prepare(case, 1))
        kinds.append({n: (t.dtype, tuple(t.shape)) for n, t in got.items()})
    assert kinds[0] == kinds[1]
