"""The 4-bit key/value cache's calls beside the library's others, and at their edges.

Bounds are those at the head of test_gpu_kv4.py where a test does not derive its own.
"""

import numpy as np
import pytest
import torch

import compressed_sparse_kv_dsv4_b200 as dsv4
import synthetic as W
from tests.parity import require_gpu
from tests.test_gpu_kv4 import cu_of, fill_cache, i32, make_cache, rand_rows

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
