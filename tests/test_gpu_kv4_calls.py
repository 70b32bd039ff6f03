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
from tests.test_gpu_kv4 import (BF16, NORM, U, cache_rows, cu_of, dev, fill_cache, i32, make_cache, pair_bound, positions,
                                rand_rows)

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


# ---------------------------------------------------------------- rows without a finite score

FORMS = [  # dim, query heads, new tokens, first position, more pages than the context has: a step, drafts, a prompt
    (64, 4, 1, 700, 0),
    (64, 4, 4, 700, 700),
    (128, 8, 1, 700, 0),
    (128, 8, 1, 700, 1000),
    (128, 8, 1, 30000, 0),
    (128, 8, 1, 30000, 1000),
    (128, 2, 4, 700, 1000),
    (128, 4, 300, 700, 0),
    (128, 4, 300, 9000, 0),
    (64, 4, 300, 700, 0),
    (64, 4, 300, 9000, 0),
]


@pytest.mark.parametrize("D,Hq,new,start,extra", FORMS)
def test_rows_without_a_finite_score(D, Hq, new, start, extra):
    """NaN wherever such a row sees a position, and zero and lse -inf only where it sees none, in every form."""
    require_gpu()
    rng = np.random.default_rng(D + new)
    lens, starts = [new], [start]
    c = make_cache(rng, lens, starts, 1, D, extra_blocks=extra)
    n = start + new
    k = torch.randn((n, 1, D), device="cuda")
    k[:, 0, 5], k[:, 0, 40] = 3.0, 49152.0  # channels whose products have one sign
    v = torch.randn((n, 1, D), device="cuda")
    dsv4.kv4_append(k, v, cu_of([n]), i32([0]), c, rope_dims=0)
    q, _ = rand_rows(rng, new, Hq, D, torch.bfloat16)
    q[..., 40] = 0
    run = lambda x, cache=c: dsv4.kv4_attention(x, cu_of(lens), i32(starts), cache, max_new=new, with_lse=True)
    clean, lse0 = run(q)
    gone = dsv4.DeviceKv4Cache(c.k_codes, c.v_codes, c.k_scales, c.v_scales, torch.full_like(c.block_table, -1))
    at = new // 2
    for channel, value in ((5, float("-inf")), (5, float("inf")), (5, float("nan")), (40, -3e38), (40, 3e38)):
        bad = q.clone()
        bad[at, 1] = 0
        bad[at, 1, channel] = value
        out, lse = run(bad)
        assert out[at, 1].isnan().all() and lse[at, 1].isnan(), (channel, value)
        out[at, 1], lse[at, 1] = clean[at, 1], lse0[at, 1]
        assert torch.equal(out, clean) and torch.equal(lse, lse0)
        out, lse = run(bad, gone)
        assert torch.all(out == 0) and torch.all(lse == -np.inf), (channel, value)


@pytest.mark.parametrize("D,Hq,new,start,extra", FORMS)
def test_scores_below_float32_beside_others(D, Hq, new, start, extra):
    """Positions whose scores leave float32's range downwards weigh nothing; the others decide."""
    require_gpu()
    rng = np.random.default_rng(D + new + 1)
    c = make_cache(rng, [new], [start], 1, D, extra_blocks=extra)
    n = start + new
    k = torch.zeros((n, 1, D), device="cuda")
    seen = [3, 131, n - new]  # the only ones in range
    k[:, 0, 40] = 49152.0
    k[seen, 0, 40] = 0
    v = torch.randn((n, 1, D), device="cuda")
    dsv4.kv4_append(k, v, cu_of([n]), i32([0]), c, rope_dims=0)
    q = torch.zeros((new, Hq, D), device="cuda", dtype=torch.bfloat16)
    q[..., 40] = -3e38
    out, lse = dsv4.kv4_attention(q, cu_of([new]), i32([start]), c, max_new=new, with_lse=True)
    _, vv = cache_rows(c, 0, n)
    want = vv[seen].mean(0)[0]
    # three equal weights, powers of two before they are divided by their sum
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= (BF16 + 8 * U) * np.abs(vv[seen]).mean(0)[0])
    assert np.all(np.abs(lse.double().cpu().numpy() - np.log(3.0)) <= 2.0 ** -20)



# ---------------------------------------------------------------- rows of q with channels far above the others

@pytest.mark.parametrize("extra", [0, 1000])  # more pages than the context has: both forms of a step
@pytest.mark.parametrize("start", [700, 20000])
@pytest.mark.parametrize("power", [12, 14, 18, 30, 60])
def test_small_channels_beside_a_large_one(power, start, extra):
    """Channels that are 2^-12 to 2^-60 of the row's largest decide where the keys are zero in that one. A score may be off by 2^-14
    (of log2) more than at the head of test_gpu_kv4.py: where the form with scores on the tensor cores (wide tables) leaves out
    more than that of a row, it adds it.

    The form for narrow tables holds q in fp16, the row's largest element at 2^14 or more. Below fp16's normal numbers the step is 2^-24:
    an element is off by at most half of it, 2^-25, which is 2^-39 of the largest, and a score by scale * 2^-39 * max |q| * sum |k|.

    Scores off by eps change each weight by a factor within exp(+-2 eps): the output by (exp(2 eps) - 1) sum p |v|. Where eps is not small
    (2^60 in the narrow form) that says nothing, but any weights make a mixture of the values: 2 max |v|."""
    require_gpu()
    rng = np.random.default_rng(power + extra)
    D, Hq, n = 128, 8, start + 1
    c = make_cache(rng, [1], [start], 1, D, extra_blocks=extra)
    large = [5, 37, 77, 127, 5, 64, 0]  # of each row but the last, which has none
    k, v = (torch.randn((n, 1, D), device="cuda") for _ in range(2))
    k[..., large] = 0
    k[1, 0, 77] = 0.5 * 2.0 ** -power  # (a position where one of them counts as much as the others)
    dsv4.kv4_append(k, v, cu_of([n]), i32([0]), c, rope_dims=0)
    q = torch.randn((1, Hq, D), device="cuda")
    for r, ch in enumerate(large):
        q[0, r, ch] = 2.0 ** power
    q = q.bfloat16()
    kk, vv = cache_rows(c, 0, n)
    for scale in (D ** -0.5, 1.0):
        out, lse = dsv4.kv4_attention(q, cu_of([1]), i32([start]), c, max_new=1, softmax_scale=scale, with_lse=True)
        want, wl, mag, top = K.attention(q.double().cpu().numpy(), kk, vv, start, scale)
        eps = 2 * (D + 4) * U * top + 2.0 ** -21 + 2 * U * 1.4427 * (top + np.abs(wl)) + 2.0 ** -14 * np.log(2)
        if extra == 0:
            eps = eps + scale * 2.0 ** -39 * q.double().abs().amax(-1).cpu().numpy() * np.abs(kk).sum(-1).max()
        moved = np.minimum(np.expm1(2 * np.minimum(eps, 100.0))[..., None] * mag, 2 * np.abs(vv).max(0))
        limit = 2.0 ** -11 * mag + moved + 2.0 ** -32 * np.abs(vv).sum(0) + BF16 * np.abs(want)
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= limit)
        assert np.all(np.abs(lse.double().cpu().numpy() - wl) <= eps + 4 * U * np.abs(wl) + 2.0 ** -21)


@pytest.mark.parametrize("fill", [0xFF, 0xC8])
@pytest.mark.parametrize("Hq,lens,starts", [(4, [2, 1], [250, 700]), (8, [1, 1], [0, 127]), (2, [3, 0, 4], [126, 5, 509])])
def test_small_channels_under_masks_and_missing_pages(Hq, lens, starts, fill):
    """The same beside positions that are masked, hold no values yet (NaN, or scales beyond fp16) or lie on a page that does not exist."""
    require_gpu()
    rng = np.random.default_rng(Hq + fill)
    D = 128
    c = make_cache(rng, lens, starts, 1, D, fill=fill, extra_blocks=700)
    tot = [n + s for n, s in zip(lens, starts)]
    k, v = (torch.randn((sum(tot), 1, D), device="cuda") for _ in range(2))
    k[..., [7, 90]] = 0
    dsv4.kv4_append(k, v, cu_of(tot), i32([0] * len(tot)), c, rope_dims=0)
    q = torch.randn((sum(lens), Hq, D), device="cuda")
    q[::2, :, 7] = 2.0 ** 18
    q[1::2, 1, 90] = -2.0 ** 20
    q = q.bfloat16()
    rows = [cache_rows(c, s, n) for s, n in enumerate(tot)]
    last = len(lens) - 1
    for gone in (False, True):
        table = c.block_table.clone()
        if gone:
            table[last, 0] = -1
        cache = dsv4.DeviceKv4Cache(c.k_codes, c.v_codes, c.k_scales, c.v_scales, table)
        out, lse = dsv4.kv4_attention(q, cu_of(lens), i32(starts), cache, max_new=max(lens), softmax_scale=1.0, with_lse=True)
        at = 0
        for s, (n, first) in enumerate(zip(lens, starts)):
            for i in range(n):
                keep = [j for j in range(first + i + 1) if not (gone and s == last and j < 256)]
                got, gl = out[at + i].double().cpu().numpy(), lse[at + i].double().cpu().numpy()
                if not keep:
                    assert np.all(got == 0) and np.all(gl == -np.inf)
                    continue
                kk, vv = rows[s][0][keep], rows[s][1][keep]
                want, wl, mag, top = K.attention(q[at + i:at + i + 1].double().cpu().numpy(), kk, vv, len(keep) - 1, 1.0)
                eps = 2 * (D + 4) * U * top + 2.0 ** -21 + 2 * U * 1.4427 * (top + np.abs(wl)) + 2.0 ** -14 * np.log(2)
                limit = (2.0 ** -11 + 2 * eps[..., None]) * mag + 2.0 ** -32 * np.abs(vv).sum(0) + BF16 * np.abs(want)
                assert np.all(np.abs(got - want[0]) <= limit[0])
                assert np.all(np.abs(gl - wl[0]) <= (eps + 4 * U * np.abs(wl) + 2.0 ** -21)[0])
            at += n


# ---------------------------------------------------------------- angles of far positions

@pytest.mark.parametrize("base", [2.0 ** -16, 0.01, 10000.0])
def test_rotation_at_the_last_positions(base):
    """Positions up to 2^31 + 4, and a base that makes their angles 2^47, where only the pair's length is left to check.

    In half steps of float64, 2^-53 relative: theta_1 comes from a pow (2, a whole step); each squaring doubles what there is and adds 1, so
    theta_1^(2^k) is off by 3 2^k, and the products of those that make up theta_1^i by 3 i and 5 of their own; the position adds 1, the
    oracle's pow and product 3: 3 i + 9 of the angle, and so much of |a| + |b| of both members of pair i."""
    require_gpu()
    rng = np.random.default_rng(61)
    D, n = 64, 6
    starts = [2 ** 31 - 1, 2 ** 30 + 12345, 77]
    lens = [n] * 3
    q, qv = rand_rows(rng, 3 * n, 2, D, torch.float32)
    out, _ = dsv4.qk_norm_rope(q, None, cu_of(lens), i32(starts), rope_dims=D, rope_base=base)
    pos = positions(lens, starts)
    want = K.norm_rotate(qv, None, 0.0, pos, D, float(np.float32(base)))
    angle = pos[:, None] * float(np.float32(base)) ** (-2.0 * np.arange(D // 2) / D)
    eps = 24 * U + np.repeat((3 * np.arange(D // 2) + 9) * 2.0 ** -53 * angle, 2, -1)[:, None]
    limit = pair_bound(want, D, 1.0) * eps
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= limit + 1e-30)
    assert np.allclose(np.hypot(out.cpu().numpy()[..., ::2], out.cpu().numpy()[..., 1::2]), np.hypot(qv[..., ::2], qv[..., 1::2]), rtol=1e-6)


# ---------------------------------------------------------------- the norm's bound, for the kernel's own order of sums

@pytest.mark.parametrize("case", NORM, ids=lambda c: f"D{c[0]}-{c[1]}and{c[2]}-{c[6]}-{len(c[3])}")
def test_norm_rope_within_its_own_roundings(case):
    """float32 outputs, in units of u = 2^-24. Squares are rounded (1) and summed at a depth of 6 (64 channels) to 10 (512), the mean
    is exact, eps adds 1: 12, halved by the root, and rsqrtf's two steps 4: 10. The products with it and with gamma: 12 on each
    channel. Sine and cosine are float64, rounded once (1), of an angle whose float64 error is below 1 at these positions (2^20 of it times
    9 2^-53 for the fast pairs); product 1 and sum 1: 16 (|a| + |b|) on each of a pair. Without gamma nothing but the rotation: 4, and 0."""
    require_gpu()
    D, Hq, Hk, lens, starts, rope, din, _, extra = case
    rng = np.random.default_rng(D + Hq + 1)
    T = sum(lens)
    q, qv = rand_rows(rng, T, max(Hq, 1), D, {"f32": torch.float32, "bf16": torch.bfloat16}[din], extra)
    g = 1 + 0.3 * rng.standard_normal(D).astype(np.float32)
    for gamma, turned, kept in ((g, 16, 12), (None, 4, 0)):
        got, _ = dsv4.qk_norm_rope(q, None, cu_of(lens), i32(starts), gamma_q=None if gamma is None else dev(gamma),
                                   rope_dims=rope, out_dtype=torch.float32)
        want = K.norm_rotate(qv, gamma, 1e-6, positions(lens, starts), rope, 10000.0)
        limit = pair_bound(want, rope, turned * U)
        limit[..., :D - rope] = kept * U * np.abs(want[..., :D - rope])
        err = np.abs(got.double().cpu().numpy() - want)
        assert np.all(err <= limit + 1e-30), (err / (limit + 1e-30)).max()


@pytest.mark.parametrize("D,rope", [(64, 64), (128, 64), (128, 20), (512, 64)])
@pytest.mark.parametrize("norm", [False, True])
def test_rotation_rounds_each_product(D, rope, norm):
    """The float32 steps are those of a plain float32 program, so that a key next to a border of its 4-bit codes gets the same
    code: the outputs agree to the last bit, but where a sine or cosine lies within its angle's float64 error (12 2^-53 of 4096 turns at the
    most, 5e-12) of a border between float32 values (6e-8 apart): one in ten thousand. Products contracted into their sums differ
    in a quarter of the rotated channels."""
    require_gpu()
    x = torch.randn((4096, 4, D), device="cuda", generator=torch.Generator("cuda").manual_seed(D + rope))
    g = (1 + 0.2 * torch.randn(D, device="cuda", generator=torch.Generator("cuda").manual_seed(1))) if norm else None
    got, _ = dsv4.qk_norm_rope(x, None, cu_of([4096]), i32([0]), gamma_q=g, rope_dims=rope, eps=operators.EPS)
    pos = torch.arange(4096, device="cuda")
    want = x
    if norm and D <= 128:  # (the plain program's row sums are those of 64 and 128 channels)
        want = operators._norm_rotate(x, g, pos, 0, 1e4)
    elif norm:
        want, _ = dsv4.qk_norm_rope(x, None, cu_of([4096]), i32([0]), gamma_q=g, rope_dims=0, eps=operators.EPS)
    theta = 1e4 ** (-2.0 / rope * torch.arange(rope // 2, dtype=torch.float64, device="cuda"))
    angle = pos.double()[:, None, None] * theta
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    a, b = want[..., D - rope::2], want[..., D - rope + 1::2]
    want = torch.cat([want[..., :D - rope], torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)], -1)
    assert torch.equal(got[..., :D - rope], want[..., :D - rope])
    assert (got != want).double().mean().item() < 1e-3
