"""The 4-bit key/value cache on the GPU against the float64 oracle.

Bounds, with u = 2^-24 (half a float32 step, relative):
- norm and rotation: a row's mean square is at most 8 fused and 9 shuffled sums (17u), its inverse
  root halves that (9u) and adds 4u of its own and 2u around it; gamma and the product 2u: 17u on
  each of the pair (a, b). The reduced angle is within pi, so its rounding is 2u absolute, and
  cos and sin add 2u each, the rotation's products and sum 3u: 24u (|a| + |b|) in all. bf16 output: half
  a step, 2^-8 relative, more.
- rounding to 4 bits: a stored value is the rounding of some number within the norm's bound of the
  oracle's, under a scale that such a number's amax has: rounding is monotone, so it lies between the
  roundings of the two ends under its own scale byte.
- attention: with S = the largest scale * sum_d |q_d k_jd| of a row, a score is off by at most
  2 (D + 4) u S (sums of D terms in float32 whose adder may drop bits, twice the rounding), the weights by that
  and 2^-21 (the hardware's 2^x, the exponent's own rounding of at most 2u (S + |lse|) log2 e),
  and each weight is rounded to fp16 (2^-11 relative; below fp16's normal numbers, where the step is
  2^-24, by 2^-25 absolute; a row's largest weight is held as 2^7 or more, so by 2^-32 of it, which
  is at most the sum of all). The output: (2^-11 + 2 eps) sum_j p_j |v_j| + 2^-32 sum_j |v_j| + 2^-8 |o|,
  lse: eps + 4u |lse| + 2^-21.
"""

import ctypes as C

import numpy as np
import pytest
import torch

import compressed_sparse_kv_dsv4_b200 as dsv4
from compressed_sparse_kv_dsv4_b200 import _abi as A
import oracle.kv4_oracle as K
from tests.parity import require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16 = 2.0 ** -8
PAGE = 256


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cu_of(lens):
    return i32(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))


def rand_rows(rng, T, H, D, dtype, extra=0):
    """[T, H, D] rows, the token axis strided by `extra` more heads; (tensor, float64 values)."""
    t = torch.from_numpy(rng.standard_normal((T, H + extra, D)).astype(np.float32)).to(dtype).cuda()[:, extra // 2:extra // 2 + H]
    return t, t.double().cpu().numpy()


def pair_bound(y, rope, eps=24 * U):
    """eps (|a| + |b|) of each rotated pair (of both its members), eps |y| elsewhere."""
    b = eps * np.abs(y)
    if rope:
        D = y.shape[-1]
        h = np.hypot(y[..., D - rope::2], y[..., D - rope + 1::2]) * np.sqrt(2)
        b[..., D - rope::2] = b[..., D - rope + 1::2] = eps * h
    return b


def positions(lens, starts):
    return np.concatenate([s + np.arange(n) for n, s in zip(lens, starts)] + [np.zeros(0)]).astype(np.int64)


# ---------------------------------------------------------------- norm and rotation

NORM = [  # dim, q heads, k heads, lengths, starts, rope dims, input, output, extra heads between tokens
    (128, 64, 8, [1], [8191], 64, "bf16", "bf16", 0),
    (64, 9, 3, [1, 0, 5, 33], [0, 7, 1000003, 255], 64, "f32", "f32", 0),
    (128, 5, 1, [17, 2], [3, 0], 128, "bf16", "f32", 4),
    (256, 3, 2, [3, 4, 1], [9, 0, 77], 64, "f32", "bf16", 2),
    (512, 2, 7, [2, 9], [5, 1 << 20], 64, "bf16", "bf16", 0),
    (64, 0, 1, [300], [40], 16, "bf16", "bf16", 2),
    (128, 3, 0, [7], [1], 0, "f32", "f32", 0),
    (128, 16, 2, [1] * 70, list(range(70)), 64, "bf16", "bf16", 0),
    (128, 6, 2, [50, 3], [17, 70000], 20, "f32", "bf16", 0),   # rotated channels that end inside a lane's eight
    (64, 11, 1, [9], [1], 62, "bf16", "f32", 0),
    (512, 1, 1, [33], [5], 2, "f32", "f32", 0),
    (64, 700, 300, [5], [3], 64, "bf16", "bf16", 0),
]


@pytest.mark.parametrize("case", NORM, ids=lambda c: f"D{c[0]}-{c[1]}and{c[2]}-{c[6]}-{len(c[3])}")
def test_norm_rope(case):
    require_gpu()
    D, Hq, Hk, lens, starts, rope, din, dout, extra = case
    rng = np.random.default_rng(D + Hq)
    T, dt = sum(lens), {"f32": torch.float32, "bf16": torch.bfloat16}
    q, qv = rand_rows(rng, T, max(Hq, 1), D, dt[din], extra)
    k, kv = rand_rows(rng, T, max(Hk, 1), D, dt[din], extra)
    gq, gk = (1 + 0.3 * rng.standard_normal(D).astype(np.float32) for _ in range(2))
    for norm in (True, False):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        oq, ok = dsv4.qk_norm_rope(q if Hq else None, k if Hk else None, cu_of(lens), i32(starts),
                                   gamma_q=dev(gq) if norm else None, gamma_k=dev(gk) if norm else None, rope_dims=rope,
                                   out_dtype=dt[dout], d_status=st)
        assert st.item() == 0
        for got, x, g, H in ((oq, qv, gq, Hq), (ok, kv, gk, Hk)):
            if not H:
                assert got is None
                continue
            want = K.norm_rotate(x, g if norm else None, 1e-6, positions(lens, starts), rope, 10000.0)
            limit = pair_bound(want, rope) + (BF16 * np.abs(want) if dout == "bf16" else 0) + 1e-30
            assert got.dtype == dt[dout] and got.shape == x.shape
            assert np.all(np.abs(got.double().cpu().numpy() - want) <= limit)


def test_norm_in_place_and_behind_the_last_token():
    require_gpu()
    rng = np.random.default_rng(8)
    q, qv = rand_rows(rng, 9, 4, 128, torch.bfloat16)
    out = torch.full((9, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    cu, start = i32([0, 2, 6]), i32([4, 0])  # three rows behind the last sequence
    dsv4.qk_norm_rope(q, None, cu, start, q_out=out)
    assert torch.all(out[6:] == 7)
    dsv4.qk_norm_rope(q, None, cu, start, q_out=q)
    assert torch.equal(q[:6], out[:6]) and np.array_equal(q[6:].double().cpu().numpy(), qv[6:])


def test_norm_of_a_zero_row_and_a_negative_position():
    require_gpu()
    q = torch.zeros((3, 2, 64), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((3, 2, 64), 5.0, device="cuda")
    dsv4.qk_norm_rope(q, None, i32([0, 2, 3]), i32([0, -4]), gamma_q=torch.ones(64, device="cuda"), q_out=out, d_status=st)
    assert torch.all(out[:2] == 0) and torch.all(out[2] == 5) and st.item() == A.DEV_BAD_LENGTH


# ---------------------------------------------------------------- append

def make_cache(rng, lens, starts, Hk, D, spare=2, fill=None, extra_blocks=0):
    """Pages in random order for positions up to start + len of each sequence."""
    blocks = max(1, max(-(-(n + s) // PAGE) for n, s in zip(lens, starts)) + extra_blocks)
    B = len(lens)
    pages = B * blocks + spare
    bt = i32(rng.permutation(pages)[:B * blocks].reshape(B, blocks).astype(np.int32))
    c = dsv4.DeviceKv4Cache.zeros(pages, Hk, D, bt)
    if fill is not None:
        for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
            t.fill_(fill)
    return c


def cache_rows(c, s, n):
    """float64 keys and values of positions 0..n-1 of sequence s: [n, Hk, D] each."""
    bt = c.block_table[s].long()
    got = []
    for codes, scales in ((c.k_codes, c.k_scales), (c.v_codes, c.v_scales)):
        co = codes[bt].permute(0, 2, 1, 3).flatten(0, 1)[:n].cpu().numpy()
        sc = scales[bt].permute(0, 2, 1, 3).flatten(0, 1)[:n].cpu().numpy()
        got.append(K.decode(K.unpack(co), sc))
    return got


def check_stored(got, scales, y, bound):
    """got: values stored; scales: their scale bytes; y +- bound: what was rounded."""
    lo, hi = K.amax_of(np.maximum(np.abs(y) - bound, 0)), K.amax_of(np.abs(y) + bound)
    assert np.all((K.scale_bytes(lo) <= scales) & (scales <= K.scale_bytes(hi)))
    a, b = K.decode(K.codes_of(y - bound, scales), scales), K.decode(K.codes_of(y + bound, scales), scales)
    assert np.all((a <= got) & (got <= b))


APPEND = [  # dim, q heads, kv heads, lengths, starts, rope, dtype, extra heads
    (128, 64, 8, [1] * 5, [0, 255, 256, 1000, 77], 64, "bf16", 0),
    (64, 0, 3, [61, 0, 300, 1], [0, 3, 250, 511], 32, "f32", 0),
    (128, 6, 2, [17, 2, 520], [250, 0, 1], 128, "bf16", 10),
    (64, 7, 1, [33], [1 << 18], 0, "f32", 3),
    (64, 12, 12, [5, 6], [0, 255], 64, "bf16", 0),
    (128, 3, 5, [40, 9], [3, 255], 44, "bf16", 2),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"D{c[0]}-{c[2]}-{c[6]}-{len(c[3])}")
def test_append(case):
    require_gpu()
    D, Hq, Hk, lens, starts, rope, din, extra = case
    rng = np.random.default_rng(D + Hk)
    T, dt = sum(lens), {"f32": torch.float32, "bf16": torch.bfloat16}[din]
    k, kv = rand_rows(rng, T, Hk, D, dt, extra)
    v, vv = rand_rows(rng, T, Hk, D, dt, extra)
    q, qv = rand_rows(rng, T, max(Hq, 1), D, dt, extra)
    g = [1 + 0.3 * rng.standard_normal(D).astype(np.float32) for _ in range(2)]
    c = make_cache(rng, lens, starts, Hk, D, fill=0xA5)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    oq, ks, vs = dsv4.kv4_append(k, v, cu_of(lens), i32(starts), c, gamma_k=dev(g[0]), rope_dims=rope,
                                 q=q if Hq else None, gamma_q=dev(g[1]), with_stored=True, d_status=st)
    assert st.item() == 0
    pos = positions(lens, starts)
    y = K.norm_rotate(kv, g[0], 1e-6, pos, rope, 10000.0)
    # where each token's row is, read back
    seq = np.repeat(np.arange(len(lens)), lens)
    page = c.block_table.cpu().numpy()[seq, pos // PAGE]
    for codes, scales, stored, want, bound in ((c.k_codes, c.k_scales, ks, y, pair_bound(y, rope)),
                                               (c.v_codes, c.v_scales, vs, vv, np.zeros_like(vv))):
        sc = scales.cpu().numpy()[page, :, pos % PAGE].astype(np.int64)
        got = K.decode(K.unpack(codes.cpu().numpy()[page, :, pos % PAGE]), sc)
        assert np.array_equal(got, stored.double().cpu().numpy())
        check_stored(got, sc, want, bound)
        # no other row was touched
        keep = np.ones(codes.shape[:3], dtype=bool)
        keep[page, :, pos % PAGE] = False
        assert np.all(codes.cpu().numpy()[keep] == 0xA5) and np.all(scales.cpu().numpy()[keep] == 0xA5)
    if Hq:
        want = K.norm_rotate(qv, g[1], 1e-6, pos, rope, 10000.0)
        assert np.all(np.abs(oq.double().cpu().numpy() - want) <= pair_bound(want, rope) + BF16 * np.abs(want))
    else:
        assert oq is None


def test_append_extremes():
    """Zero blocks, the ends of the exponent range, saturation, infinities and NaN."""
    require_gpu()
    x = np.zeros((7, 1, 64), dtype=np.float32)
    x[1, 0, :32], x[1, 0, 32:] = 6.0, np.nextafter(np.float32(6), np.float32(7))
    x[2, 0, :] = 2.0 ** -40
    x[3, 0, :], x[3, 0, 5] = 3.0e38, -3.0e38
    x[4, 0, 3], x[4, 0, 40] = np.inf, 1.0
    x[5, 0, 40], x[5, 0, 3] = np.nan, -1.0
    x[6, 0, :] = np.float32(1e-42)
    t = dev(x)
    c = make_cache(np.random.default_rng(1), [7], [0], 1, 64)
    _, ks, vs = dsv4.kv4_append(t, t, i32([0, 7]), i32([0]), c, rope_dims=0, with_stored=True)
    assert torch.equal(ks.isnan(), vs.isnan()) and torch.equal(ks.nan_to_num(), vs.nan_to_num())
    got = vs.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        want = K.round4(x)
    np.testing.assert_array_equal(got, want)
    rows = cache_rows(c, 0, 7)
    np.testing.assert_array_equal(rows[0], want)
    np.testing.assert_array_equal(rows[1], want)
    assert got[3].max() == 6 * 2.0 ** 13 and np.isnan(got[4, 0, :32]).all() and np.isnan(got[5, 0, 32:]).all()


def test_append_reports_what_it_cannot_place():
    require_gpu()
    rng = np.random.default_rng(2)
    for starts, spoil, bit, bad in (([0, 510], None, A.DEV_BAD_LENGTH, [5, 6, 7]), ([0, 100], 999, A.DEV_BAD_PAGE, range(3, 8)),
                                    ([0, 100], -1, A.DEV_BAD_PAGE, range(3, 8)), ([0, -3], None, A.DEV_BAD_LENGTH, range(3, 8))):
        k, _ = rand_rows(rng, 8, 2, 64, torch.bfloat16)
        c = make_cache(rng, [3, 5], [0, 500], 2, 64)
        if spoil is not None:
            c.block_table[1, 0] = spoil
        before = [t.clone() for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)]
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        ks = torch.full((8, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        q_out = torch.full((8, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        dsv4.kv4_append(k, k, i32([0, 3, 8]), i32(starts), c, k_stored=ks, q=k, q_out=q_out, d_status=st)
        assert st.item() == bit
        good = [i for i in range(8) if i not in bad]
        assert torch.all(ks[list(bad)] == 9) and not torch.any((ks[good] == 9).all(-1))
        assert torch.all(q_out[list(bad)] == 9) == (starts[1] < 0)
        page = c.block_table[0, 0].item()
        for t, b in zip((c.k_codes, c.v_codes, c.k_scales, c.v_scales), before):
            same = (t == b).all(-1).all(1)  # [page, row]
            touched = {(int(p), int(r)) for p, r in (~same).nonzero()}
            allowed = {(page, r) for r in range(3)} | {(c.block_table[1, 1].item(), 254), (c.block_table[1, 1].item(), 255)}
            assert touched <= allowed


# ---------------------------------------------------------------- attention

def fill_cache(rng, c, lens, starts, scale=1.0):
    """Positions 0..start + len of each sequence through the append (no norm, no rotation)."""
    tot = [n + s for n, s in zip(lens, starts)]
    Hk, D = c.kv_heads, c.dim
    k, _ = rand_rows(rng, sum(tot), Hk, D, torch.bfloat16)
    v, _ = rand_rows(rng, sum(tot), Hk, D, torch.bfloat16)
    dsv4.kv4_append(k * scale, v, cu_of(tot), i32([0] * len(tot)), c, rope_dims=0)


def check_attention(c, q, lens, starts, out, lse, scale=None, sample=None, ctx=""):
    D = c.dim
    scale = scale or D ** -0.5
    at = 0
    ov, lv, qv = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for s, (n, first) in enumerate(zip(lens, starts)):
        if n:
            kk, vv = cache_rows(c, s, first + n)
            rows = range(n) if sample is None or n <= sample else sorted({0, 1, n // 2, n - 1} | set(range(7, n, max(1, n // sample))))
            for i in rows:
                want, wl, mag, top = K.attention(qv[at + i:at + i + 1], kk[:first + i + 1], vv[:first + i + 1], first + i, scale)
                eps = 2 * (D + 4) * U * top + 2.0 ** -21 + 2 * U * 1.4427 * (top + np.abs(wl))
                tiny = 2.0 ** -32 * np.repeat(np.abs(vv[:first + i + 1]).sum(0), q.shape[1] // c.kv_heads, 0)
                limit = (2.0 ** -11 + 2 * eps[..., None]) * mag + tiny + BF16 * np.abs(want) + 1e-30
                err = np.abs(ov[at + i] - want[0])
                assert np.all(err <= limit[0]), (ctx, s, i, (err / limit[0]).max())
                le = np.abs(lv[at + i] - wl[0])
                assert np.all(le <= (eps + 4 * U * np.abs(wl) + 2.0 ** -21)[0]), (ctx, s, i, le.max())
        at += n


ATTEND = [  # dim, q heads, kv heads, new tokens, first positions
    (128, 8, 1, [1], [0]),
    (128, 8, 2, [1, 1, 1, 1, 1, 1], [62, 63, 64, 255, 256, 257]),
    (64, 8, 8, [1, 1, 1], [0, 5, 700]),                       # one query head a key head
    (64, 5, 1, [1] * 9, [3, 100, 15, 16, 17, 1023, 31, 0, 2]),
    (128, 16, 1, [1, 1], [999, 64]),                          # sixteen rows
    (128, 40, 2, [1, 1], [300, 10]),                          # twenty rows: two row tiles
    (128, 64, 1, [1], [2047]),
    (64, 6, 2, [5, 3, 1, 0, 4], [60, 61, 900, 4, 0]),         # draft tokens; a sequence that brings none
    (128, 4, 4, [9, 2], [250, 0]),
    (128, 8, 2, [100, 1, 37], [0, 500, 219]),                 # pieces of prompts beside a step
    (64, 4, 1, [257, 64], [0, 1]),
    (128, 32, 8, [1], [20000]),                               # one long sequence, split over the card
    (128, 14, 2, [130, 129, 128, 127, 1], [0, 127, 128, 129, 3]),
    (64, 3, 3, [300, 17], [513, 0]),
    (128, 4, 1, [700], [333]),
]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"D{c[0]}-{c[1]}over{c[2]}-{max(c[3])}new-{max(c[4])}")
def test_attention(case):
    require_gpu()
    D, Hq, Hk, lens, starts = case
    rng = np.random.default_rng(sum(starts) + Hq)
    c = make_cache(rng, lens, starts, Hk, D, fill=0xFF)  # rows behind the ends read as NaN
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, sum(lens), Hq, D, torch.bfloat16, 2)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = None
    for max_new in (max(lens), 1, 17, 5000):  # a hint: any value gives right results
        out, lse = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=max_new, with_lse=True, d_status=st)
        assert st.item() == 0
        check_attention(c, q, lens, starts, out, lse, sample=24, ctx=f"max_new {max_new}")
        if first is None:
            first = (out, lse)
            again = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=max_new, with_lse=True)
            assert torch.equal(out, again[0]) and torch.equal(lse, again[1])  # to the last bit
    only = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=max(lens))
    assert torch.equal(only, first[0])


def test_attention_of_many_sequences():
    """More sequences than a block has threads, most of one length, some empty."""
    require_gpu()
    rng = np.random.default_rng(12)
    B = 403
    lens = [0 if i % 7 == 3 else 1 for i in range(B)]
    starts = [int(i * 37 % 90) for i in range(B)]
    c = make_cache(rng, lens, starts, 1, 64, fill=0xC8)  # rows behind the ends hold scales that are infinite in fp16
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, sum(lens), 2, 64, torch.bfloat16)
    for max_new in (1, 5):
        out, lse = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=max_new, with_lse=True)
        check_attention(c, q, lens, starts, out, lse)


@pytest.mark.parametrize("Hq,Hk,lens,starts", [(4, 1, [300], [9000]), (16, 2, [33, 1], [5000, 7000]), (8, 1, [700, 300], [3000, 0]),
                                               (80, 20, [300, 280], [2100, 0])])  # the last: more blocks than SMs, a partial wave
def test_attention_splits_the_keys_of_few_rows(Hq, Hk, lens, starts):
    """Few blocks of rows over a long context: the keys are shared out; a hint that is too small leaves rows to walk on over."""
    require_gpu()
    rng = np.random.default_rng(21)
    c = make_cache(rng, lens, starts, Hk, 64, fill=0xFF)
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, sum(lens), Hq, 64, torch.bfloat16)
    for max_new in (max(lens), max(lens) // 3, 20):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=max_new, with_lse=True, d_status=st)
        assert st.item() == 0
        check_attention(c, q, lens, starts, out, lse, sample=12, ctx=f"max_new {max_new}")


def test_a_cache_of_more_than_32_bits():
    """Codes beyond 2^32 bytes: the last pages of a pool of 36000 (4.7 GB of keys, as much of values)."""
    require_gpu()
    rng = np.random.default_rng(22)
    pages = 36000
    bt = i32([[pages - 1, 3], [pages - 2, pages - 3]])
    c = dsv4.DeviceKv4Cache.zeros(pages, 8, 128, bt)
    assert c.k_codes.numel() > 1 << 32
    for new in (1, 100):
        lens, starts = [new, new], [300, 200]
        fill_cache(rng, c, lens, starts)
        q, _ = rand_rows(rng, 2 * new, 16, 128, torch.bfloat16)
        out, lse = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=new, with_lse=True)
        check_attention(c, q, lens, starts, out, lse, sample=6)
    assert not c.k_codes[4:pages - 3].any()


def test_the_first_call_may_be_captured():
    """A process whose first attention and append are inside a graph capture (modules load lazily)."""
    require_gpu()
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch, compressed_sparse_kv_dsv4_b200 as dsv4
dsv4.load()
def i32(v): return torch.tensor(v, dtype=torch.int32, device='cuda')
runs = []
for new in (1, 200):
    c = dsv4.DeviceKv4Cache.zeros(8, 1, 64, i32([[1, 2]]))
    q = torch.randn(new, 4, 64, device='cuda').bfloat16()
    k = torch.randn(new, 1, 64, device='cuda').bfloat16()
    cu, start = i32([0, new]), i32([0])
    ws = dsv4.kv4_attention_workspace(q, cu, c, max_new=new)
    out = torch.empty_like(q)
    runs.append((c, q, k, cu, start, ws, out, new))
def go(r):
    c, q, k, cu, start, ws, out, new = r
    dsv4.kv4_append(k, k, cu, start, c, rope_dims=0)
    dsv4.kv4_attention(q, cu, start, c, max_new=new, out=out, workspace=ws)
for r in runs:
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(r)
    g.replay()
    torch.cuda.synchronize()
    got = r[6].clone()
    go(r)
    torch.cuda.synchronize()
    assert torch.equal(got, r[6])
print('captured')
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("new", [3, 200])
def test_attention_scales_and_large_scores(new):
    require_gpu()
    rng = np.random.default_rng(13)
    lens, starts = [new, 1], [400, 90]
    c = make_cache(rng, lens, starts, 2, 128)
    fill_cache(rng, c, lens, starts, scale=30.0)
    q, _ = rand_rows(rng, sum(lens), 4, 128, torch.bfloat16)
    for mul, scale in ((1.0, 0.7), (2.0 ** 60, 2.0 ** -62), (2.0 ** -100, 2.0 ** 97)):
        qq = q * mul
        out, lse = dsv4.kv4_attention(qq, cu_of(lens), i32(starts), c, max_new=new, softmax_scale=scale, with_lse=True)
        check_attention(c, qq, lens, starts, out, lse, scale=scale, sample=8)


@pytest.mark.parametrize("new,Hq", [(1, 8), (6, 4), (300, 4)])
def test_attention_nan_stays_with_the_rows_that_see_it(new, Hq):
    """A NaN key block and a NaN value block: rows before them keep finite, equal results."""
    require_gpu()
    rng = np.random.default_rng(14)
    lens, starts = [new], [130]
    c = make_cache(rng, lens, starts, 2, 128)
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, new, Hq, 128, torch.bfloat16)
    clean, _ = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=new, with_lse=True)
    for where in {130 + new // 2, 130 + new - 1}:
        page, row = c.block_table[0, where // PAGE].item(), where % PAGE
        g = Hq // 2
        # values: head 1, block 2 only
        old = c.v_scales[page, 1, row, 2].clone()
        c.v_scales[page, 1, row, 2] = 255
        out, lse = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=new, with_lse=True)
        sees = torch.arange(new, device="cuda") + 130 >= where
        nan = out.isnan()
        want = torch.zeros_like(nan)
        want[sees, g:, 64:96] = True
        assert torch.equal(nan, want) and lse.isfinite().all()
        assert torch.equal(out[~sees], clean[~sees])
        assert torch.equal(out[:, :g], clean[:, :g])
        c.v_scales[page, 1, row, 2] = old
        # keys: the whole row of head 0 becomes NaN
        old = c.k_scales[page, 0, row, 1].clone()
        c.k_scales[page, 0, row, 1] = 255
        out, lse = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=new, with_lse=True)
        want = torch.zeros_like(nan)
        want[sees, :g] = True
        assert torch.equal(out.isnan(), want) and torch.equal(lse.isnan(), want[..., 0])
        assert torch.equal(out[~sees], clean[~sees])
        c.k_scales[page, 0, row, 1] = old


@pytest.mark.parametrize("new", [4, 300])
def test_attention_of_a_nan_query_is_that_rows_alone(new):
    require_gpu()
    rng = np.random.default_rng(19)
    c = make_cache(rng, [new], [100], 1, 64)
    fill_cache(rng, c, [new], [100])
    q, _ = rand_rows(rng, new, 2, 64, torch.bfloat16)
    clean, lse0 = dsv4.kv4_attention(q, cu_of([new]), i32([100]), c, max_new=new, with_lse=True)
    q = q.clone()
    q[2, 1, 5] = float("nan")
    out, lse = dsv4.kv4_attention(q, cu_of([new]), i32([100]), c, max_new=new, with_lse=True)
    assert out[2, 1].isnan().all() and lse[2, 1].isnan()
    out[2, 1], lse[2, 1] = clean[2, 1], lse0[2, 1]
    assert torch.equal(out, clean) and torch.equal(lse, lse0)


@pytest.mark.parametrize("new", [1, 40, 300])
def test_attention_reports_bad_pages_and_lengths(new):
    require_gpu()
    rng = np.random.default_rng(15)
    lens, starts = [new, new], [600, 20]
    c = make_cache(rng, lens, starts, 1, 64)
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, 2 * new, 4, 64, torch.bfloat16)
    good, _ = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=new, with_lse=True)
    kk, vv = cache_rows(c, 0, 600 + new)
    for spoil in (1 << 30, -1):
        old = c.block_table[0, 1].clone()
        c.block_table[0, 1] = spoil
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=new, with_lse=True, d_status=st)
        c.block_table[0, 1] = old
        assert st.item() == A.DEV_BAD_PAGE
        assert torch.equal(out[new:], good[new:])
        # the page's positions (256..511) are left out
        for i in {0, new - 1}:
            m = 600 + i + 1
            keep = [j for j in range(m) if not 256 <= j < 512]
            want, wl, mag, top = K.attention(q[i:i + 1].double().cpu().numpy(), kk[keep], vv[keep], len(keep) - 1, 0.125)
            eps = 2 * 68 * U * top + 2.0 ** -21 + 2 * U * 1.4427 * (top + np.abs(wl))
            limit = (2.0 ** -11 + 2 * eps[..., None]) * mag + BF16 * np.abs(want)
            assert np.all(np.abs(out[i].double().cpu().numpy() - want[0]) <= limit[0])
    # every page gone: zero, and -inf
    bad = dsv4.DeviceKv4Cache(c.k_codes, c.v_codes, c.k_scales, c.v_scales, torch.full_like(c.block_table, -1))
    out, lse = dsv4.kv4_attention(q, cu_of(lens), i32(starts), bad, max_new=new, with_lse=True)
    assert torch.all(out == 0) and torch.all(lse == -np.inf)
    # negative and over-long positions, lengths that run backwards or past the tokens
    for cu, start, skipped in (([0, new, 2 * new], [600, -1], slice(new, None)), ([0, new, 5 * new], [600, 20], slice(new, None)),
                               ([0, new, new - 1], [600, 20], slice(new, None))):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = torch.full_like(out, 3.0)
        o, lse = dsv4.kv4_attention(q, i32(cu), i32(start), c, max_new=new, out=o, with_lse=True, d_status=st)
        assert st.item() == A.DEV_BAD_LENGTH
        assert torch.all(o[skipped] == 3)
        # (where the line of work is cut depends on the batch, and with it the last bits)
        check_attention(c, q[:new], [new], [600], o[:new], lse[:new], sample=4)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = dsv4.kv4_attention(q, cu_of(lens), i32([2 ** 31 - 1, 20]), c, max_new=new, with_lse=True, d_status=st)
    assert st.item() == A.DEV_BAD_LENGTH
    second = dsv4.DeviceKv4Cache(c.k_codes, c.v_codes, c.k_scales, c.v_scales, c.block_table[1:])
    check_attention(second, q[new:], [new], [20], o[new:], lse[new:], sample=4)


def test_attention_leaves_the_rows_behind():
    require_gpu()
    rng = np.random.default_rng(16)
    for lens in ([2, 3], [150, 3]):
        T = sum(lens)
        c = make_cache(rng, lens, [70, 0], 2, 128)
        fill_cache(rng, c, lens, [70, 0])
        q, _ = rand_rows(rng, T + 140, 8, 128, torch.bfloat16)
        out = torch.full((T + 140, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T + 140, 8), 3.0, device="cuda")
        dsv4.kv4_attention(q, cu_of(lens), i32([70, 0]), c, max_new=max(lens), out=out, lse=lse)
        assert torch.all(out[T:] == 3) and torch.all(lse[T:] == 3)
        check_attention(c, q, lens, [70, 0], out, lse, sample=8)


# ---------------------------------------------------------------- few rows over tables with room for long contexts

# Here a score also carries a rounding of q's elements 2^-14 below the row's largest, by at most 2^-22 of that. Of a
# normal row one element in 4000 is that small (all are under 5): m of them move a score by m 2^-22 * 5 max |k| scale, while S
# sums 128 products of means 0.8 each and max |k| is under 5: m 2^-22 * 25 / 80 S < m 2^-23 S, of the bound's 2^-16 S.

ROOMY = [  # q heads, kv heads, new tokens, first positions
    (8, 1, [1], [0]),
    (8, 2, [1] * 8, [62, 63, 64, 126, 127, 128, 255, 256]),
    (4, 4, [1, 1], [5, 700]),                    # one query head a key head
    (6, 1, [1, 1, 1], [127, 129, 511]),          # rows that are not there
    (4, 2, [4, 3, 0, 1], [60, 126, 900, 4]),     # draft tokens; a sequence that brings none
    (16, 1, [1, 1], [999, 64]),                  # sixteen rows: two row tiles
    (4, 1, [5, 6], [124, 250]),                  # row tiles that see fewer positions than the last
    (32, 8, [1], [20000]),
    (8, 1, [1, 1], [40000, 3]),
    (16, 4, [1] * 150, [i * 13 % 700 for i in range(150)]),
    (2, 1, [0 if i % 7 == 3 else 1 for i in range(330)], [i * 37 % 290 for i in range(330)]),
]


def roomy(rng, lens, starts, Hk, fill=None):
    return make_cache(rng, lens, starts, Hk, 128, fill=fill, extra_blocks=-(-1000 // (Hk * len(lens))))


@pytest.mark.parametrize("case", ROOMY, ids=lambda c: f"{c[0]}over{c[1]}-{len(c[2])}-{max(c[3])}")
@pytest.mark.parametrize("fill", [0xFF, 0xC8])
def test_roomy_attention(case, fill):
    require_gpu()
    Hq, Hk, lens, starts = case
    rng = np.random.default_rng(sum(starts) + Hq)
    c = roomy(rng, lens, starts, Hk, fill)  # what lies behind the ends is NaN, or infinite in fp16
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, sum(lens), Hq, 128, torch.bfloat16, 2)
    first = None
    for max_new in (max(lens), 1):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=max_new, with_lse=True, d_status=st)
        assert st.item() == 0
        check_attention(c, q, lens, starts, out, lse, sample=24, ctx=f"max_new {max_new}")
        if first is None:
            first = (out, lse)
            again = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=max_new, with_lse=True)
            assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_roomy_scales_and_rising_scores():
    """Large scores whose maximum moves along the keys, in both directions; rows far from 1."""
    require_gpu()
    rng = np.random.default_rng(31)
    lens, starts = [2, 1], [1500, 3000]
    for order in (1, -1):
        c = roomy(rng, lens, starts, 2)
        tot = [n + s for n, s in zip(lens, starts)]
        k, _ = rand_rows(rng, sum(tot), 2, 128, torch.bfloat16)
        v, _ = rand_rows(rng, sum(tot), 2, 128, torch.bfloat16)
        ramp = torch.cat([torch.linspace(0.01, 30, n, device="cuda") for n in tot])[:, None, None]
        dsv4.kv4_append((k * (ramp if order > 0 else ramp.flip(0))).bfloat16(), v, cu_of(tot), i32([0, 0]), c, rope_dims=0)
        q, _ = rand_rows(rng, 3, 4, 128, torch.bfloat16)
        for mul, scale in ((1.0, 0.7), (2.0 ** 60, 2.0 ** -62), (2.0 ** -100, 2.0 ** 97)):
            out, lse = dsv4.kv4_attention(q * mul, cu_of(lens), i32(starts), c, max_new=2, softmax_scale=scale, with_lse=True)
            check_attention(c, q * mul, lens, starts, out, lse, scale=scale)
    # scores that vanish, under a factor below float32's normal numbers: the mean of the values
    out = dsv4.kv4_attention(q * 2.0 ** -100, cu_of(lens), i32(starts), c, max_new=2, softmax_scale=2.0 ** -60)
    for s, at in ((0, 1), (1, 2)):
        _, vv = cache_rows(c, s, tot[s])
        mean = np.repeat(vv.mean(0), 2, 0)
        assert np.all(np.abs(out[at].double().cpu().numpy() - mean) <= BF16 * np.abs(mean) + 2.0 ** -10 * np.abs(vv).mean(0).max())


def test_roomy_elements_of_all_magnitudes():
    """Rows of q whose elements lie up to 2^-30 apart: the bound's term for the small ones, by the largest."""
    require_gpu()
    rng = np.random.default_rng(32)
    lens, starts = [1, 1], [700, 33]
    c = roomy(rng, lens, starts, 1)
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, 2, 8, 128, torch.bfloat16)
    q = (q * torch.exp2(-torch.from_numpy(rng.integers(0, 30, (2, 8, 128))).cuda().double())).bfloat16()
    out, lse = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=1, softmax_scale=4.0, with_lse=True)
    qv = q.double().cpu().numpy()
    for s in range(2):
        kk, vv = cache_rows(c, s, starts[s] + 1)
        want, wl, mag, top = K.attention(qv[s:s + 1], kk, vv, starts[s], 4.0)
        lost = 4.0 * 2.0 ** -22 * np.abs(qv[s]).max(-1) * np.abs(kk).sum(-1).max()
        eps = 2 * 132 * U * top + lost + 2.0 ** -21 + 2 * U * 1.4427 * (top + np.abs(wl))
        limit = (2.0 ** -11 + 2 * eps[..., None]) * mag + 2.0 ** -32 * np.abs(vv).sum(0) + BF16 * np.abs(want)
        assert np.all(np.abs(out[s].double().cpu().numpy() - want[0]) <= limit[0])
        assert np.all(np.abs(lse[s].double().cpu().numpy() - wl[0]) <= (eps + 4 * U * np.abs(wl) + 2.0 ** -21)[0])


def test_roomy_nan_stays_with_the_rows_that_see_it():
    require_gpu()
    rng = np.random.default_rng(33)
    for new, Hq in ((1, 16), (4, 4)):
        lens, starts = [new], [600]
        c = roomy(rng, lens, starts, 2)
        fill_cache(rng, c, lens, starts)
        q, _ = rand_rows(rng, new, Hq, 128, torch.bfloat16)
        g = Hq // 2
        run = lambda q=q: dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=new, with_lse=True)
        clean, lse0 = run()
        for where in {600 + new // 2, 600 + new - 1, 5}:
            page, row = c.block_table[0, where // PAGE].item(), where % PAGE
            sees = torch.arange(new, device="cuda") + 600 >= where
            for scales, head, blk, cols in ((c.v_scales, 1, 2, slice(64, 96)), (c.k_scales, 0, 1, slice(None))):
                old = scales[page, head, row, blk].clone()
                scales[page, head, row, blk] = 255
                out, lse = run()
                scales[page, head, row, blk] = old
                want = torch.zeros_like(out, dtype=torch.bool)
                want[:, head * g:(head + 1) * g, cols] = sees[:, None, None]
                assert torch.equal(out.isnan(), want) and torch.equal(out[~want], clean[~want])
                assert torch.equal(lse.isnan(), want[..., 0] if scales is c.k_scales else torch.zeros_like(lse, dtype=torch.bool))
        for x in (float("nan"), float("inf")):
            bad = q.clone()
            bad[0, 1, 77] = x
            out, lse = run(bad)
            assert out[0, 1].isnan().all() and lse[0, 1].isnan()
            out[0, 1], lse[0, 1] = clean[0, 1], lse0[0, 1]
            assert torch.equal(out, clean) and torch.equal(lse, lse0)


def test_roomy_bad_pages_and_rows_behind():
    require_gpu()
    rng = np.random.default_rng(34)
    lens, starts = [1, 1], [600, 20]
    c = roomy(rng, lens, starts, 1)
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, 5, 4, 128, torch.bfloat16)
    out = torch.full((5, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 4), 3.0, device="cuda")
    good = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=1, out=out, lse=lse)
    assert torch.all(out[2:] == 3) and torch.all(lse[2:] == 3)
    good = good.clone()
    kk, vv = cache_rows(c, 0, 601)
    keep = [j for j in range(601) if not 256 <= j < 512]
    for spoil in (1 << 30, -1, c.k_codes.shape[0]):
        old = c.block_table[0, 1].clone()
        c.block_table[0, 1] = spoil
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, l = dsv4.kv4_attention(q[:2], cu_of(lens), i32(starts), c, max_new=1, with_lse=True, d_status=st)
        c.block_table[0, 1] = old
        assert st.item() == A.DEV_BAD_PAGE and torch.equal(o[1], good[1])
        want, wl, mag, top = K.attention(q[:1].double().cpu().numpy(), kk[keep], vv[keep], len(keep) - 1, 128 ** -0.5)
        eps = 2 * 132 * U * top + 2.0 ** -21 + 2 * U * 1.4427 * (top + np.abs(wl))
        limit = (2.0 ** -11 + 2 * eps[..., None]) * mag + BF16 * np.abs(want)
        assert np.all(np.abs(o[0].double().cpu().numpy() - want[0]) <= limit[0])
    gone = dsv4.DeviceKv4Cache(c.k_codes, c.v_codes, c.k_scales, c.v_scales, torch.full_like(c.block_table, -1))
    o, l = dsv4.kv4_attention(q[:2], cu_of(lens), i32(starts), gone, max_new=1, with_lse=True)
    assert torch.all(o == 0) and torch.all(l == -np.inf)
    for start in ([600, -1], [2 ** 31 - 1, 20]):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        dsv4.kv4_attention(q[:2], cu_of(lens), i32(start), c, max_new=1, with_lse=True, d_status=st)
        assert st.item() & A.DEV_BAD_LENGTH


def test_roomy_codes_at_any_sixteen_bytes():
    """Codes that start 16 bytes off a multiple of 32 are read all the same."""
    require_gpu()
    rng = np.random.default_rng(35)
    lens, starts = [1, 1], [300, 90]
    c = roomy(rng, lens, starts, 1)
    fill_cache(rng, c, lens, starts)
    raw = torch.empty(c.k_codes.numel() + 64, dtype=torch.uint8, device="cuda")
    at = (16 - raw.data_ptr()) % 32
    moved = raw[at:at + c.k_codes.numel()].view(c.k_codes.shape)
    moved.copy_(c.k_codes)
    c2 = dsv4.DeviceKv4Cache(moved, c.v_codes, c.k_scales, c.v_scales, c.block_table)
    q, _ = rand_rows(rng, 2, 8, 128, torch.bfloat16)
    for x in (c, c2):
        out, lse = dsv4.kv4_attention(q, cu_of(lens), i32(starts), x, max_new=1, with_lse=True)
        check_attention(x, q, lens, starts, out, lse)


def test_roomy_graphs():
    """Captured beside other attention kernels that take tensor memory, replayed over a cache that has moved on."""
    require_gpu()
    rng = np.random.default_rng(36)
    lens, starts = [1, 1], [250, 90]
    c = roomy(rng, lens, [260, 100], 2)
    fill_cache(rng, c, [0, 0], [260, 100])
    q, _ = rand_rows(rng, 2, 8, 128, torch.bfloat16)
    many, _ = rand_rows(rng, 300, 8, 128, torch.bfloat16)
    start, cu, one = i32(starts), cu_of(lens), i32([0])
    first = dsv4.DeviceKv4Cache(c.k_codes, c.v_codes, c.k_scales, c.v_scales, c.block_table[:1, :4].contiguous())

    cu150 = cu_of([150])
    dsv4.kv4_attention(q, cu, start, c, max_new=1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = dsv4.kv4_attention(q, cu, start, c, max_new=1, with_lse=True)
        b = dsv4.kv4_attention(many[:150], cu150, one, first, max_new=150, with_lse=True)
        d = dsv4.kv4_attention(q, cu, start, c, max_new=1, with_lse=True)
    for s in (starts, [256, 91], [0, 0]):
        start.copy_(i32(s))
        g.replay()
        torch.cuda.synchronize()
        check_attention(c, q, lens, s, *a)
        assert torch.equal(a[0], d[0]) and torch.equal(a[1], d[1])
        check_attention(first, many[:150], [150], [0], *b, sample=8)


def test_roomy_pool_of_more_than_32_bits():
    """The last pages of a pool of 4.7 GB of keys and as much of values, under a wide table."""
    require_gpu()
    rng = np.random.default_rng(37)
    pages = 36000
    bt = np.full((2, 70), -1, dtype=np.int32)
    bt[:, :2] = [[pages - 1, 3], [pages - 2, pages - 3]]
    c = dsv4.DeviceKv4Cache.zeros(pages, 8, 128, dev(bt))
    lens, starts = [1, 1], [300, 200]
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, 2, 16, 128, torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = dsv4.kv4_attention(q, cu_of(lens), i32(starts), c, max_new=1, with_lse=True, d_status=st)
    assert st.item() == 0
    check_attention(c, q, lens, starts, out, lse)


def test_roomy_first_call_may_be_captured():
    require_gpu()
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch, compressed_sparse_kv_dsv4_b200 as dsv4
dsv4.load()
def i32(v): return torch.tensor(v, dtype=torch.int32, device='cuda')
c = dsv4.DeviceKv4Cache.zeros(8, 1, 128, i32([[1, 2] + [-1] * 998]))
k = torch.randn(300, 1, 128, device='cuda').bfloat16()
q = torch.randn(1, 4, 128, device='cuda').bfloat16()
dsv4.kv4_append(k, k, i32([0, 300]), i32([0]), c, rope_dims=0)
cu, start = i32([0, 1]), i32([299])
ws = dsv4.kv4_attention_workspace(q, cu, c, max_new=1)
out = torch.empty_like(q)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    dsv4.kv4_attention(q, cu, start, c, max_new=1, out=out, workspace=ws)
g.replay()
torch.cuda.synchronize()
got = out.clone()
dsv4.kv4_attention(q, cu, start, c, max_new=1, out=out, workspace=ws)
torch.cuda.synchronize()
assert torch.equal(got, out) and out.float().abs().max() > 0
print('captured')
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_roomy_calls_beside_others():
    """Steps on two streams and a prompt on a third at once, each with its own workspace: all want tensor memory."""
    require_gpu()
    rng = np.random.default_rng(38)
    lens, starts = [1] * 4, [3000, 700, 90, 0]
    c = roomy(rng, lens, starts, 4)
    fill_cache(rng, c, lens, starts)
    q, _ = rand_rows(rng, 4, 32, 128, torch.bfloat16)
    many, _ = rand_rows(rng, 600, 32, 128, torch.bfloat16)
    first = dsv4.DeviceKv4Cache(c.k_codes, c.v_codes, c.k_scales, c.v_scales, c.block_table[:1, :12].contiguous())
    calls = [(q, cu_of(lens), i32(starts), c, 1), (q, cu_of(lens), i32(starts), c, 1), (many, cu_of([600]), i32([2000]), first, 600)]
    alone = [dsv4.kv4_attention(a, cu, st, x, max_new=m) for a, cu, st, x, m in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    spaces = [dsv4.kv4_attention_workspace(a, cu, x, max_new=m) for a, cu, st, x, m in calls]
    outs = [torch.zeros_like(o) for o in alone]
    torch.cuda.synchronize()
    for _ in range(30):
        for (a, cu, st, x, m), s, ws, o in zip(calls, streams, spaces, outs):
            with torch.cuda.stream(s):
                dsv4.kv4_attention(a, cu, st, x, max_new=m, out=o, workspace=ws)
    torch.cuda.synchronize()
    for o, want in zip(outs, alone):
        assert torch.equal(o, want)
    check_attention(c, q, lens, starts, *dsv4.kv4_attention(*calls[0][:4], max_new=1, with_lse=True))


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("D,Hq,Hk", [(128, 8, 2), (64, 6, 3)])
def test_a_layers_run(D, Hq, Hk):
    """A prompt, then steps and draft tokens: append (with the queries) and attention, against the
    oracle's norm, and its attention over what the cache holds."""
    require_gpu()
    rng = np.random.default_rng(17)
    B = 3
    g = [dev(1 + 0.2 * rng.standard_normal(D).astype(np.float32)) for _ in range(2)]
    ends = np.array([0, 0, 0])
    plan = [[150, 40, 1], [1, 1, 1], [4, 1, 0], [1, 1, 1], [20, 130, 70]]
    c = make_cache(rng, [sum(p[i] for p in plan) for i in range(B)], [0] * B, Hk, D, fill=0xFF)
    for new in plan:
        T = sum(new)
        qkv = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hk, D)).astype(np.float32)).bfloat16().cuda()
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        cu, start = cu_of(new), i32(ends.astype(np.int32))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        qn, ks, vs = dsv4.kv4_append(k, v, cu, start, c, gamma_k=g[1], q=q, gamma_q=g[0], with_stored=True, d_status=st)
        # the queries and keys of the one-pass call and of the separate one are the same
        q2, k2 = dsv4.qk_norm_rope(q, k, cu, start, gamma_q=g[0], gamma_k=g[1])
        assert torch.equal(qn, q2)
        assert torch.all((ks - k2).abs().float() <= k2.abs().float().amax(-1, keepdim=True) / 3)
        out, lse = dsv4.kv4_attention(qn, cu, start, c, max_new=max(new), with_lse=True, d_status=st)
        assert st.item() == 0
        check_attention(c, qn, new, list(ends), out, lse, sample=12)
        ends = ends + np.array(new)


def test_no_tokens():
    require_gpu()
    c = make_cache(np.random.default_rng(1), [4, 4], [0, 0], 2, 64)
    none = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    cu, start = i32([0, 0, 0]), i32([5, 0])
    out, lse = dsv4.kv4_attention(none, cu, start, c, max_new=1, with_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    q, k, v = dsv4.kv4_append(none[:, :2], none[:, :2], cu, start, c, q=none, with_stored=True)
    assert q.shape == (0, 4, 64) and k.shape == v.shape == (0, 2, 64)
    assert dsv4.qk_norm_rope(none, none[:, :2], cu, start)[1].shape == (0, 2, 64)
    # tokens, but none of them any sequence's
    some = torch.ones((300, 4, 64), dtype=torch.bfloat16, device="cuda")
    for max_new in (1, 300):
        out = torch.full_like(some, 3.0)
        dsv4.kv4_attention(some, cu, start, c, max_new=max_new, out=out)
        assert torch.all(out == 3)
    assert torch.all(c.k_codes == 0)


def test_streams_and_graphs():
    """Another stream than the current one; two graphs with workspaces of their own, replayed together
    with changed contents (lengths included: they are read on the device)."""
    require_gpu()
    rng = np.random.default_rng(18)
    D, Hq, Hk = 128, 16, 2
    runs = []
    for n, seed in ((1, 0), (200, 1)):
        lens, starts = [n, n], [500 + seed, 9]
        c = make_cache(rng, lens, [800, 800], Hk, D)
        fill_cache(rng, c, lens, [700, 700])
        k, _ = rand_rows(rng, 2 * n, Hk, D, torch.bfloat16)
        q, _ = rand_rows(rng, 2 * n, Hq, D, torch.bfloat16)
        cu, start = cu_of(lens), i32(starts)
        ws = dsv4.kv4_attention_workspace(q, cu, c, max_new=n)
        out, lse = torch.empty_like(q), torch.empty((2 * n, Hq), device="cuda")
        qn = torch.empty_like(q)
        runs.append((n, c, k, q, cu, start, ws, out, lse, qn))

    def go(r, **kw):
        n, c, k, q, cu, start, ws, out, lse, qn = r
        dsv4.kv4_append(k, k, cu, start, c, q=q, q_out=qn, **kw)
        dsv4.kv4_attention(qn, cu, start, c, max_new=n, out=out, lse=lse, workspace=ws, **kw)

    side = torch.cuda.Stream()
    graphs = []
    for r in runs:
        go(r)
        torch.cuda.synchronize()
        want = (r[7].clone(), r[8].clone())
        r[7].zero_()
        side.wait_stream(torch.cuda.current_stream())
        go(r, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(r[7], want[0]) and torch.equal(r[8], want[1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go(r)
        graphs.append(g)
    for shift in (0, 63):
        for r in runs:
            r[5].add_(shift)
            r[3].mul_(0.5)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        got = [(r[7].clone(), r[8].clone()) for r in runs]
        for r, w in zip(runs, got):
            go(r)
            torch.cuda.synchronize()
            assert torch.equal(r[7], w[0]) and torch.equal(r[8], w[1])


def test_the_binding_refuses():
    require_gpu()
    c = make_cache(np.random.default_rng(1), [4, 4], [0, 0], 2, 64)
    q = torch.zeros((8, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((8, 2, 64), dtype=torch.bfloat16, device="cuda")
    cu, start = i32([0, 4, 8]), i32([0, 0])
    ok = dict(max_new=4)
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:, :3]), dict(q=q.transpose(0, 1)), dict(cu=cu.long()),
                dict(cu=i32([0, 8])), dict(start=i32([0])), dict(start=start.cpu()), dict(out=q[:4]),
                dict(lse=torch.zeros(8, 5, device="cuda")), dict(d_status=torch.zeros(1, device="cuda"))):
        a = dict(q=q, cu=cu, start=start)
        more = {n: v for n, v in bad.items() if n not in a}
        a.update({n: v for n, v in bad.items() if n in a})
        with pytest.raises((ValueError, dsv4.Dsv4Error)):
            dsv4.kv4_attention(a["q"], a["cu"], a["start"], c, **ok, **more)
    with pytest.raises(ValueError):  # expanded: all tokens are one row
        dsv4.kv4_attention(q[:1].expand(8, 4, 64), cu, start, c, max_new=4)
    with pytest.raises(dsv4.Dsv4Error):
        dsv4.kv4_attention(q, cu, start, c, max_new=0)
    with pytest.raises(dsv4.Dsv4Error):
        dsv4.kv4_attention(q, cu, start, c, max_new=4, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    for bad in (dict(v=k[:4]), dict(v=k.float()), dict(k=k[..., :32]), dict(q_out=q), dict(q=q.float()),
                dict(gamma_k=torch.zeros(64, dtype=torch.bfloat16, device="cuda")), dict(k_stored=k.float())):
        a = dict(k=k, v=k, **{n: v for n, v in bad.items() if n not in ("k", "v")})
        a.update({n: v for n, v in bad.items() if n in ("k", "v")})
        with pytest.raises((ValueError, dsv4.Dsv4Error)):
            dsv4.kv4_append(a.pop("k"), a.pop("v"), cu, start, c, **a)
    with pytest.raises((ValueError, dsv4.Dsv4Error)):
        dsv4.qk_norm_rope(q, k.float(), cu, start)
    with pytest.raises(dsv4.Dsv4Error):
        dsv4.qk_norm_rope(q, k, cu, start, out_dtype=torch.float16)
