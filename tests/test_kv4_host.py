"""The 4-bit key/value cache without a GPU: the oracle's pins and the refusals of the entry points."""

import ctypes as C
import math

import numpy as np
import pytest
import torch

import compressed_sparse_kv_dsv4_b200 as dsv4
from compressed_sparse_kv_dsv4_b200 import _abi as A
import oracle.dsv4_oracle as O
import oracle.kv4_oracle as K

FAKE = 0x10000  # a 16-byte-aligned dummy address; validation never dereferences pointers


# ---------------------------------------------------------------- the oracle

def test_rounding_takes_the_nearest_value_and_the_smallest_scale_that_holds():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((40, 64)) * np.exp2(rng.integers(-30, 20, (40, 1)))
    x[0] = 0
    x[1, :32] = 6.0 * 2.0 ** 5          # the border itself needs no larger scale
    x[2, :32] = np.nextafter(6.0 * 2.0 ** 5, 1e9)
    y = K.round4(x)
    sb = K.scale_bytes(K.amax_of(x))
    assert sb[1, 0] == 127 + 5 and sb[2, 0] == 127 + 6 and np.all(sb[0] == 127)
    grid = np.concatenate([-K.GRID[::-1], K.GRID])
    for i in range(x.shape[0]):
        for b in range(2):
            s = 2.0 ** (sb[i, b] - 127)
            blk, got = x[i, 32 * b:32 * b + 32], y[i, 32 * b:32 * b + 32]
            best = np.abs(grid[None] * s - blk[:, None]).min(1)
            assert np.all(np.abs(got - blk) == best)
            if K.K_MIN + 127 < sb[i, b] < K.K_MAX + 127 and np.any(blk):
                assert 3.0 * s < np.abs(blk).max() <= 6.0 * s


def test_rounding_ties_go_to_the_even_code():
    s = 2.0 ** -3
    x = np.zeros((1, 32))
    x[0, :8] = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]) * s
    assert np.array_equal(K.round4(x)[0, :8] / s, [0, 1, 1, 2, 2, 4, 4, 6])


def test_codes_agree_with_the_other_oracles_e2m1():
    codes = np.arange(16, dtype=np.uint8)
    packed = O.fp4_pack(codes)
    assert np.array_equal(K.unpack(packed), codes)
    mine = K.decode(K.unpack(np.tile(packed, 2)), np.array([127]))[:16]
    assert np.array_equal(mine, O.e2m1_decode(codes))
    assert np.array_equal(mine[:8], [0, .5, 1, 1.5, 2, 3, 4, 6]) and np.array_equal(mine[8:], -mine[:8])


def test_nonfinite_blocks_read_as_nan():
    x = np.ones((2, 64))
    x[0, 3], x[1, 40] = np.inf, np.nan
    y = K.round4(x)
    assert np.isnan(y[0, :32]).all() and np.isfinite(y[0, 32:]).all()
    assert np.isfinite(y[1, :32]).all() and np.isnan(y[1, 32:]).all()


def test_attention_against_torch_float64():
    rng = np.random.default_rng(4)
    for n, start, Hq, Hk in ((1, 0, 2, 1), (5, 11, 4, 2), (3, 0, 3, 3)):
        q = rng.standard_normal((n, Hq, 16))
        k, v = rng.standard_normal((2, start + n, Hk, 16))
        out, lse, mag, top = K.attention(q, k, v, start, 0.25)
        t = [torch.from_numpy(a).transpose(0, 1) for a in (q, k, v)]
        t[1], t[2] = (a.repeat_interleave(Hq // Hk, 0) for a in t[1:])
        mask = torch.arange(start + n)[None] <= start + torch.arange(n)[:, None]
        ref = torch.nn.functional.scaled_dot_product_attention(*t, attn_mask=mask, scale=0.25).transpose(0, 1)
        assert np.abs(out - ref.numpy()).max() < 1e-12
        assert np.all(mag >= np.abs(out) - 1e-15) and np.all(np.isfinite(lse))


# ---------------------------------------------------------------- the entry points' checks

@pytest.fixture(scope="module")
def lib():
    return dsv4.load()


def _cache(**kw):
    c = A.Kv4Cache(FAKE, FAKE, FAKE, FAKE, FAKE, 16, 8, 2, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _attention(**kw):
    a = A.Kv4AttentionArgs(batch=2, total_tokens=2, max_new=1, heads=8, dim=128, q=FAKE, q_stride=0, cu_seqlens=FAKE,
                           start_pos=FAKE, cache=_cache(), softmax_scale=0.0, out=FAKE, lse=None, d_status=None)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _append(**kw):
    a = A.Kv4AppendArgs(batch=2, total_tokens=2, k=FAKE, v=FAKE, k_stride=0, v_stride=0, dtype=A.BF16, gamma_k=FAKE,
                        eps=1e-6, rope=A.Rope(64, 1e4), cu_seqlens=FAKE, start_pos=FAKE, cache=_cache(), q_heads=0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _norm(**kw):
    a = A.QkNormRopeArgs(batch=2, total_tokens=2, q_heads=8, k_heads=2, dim=128, q=FAKE, k=FAKE, dtype=A.BF16,
                         out_dtype=A.BF16, gamma_q=FAKE, gamma_k=FAKE, eps=1e-6, rope=A.Rope(64, 1e4), cu_seqlens=FAKE,
                         start_pos=FAKE, q_out=FAKE, k_out=FAKE, d_status=None)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_CACHE = [dict(k_codes=None), dict(v_scales=None), dict(block_table=None), dict(num_pages=0), dict(max_blocks=0),
             dict(max_blocks=(1 << 22) + 1), dict(kv_heads=0), dict(k_scales=FAKE + 4), dict(dim=0)]


def test_attention_refusals(lib):
    assert lib.dsv4_kv4_attention(None, None, 0, None) == A.ERR_INVALID_ARG
    assert lib.dsv4_kv4_attention_workspace_size(None) == 0
    bad = [dict(batch=0), dict(batch=65536), dict(total_tokens=-1), dict(total_tokens=(1 << 26) + 1), dict(max_new=0),
           dict(heads=0), dict(heads=7), dict(dim=64), dict(q=None), dict(q=FAKE + 8), dict(q_stride=1000),
           dict(q_stride=8 * 128 + 4), dict(cu_seqlens=None), dict(start_pos=None), dict(out=None), dict(out=FAKE + 2),
           dict(softmax_scale=float("nan")), dict(softmax_scale=float("inf"))]
    for kw in bad + [dict(cache=_cache(**c)) for c in BAD_CACHE]:
        a = _attention(**kw)
        assert lib.dsv4_kv4_attention(C.byref(a), C.c_void_p(FAKE), 1 << 30, None) == A.ERR_INVALID_ARG, kw
    for dim in (32, 96, 256):
        a = _attention(dim=dim, cache=_cache(dim=dim))
        assert lib.dsv4_kv4_attention(C.byref(a), C.c_void_p(FAKE), 1 << 30, None) == A.ERR_UNSUPPORTED
        assert lib.dsv4_kv4_attention_workspace_size(C.byref(a)) == 0
    # the workspace: present, aligned, large enough; its size asks for no rows
    a = _attention()
    need = lib.dsv4_kv4_attention_workspace_size(C.byref(a))
    assert need > 0 and lib.dsv4_kv4_attention_workspace_size(C.byref(_attention(q=None, out=None))) == need
    for ws, n in ((None, need), (FAKE + 16, need), (FAKE, need - 1)):
        assert lib.dsv4_kv4_attention(C.byref(a), C.c_void_p(ws), n, None) == A.ERR_INVALID_ARG
    # nothing to do: nothing is launched
    before = lib.dsv4_launch_count()
    assert lib.dsv4_kv4_attention(C.byref(_attention(total_tokens=0, q=None, out=None)), None, 0, None) == A.OK
    assert lib.dsv4_launch_count() == before


def test_append_refusals(lib):
    assert lib.dsv4_kv4_append(None, None) == A.ERR_INVALID_ARG
    bad = [dict(batch=0), dict(total_tokens=-1), dict(k=None), dict(v=None), dict(v=FAKE + 4), dict(k_stride=100),
           dict(v_stride=2 * 128 + 4), dict(eps=-1.0), dict(eps=float("nan")), dict(rope=A.Rope(63, 1e4)),
           dict(rope=A.Rope(130, 1e4)), dict(rope=A.Rope(64, 0.0)), dict(cu_seqlens=None), dict(q_heads=-1),
           dict(q_heads=4, q=None, q_out=FAKE, q_out_dtype=A.BF16), dict(q_heads=4, q=FAKE, q_out=None, q_out_dtype=A.BF16),
           dict(k_stored=FAKE + 2), dict(v_stored=FAKE + 8)]
    for kw in bad + [dict(cache=_cache(**c)) for c in BAD_CACHE]:
        assert lib.dsv4_kv4_append(C.byref(_append(**kw)), None) == A.ERR_INVALID_ARG, kw
    for kw in (dict(dtype=A.FP8), dict(cache=_cache(dim=256)), dict(cache=_cache(dim=32), rope=A.Rope(32, 1e4)),
               dict(q_heads=4, q=FAKE, q_out=FAKE, q_out_dtype=A.FP8)):
        assert lib.dsv4_kv4_append(C.byref(_append(**kw)), None) == A.ERR_UNSUPPORTED, kw
    assert lib.dsv4_kv4_append(C.byref(_append(total_tokens=0, k=None, v=None)), None) == A.OK


def test_norm_refusals(lib):
    assert lib.dsv4_qk_norm_rope(None, None) == A.ERR_INVALID_ARG
    for kw in (dict(batch=0), dict(q_heads=0, k_heads=0), dict(q_heads=-1), dict(k_heads=1 << 15), dict(dim=0),
               dict(q=None), dict(k=FAKE + 8), dict(q_out=None), dict(k_out=FAKE + 4), dict(q_stride=12),
               dict(eps=-1e-6), dict(rope=A.Rope(3, 1e4)), dict(rope=A.Rope(64, -1.0)), dict(start_pos=None)):
        assert lib.dsv4_qk_norm_rope(C.byref(_norm(**kw)), None) == A.ERR_INVALID_ARG, kw
    for kw in (dict(dim=96), dict(dim=1024), dict(dtype=A.FP8), dict(out_dtype=A.FP4)):
        assert lib.dsv4_qk_norm_rope(C.byref(_norm(**kw)), None) == A.ERR_UNSUPPORTED, kw


def test_the_ctypes_mirror_has_the_headers_layout(tmp_path):
    """Field offsets of the argument structs, as a C compiler lays them out."""
    import os
    import subprocess

    structs = {"dsv4_kv4_cache": A.Kv4Cache, "dsv4_qk_norm_rope_args": A.QkNormRopeArgs,
               "dsv4_kv4_append_args": A.Kv4AppendArgs, "dsv4_kv4_attention_args": A.Kv4AttentionArgs}
    body = "".join(f'printf("%zu\\n", sizeof({n}));' + "".join(
        f'printf("%zu\\n", offsetof({n}, {f[0]}));' for f in s._fields_) for n, s in structs.items())
    src = tmp_path / "layout.c"
    src.write_text(f'#include <stdio.h>\n#include "dsv4.h"\nint main(void) {{ {body} return 0; }}\n')
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for s in structs.values():
        want += [C.sizeof(s)] + [getattr(s, f[0]).offset for f in s._fields_]
    assert got == want


def test_the_binding_checks_shapes_before_it_calls():
    """Host tensors are enough: the checks come before any pointer is taken."""
    bt = torch.zeros((2, 3), dtype=torch.int32)
    c = dsv4.DeviceKv4Cache.zeros(4, 2, 64, bt)
    assert (c.kv_heads, c.dim) == (2, 64)
    for name, t in (("v_codes", c.v_codes[:, :1]), ("k_scales", c.k_scales[..., :1]), ("v_scales", c.v_scales.int()),
                    ("block_table", bt.long()), ("k_codes", c.k_codes.transpose(0, 1))):
        d = dsv4.DeviceKv4Cache(**{**c.__dict__, name: t})
        with pytest.raises(ValueError):
            d.struct()
    with pytest.raises(ValueError):
        dsv4.qk_norm_rope(None, None, bt[0], bt[0])
    assert math.isclose(c.k_codes.numel() + c.k_scales.numel(), 4 * 2 * 256 * 64 * 4.25 / 8)
