"""dsv4_kv4_attention_plan without a GPU: its refusals, its struct, and the kernels that sizes lead to (148 SMs)."""

import ctypes as C
import os
import random
import subprocess

import pytest

import compressed_sparse_kv_dsv4_b200 as dsv4
from compressed_sparse_kv_dsv4_b200 import _abi as A

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    return dsv4.load()


def args(D=128, Hq=64, Hk=8, B=1, T=1, max_new=1, blocks=8, pages=4096, codes=FAKE):
    return A.Kv4AttentionArgs(batch=B, total_tokens=T, max_new=max_new, heads=Hq, dim=D, cu_seqlens=FAKE, start_pos=FAKE,
                              cache=A.Kv4Cache(codes, FAKE, FAKE, FAKE, FAKE, pages, blocks, Hk, D))


def test_plan_refusals(lib):
    plan = A.Kv4Plan()
    assert lib.dsv4_kv4_attention_plan(None, C.byref(plan)) == A.ERR_INVALID_ARG
    assert lib.dsv4_kv4_attention_plan(C.byref(args()), None) == A.ERR_INVALID_ARG
    assert lib.dsv4_kv4_attention_plan(C.byref(args(max_new=0)), C.byref(plan)) == A.ERR_INVALID_ARG
    assert lib.dsv4_kv4_attention_plan(C.byref(args(D=96)), C.byref(plan)) == A.ERR_UNSUPPORTED
    with pytest.raises(dsv4.Dsv4Error):
        dsv4.kv4_attention_plan(args(Hq=7))


def test_plan_has_the_headers_layout(tmp_path):
    src = tmp_path / "layout.c"
    fields = [f[0] for f in A.Kv4Plan._fields_]
    body = 'printf("%zu %d %d %d", sizeof(dsv4_kv4_plan), DSV4_KV4_STEP, DSV4_KV4_STEP_TENSOR, DSV4_KV4_PROMPT);' + "".join(
        f'printf(" %zu", offsetof(dsv4_kv4_plan, {f}));' for f in fields)
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "dsv4.h"\nint main(void) {{ {body} return 0; }}\n')
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [C.sizeof(A.Kv4Plan), A.KV4_STEP, A.KV4_STEP_TENSOR, A.KV4_PROMPT] + [getattr(A.Kv4Plan, f).offset for f in fields]


def test_plans():
    def plan(**kw):
        p = dsv4.kv4_attention_plan(args(**kw))
        return p.form, p.rows, p.units, p.shared, p.splits
    step8, step16, tensor = (A.KV4_STEP, 8, 0, 0, 0), (A.KV4_STEP, 16, 0, 0, 0), (A.KV4_STEP_TENSOR, 8, 0, 0, 0)
    assert plan() == step8                                                     # one short step
    assert plan(B=32, T=32, blocks=128) == tensor                              # steps of up to 32768 positions
    assert plan(B=32, T=32, blocks=128, D=64) == step8                         # tensor scores are for 128 channels
    assert plan(B=32, T=32, blocks=128, codes=FAKE + 16) == step8              # ... with codes at a multiple of 32 bytes
    assert plan(B=32, T=32, blocks=128, pages=1 << 21) == step8                # ... and rows that an int counts
    assert plan(D=64, Hq=24, Hk=6, B=13, T=65, max_new=5, blocks=36) == step16  # drafts
    assert plan(D=128, Hq=16, Hk=4, B=20, T=100, max_new=5, blocks=60) == step16
    assert plan(Hq=32, B=8, T=8 * 4096, max_new=4096, blocks=16) == (A.KV4_PROMPT, 256, 1024 * 4, 0, 1)
    assert plan(Hq=32, T=2048, max_new=2048, blocks=64) == (A.KV4_PROMPT, 256, 256, 108, 4)  # its last wave is shared out
    assert plan(Hq=4, Hk=1, T=300, max_new=300, blocks=64) == (A.KV4_PROMPT, 256, 5, 5, 29)  # few blocks: all are
    # a hint above the tokens there are is the tokens there are
    assert plan(B=4, T=4, max_new=4000, blocks=8) == plan(B=4, T=4, max_new=4, blocks=8)


# ---------------------------------------------------------------- the workspace

def test_one_workspace_holds_for_all_smaller_calls(lib):
    """A call may need more than a larger one (a prompt of 2048 tokens 57 MB, eight of 4096 none); the limit of the largest
    covers every call below it."""
    size = lambda a: lib.dsv4_kv4_attention_workspace_size(C.byref(a))
    limit = lambda a: lib.dsv4_kv4_attention_workspace_limit(C.byref(a))
    large, one = args(Hq=32, B=8, T=8 * 4096, max_new=4096, blocks=64), args(Hq=32, T=2048, max_new=2048, blocks=64)
    assert size(large) < size(one) <= limit(large)
    assert lib.dsv4_kv4_attention_workspace_limit(None) == 0 and limit(args(D=96)) == 0 and limit(args(max_new=0)) == 0
    rng = random.Random(7)
    for _ in range(4000):
        D, Hk, G = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 6, 8, 16, 20]), rng.choice([1, 2, 4, 5, 8, 16])
        B, new, blocks = rng.randint(1, 64), int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(0, 11))
        T = rng.randint(new, B * new)
        top = args(D=D, Hq=Hk * G, Hk=Hk, B=B, T=T, max_new=new, blocks=blocks)
        most = limit(top)
        assert size(top) <= most
        for _ in range(8):
            b, m, w = rng.randint(1, B), rng.randint(1, new), rng.randint(1, blocks)
            t = rng.randint(1, min(T, b * m))
            below = args(D=D, Hq=Hk * G, Hk=Hk, B=b, T=t, max_new=m, blocks=w)
            assert size(below) <= most and limit(below) <= most, (D, Hk, G, (B, T, new, blocks), (b, t, m, w))
    # all that any call at all may need
    assert limit(args(B=4096, T=1 << 26, max_new=1 << 26, blocks=1 << 22)) < 120e6


def test_the_limit_is_not_far_above_what_some_call_needs(lib):
    need = max(lib.dsv4_kv4_attention_workspace_size(C.byref(args(Hq=4 * Hk, Hk=Hk, T=t, max_new=t, blocks=128)))
               for Hk in (1, 2, 4, 8) for t in range(64, 8192, 64))
    assert need <= lib.dsv4_kv4_attention_workspace_limit(C.byref(args(Hq=32, T=8192, max_new=8192, blocks=128))) < 1.1 * need


# ---------------------------------------------------------------- the rotation's base

def test_a_base_whose_angles_cannot_be_reduced_is_refused(lib):
    """Below 2^-16 a pair's angle leaves what the sine and cosine reduce (they would come out of any size)."""
    from tests.test_kv4_host import _append, _norm
    nan, inf = float("nan"), float("inf")
    for base, ok in ((2.0 ** -17, False), (1e-30, False), (nan, False), (-1e4, False), (2.0 ** -16, True), (0.5, True), (inf, True)):
        for a, call in ((_norm(total_tokens=0), lib.dsv4_qk_norm_rope), (_append(total_tokens=0), lib.dsv4_kv4_append)):
            a.rope = A.Rope(64, base)
            assert call(C.byref(a), None) == (A.OK if ok else A.ERR_INVALID_ARG), base
            a.rope = A.Rope(0, base)  # nothing is turned
            assert call(C.byref(a), None) == A.OK
