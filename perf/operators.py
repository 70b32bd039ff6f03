"""The 4-bit paged key/value cache and what works on it: cases, plain forms, exact values.

Three operators, in the order in which an attention layer of a served model calls them:

- `norm`    RMSNorm of each query and key head, then the position rotation, in one pass
- `append`  new tokens' keys (normed, rotated) and values rounded to 4 bits and written to their pages; the step's
            queries take the same pass
- `attend`  causal attention of the new tokens over the 4-bit cache: one token a sequence, a few, or a whole prompt

A sequence s brings the tokens cu[s] .. cu[s+1]-1 at positions start[s], start[s]+1, ...; position p of a sequence is
row p % 256 of page table[s][p / 256]. A page holds, for each key/value head, 256 rows of dim/2 bytes (two e2m1 codes a
byte, the even channel in the low nibble) and dim/32 scale bytes (2^(byte-127), one for 32 channels). A block's scale is
the smallest power of two 2^k with amax <= 6 * 2^k, -23 <= k <= 13, and 2^0 where the block is zero.
"""

import math
import random

import torch

own = False

PAGE = 256
BLOCK = 32
EPS = 1e-6
K_MIN, K_MAX = -23, 13
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one token of one sequence, a layer whose keys stay outside the 4-bit cache: the latency of a decode step
        dict(name="norm step", op="norm", batch=1, new=1, ctx=8191, ragged=False, heads=64, kv_heads=8, dim=128, rope=64,
             dtype="bf16"),
        # the prompts of a small model in float32, of all lengths, the whole head rotated
        dict(name="norm odd f32", op="norm", batch=7, new=357, ctx=100001, ragged=True, heads=9, kv_heads=3, dim=64,
             rope=64, dtype="f32"),
        # eight prompts of 4096 tokens
        dict(name="norm prompt", op="norm", batch=8, new=4096, ctx=0, ragged=False, heads=64, kv_heads=8, dim=128, rope=64,
             dtype="bf16"),
        # a decode step of 32 sequences
        dict(name="append step", op="append", batch=32, new=1, ctx=131072, ragged=True, heads=64, kv_heads=8, dim=128,
             rope=64, dtype="bf16"),
        # pieces of prompts of all lengths, float32, a few heads, without the queries
        dict(name="append odd f32", op="append", batch=5, new=611, ctx=777, ragged=True, heads=0, kv_heads=3, dim=64,
             rope=32, dtype="f32"),
        # eight prompts of 4096 tokens
        dict(name="append prompt", op="append", batch=8, new=4096, ctx=0, ragged=False, heads=64, kv_heads=8, dim=128,
             rope=64, dtype="bf16"),
        # one chat turn's next token: latency
        dict(name="attend step 1", op="attend", batch=1, new=1, ctx=2000, ragged=False, heads=32, kv_heads=8, dim=128),
        # a decode step of 32 sequences of up to 32768 tokens
        dict(name="attend step 32", op="attend", batch=32, new=1, ctx=32767, ragged=True, heads=64, kv_heads=8, dim=128),
        # a decode step at a long context: few sequences, so the axis of the keys is what can be split
        dict(name="attend long", op="attend", batch=4, new=1, ctx=262143, ragged=False, heads=64, kv_heads=8, dim=128),
        # draft tokens to be verified together, odd lengths, small heads
        dict(name="attend draft", op="attend", batch=13, new=5, ctx=9001, ragged=True, heads=24, kv_heads=6, dim=64),
        # a piece of a long prompt behind what the cache holds already
        dict(name="attend piece", op="attend", batch=1, new=2048, ctx=14336, ragged=False, heads=32, kv_heads=8, dim=128),
        # eight prompts of 4096 tokens
        dict(name="attend prompt", op="attend", batch=8, new=4096, ctx=0, ragged=False, heads=32, kv_heads=8, dim=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["norm", "append", "attend", "attend", "attend"])
        c = dict(op=op, ragged=rng.random() < 0.6)
        kv, group = rng.choice([1, 2, 3, 4, 6, 8, 16]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        if kv * group > 64:
            continue
        c["heads"], c["kv_heads"] = kv * group, kv
        if op == "attend":
            c["dim"] = rng.choice([64, 128, 128])
            kind = rng.choice(["step", "draft", "prompt"])
            if kind == "step":
                c["batch"], c["new"], c["ctx"] = _log(rng, 1, 64), 1, _log(rng, 1, 200000) - 1
            elif kind == "draft":
                c["batch"], c["new"], c["ctx"] = _log(rng, 1, 32), rng.randint(2, 9), _log(rng, 1, 60000) - 1
            else:
                c["batch"], c["new"], c["ctx"] = _log(rng, 1, 8), _log(rng, 10, 4096), rng.choice([0, 0, _log(rng, 1, 16000)])
            n = c["ctx"] + c["new"]
            if c["batch"] * n * kv * c["dim"] > 1 << 30 or c["batch"] * c["new"] * n * c["heads"] > 1 << 31:
                continue
        else:
            c["batch"], c["new"], c["ctx"] = _log(rng, 1, 64), _log(rng, 1, 4096), rng.choice([0, _log(rng, 1, 1000000)])
            c["dim"] = rng.choice([64, 128])
            c["rope"] = rng.choice([0, 16, 32, 64, c["dim"]])
            c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
            if op == "append":
                c["ctx"] = min(c["ctx"], 200000)
                if c["batch"] * (c["ctx"] + c["new"]) * kv * c["dim"] > 1 << 31:
                    continue
                if rng.random() < 0.4:
                    c["heads"] = 0
            if c["batch"] * c["new"] * (c["heads"] + 2 * kv) * c["dim"] * (2 if c["dtype"] == "f32" else 1) > 32768 * 72 * 128:
                continue
        return c


def _lengths(case):
    """(first position, new tokens) of each sequence; the first one has the case's full lengths."""
    got = []
    for i in range(case["batch"]):
        f = (i * 0.6180339887498949) % 1.0 if case["ragged"] else 0.0
        g = (i * 0.7548776662466927) % 1.0 if case["ragged"] else 0.0
        got.append((case["ctx"] - int(0.9 * f * case["ctx"]), case["new"] - int(0.8 * g * (case["new"] - 1))))
    return got


# ---------------------------------------------------------------------------------------------------------------
# number formats, plain

def _magnitude(mag):
    """0, 0.5, 1, 1.5, 2, 3, 4, 6 for the magnitude codes 0..7 (floating)."""
    return torch.where(mag < 4, 0.5 * mag, torch.where(mag < 6, mag - 2, 2 * mag - 8))


def _value_table(device, dtype):
    nib = torch.arange(16, device=device)
    nib = _magnitude((nib & 7).to(dtype)) * (1 - 2 * (nib >> 3).to(dtype))
    byte = torch.arange(256, device=device)
    return torch.stack([nib[byte & 15], nib[byte >> 4]], -1)  # [256][2]: a byte's two values


def _values(codes, scales, dtype=torch.float32):
    """What codes [..., dim/2] and scales [..., dim/32] stand for, [..., dim]."""
    v = _value_table(codes.device, dtype)[codes.int()].flatten(-2)
    s = torch.exp2(scales.to(dtype) - 127)
    return (v.unflatten(-1, (-1, BLOCK)) * s[..., None]).flatten(-2)


def _round4(x):
    """Codes [..., dim/2] and scales [..., dim/32] of x [..., dim], and the values that they stand for."""
    b = x.unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1)
    mant, ex = torch.frexp(amax)  # amax = mant * 2^ex, 0.5 <= mant < 1: amax <= 6 * 2^k where mant * 2^ex <= 0.75 * 2^(k+3)
    k = torch.where(mant <= 0.75, ex - 3, ex - 2).clamp(K_MIN, K_MAX)
    k = torch.where(amax == 0, torch.zeros_like(k), k)
    scale = torch.exp2(k.to(x.dtype))[..., None]
    a = (b / scale).abs()
    mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    values = torch.copysign(_magnitude(mag.to(x.dtype)) * scale, b).flatten(-2)
    code = (mag + 8 * torch.signbit(b).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], (k + 127).to(torch.uint8), values


def _norm_rotate(x, gamma, pos, rope, base):
    """RMSNorm over the last axis (x [tokens][heads][dim]) with gamma, then the last `rope` dims' pairs turned by pos * theta."""
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.to(x.dtype)
    if not rope:
        return x
    theta = base ** (-2.0 / rope * torch.arange(rope // 2, dtype=torch.float64, device=x.device))
    angle = pos.to(torch.float64)[:, None] * theta
    c, s = torch.cos(angle).to(x.dtype)[:, None], torch.sin(angle).to(x.dtype)[:, None]
    a, b = x[..., -rope::2], x[..., x.shape[-1] - rope + 1::2]
    turned = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([x[..., :x.shape[-1] - rope], turned], -1)


def _places(cu, start, tokens):
    """The sequence and the position of each token."""
    t = torch.arange(tokens, device=cu.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq, start[seq] + t - cu[seq]


# ---------------------------------------------------------------------------------------------------------------
# what a program has in hand

def _pages(case, lengths, gen):
    """A pool of pages that holds normally distributed keys (with strong and weak channels) and values, and its table."""
    dev = gen.device
    B, Hk, D = case["batch"], case["kv_heads"], case["dim"]
    blocks = max(-(-(p + n) // PAGE) for p, n in lengths)
    pages = B * blocks + 3
    table = torch.randperm(pages, generator=gen, device=dev)[:B * blocks].view(B, blocks).int()
    gain = torch.exp(0.5 * torch.randn(Hk, 1, D, generator=gen, device=dev))
    codes, scales = [], []
    step = max(1, (1 << 27) // (Hk * PAGE * D))
    for which in range(2):
        c = torch.empty(pages, Hk, PAGE, D // 2, dtype=torch.uint8, device=dev)
        s = torch.empty(pages, Hk, PAGE, D // BLOCK, dtype=torch.uint8, device=dev)
        for at in range(0, pages, step):
            x = torch.randn(min(step, pages - at), Hk, PAGE, D, generator=gen, device=dev)
            c[at:at + step], s[at:at + step], _ = _round4(x * gain if which == 0 else x)
        codes.append(c)
        scales.append(s)
    return dict(k_codes=codes[0], v_codes=codes[1], k_scales=scales[0], v_scales=scales[1], table=table)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    lengths = _lengths(case)
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    T = sum(n for _, n in lengths)
    s = dict(case=case, tokens=T, most=max(n for _, n in lengths), keys=max(p + n for p, n in lengths))
    s["start"] = torch.tensor([p for p, _ in lengths], dtype=torch.int32, device=dev)
    s["cu"] = torch.tensor([0] + [n for _, n in lengths], device=dev).cumsum(0).int()

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if case["op"] == "attend":
        s["q"] = normal(T, H, D).bfloat16()
    else:
        # one projection's output: queries, keys and values of a token lie side by side
        both = normal(T, (H + 2 * Hk) * D).to(DTYPES[case["dtype"]])
        s["q"] = both[:, :H * D].view(T, H, D)
        s["k"] = both[:, H * D:(H + Hk) * D].view(T, Hk, D)
        s["v"] = both[:, (H + Hk) * D:].view(T, Hk, D)
        s["gamma_q"] = 1 + 0.2 * normal(D)
        s["gamma_k"] = 1 + 0.2 * normal(D)
    if case["op"] != "norm":
        s.update(_pages(case, lengths, gen))
    if own and case["op"] != "norm":
        import compressed_sparse_kv_dsv4_b200 as dsv4

        s["cache"] = dsv4.DeviceKv4Cache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], s["table"])
        if case["op"] == "attend":
            s["workspace"] = dsv4.kv4_attention_workspace(s["q"], s["cu"], s["cache"], max_new=s["most"])
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass

BASE = 10000.0


def run(state):
    op = state["case"]["op"]
    return _own(state) if own else _norm(state) if op == "norm" else _append(state) if op == "append" else _attend(state)


def _own(s):
    import compressed_sparse_kv_dsv4_b200 as dsv4

    c = s["case"]
    if c["op"] == "norm":
        q, k = dsv4.qk_norm_rope(s["q"], s["k"], s["cu"], s["start"], gamma_q=s["gamma_q"], gamma_k=s["gamma_k"], eps=EPS,
                                 rope_dims=c["rope"], rope_base=BASE)
        return dict(q=q, k=k)
    if c["op"] == "append":
        more = dict(q=s["q"], gamma_q=s["gamma_q"]) if c["heads"] else {}
        if c["heads"] and c["dtype"] != "bf16":  # (the call's own output is bfloat16 whatever the queries are)
            more["q_out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=s["q"].device)
        q, k, v = dsv4.kv4_append(s["k"], s["v"], s["cu"], s["start"], s["cache"], gamma_k=s["gamma_k"], eps=EPS,
                                  rope_dims=c["rope"], rope_base=BASE, with_stored=True, **more)
        return dict(q=q, k=k, v=v)
    out, lse = dsv4.kv4_attention(s["q"], s["cu"], s["start"], s["cache"], max_new=s["most"], with_lse=True,
                                  workspace=s["workspace"])
    return dict(out=out, lse=lse)


def _norm(s):
    c = s["case"]
    _, pos = _places(s["cu"], s["start"], s["tokens"])
    q = _norm_rotate(s["q"].float(), s["gamma_q"], pos, c["rope"], BASE)
    k = _norm_rotate(s["k"].float(), s["gamma_k"], pos, c["rope"], BASE)
    return dict(q=q.to(s["q"].dtype), k=k.to(s["k"].dtype))


def _append(s):
    c = s["case"]
    seq, pos = _places(s["cu"], s["start"], s["tokens"])
    q = _norm_rotate(s["q"].float(), s["gamma_q"], pos, c["rope"], BASE).to(s["q"].dtype) if c["heads"] else None
    k_codes, k_scales, k = _round4(_norm_rotate(s["k"].float(), s["gamma_k"], pos, c["rope"], BASE))
    v_codes, v_scales, v = _round4(s["v"].float())
    page, row = s["table"][seq, pos // PAGE].long(), pos % PAGE
    s["k_codes"][page, :, row], s["k_scales"][page, :, row] = k_codes, k_scales
    s["v_codes"][page, :, row], s["v_scales"][page, :, row] = v_codes, v_scales
    return dict(q=q, k=k.bfloat16(), v=v.bfloat16())


def _attend(s):
    c = s["case"]
    B, H, Hk, D, most = c["batch"], c["heads"], c["kv_heads"], c["dim"], s["most"]
    table, start, cu, n = s["table"].long(), s["start"].long(), s["cu"].long(), s["keys"]
    seq, pos = _places(cu, start, s["tokens"])
    # queries [B][Hk][most * group][D]; the rows behind a sequence's last token repeat it and are not read again
    i = torch.arange(most, device=cu.device)
    at = torch.minimum(cu[:-1, None] + i, cu[1:, None] - 1)
    q = s["q"].float()[at].view(B, most, Hk, H // Hk, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, most * (H // Hk), D)
    k, v = (_values(s[w + "_codes"][table], s[w + "_scales"][table]).transpose(1, 2).reshape(B, Hk, -1, D)[:, :, :n]
            for w in "kv")
    x = torch.matmul(q, k.transpose(-1, -2)).view(B, Hk, most, H // Hk, n)
    x *= D ** -0.5
    hidden = torch.arange(n, device=cu.device) > (start[:, None] + i)[:, :, None]  # [B][most][n]
    x.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    x -= m
    x.exp_()
    total = x.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    x /= total
    out = torch.matmul(x.view(B, Hk, most * (H // Hk), n), v).view(B, Hk, most, H // Hk, D)
    out = out.permute(0, 2, 1, 3, 4).reshape(B, most, H, D)[seq, pos - start[seq]]
    lse = lse.permute(0, 2, 1, 3).reshape(B, most, H)[seq, pos - start[seq]]
    return dict(out=out.bfloat16(), lse=lse)


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    lengths = _lengths(case)
    T, B = sum(n for _, n in lengths), case["batch"]
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    row = Hk * (D // 2 + D // BLOCK)  # bytes of one position's keys (or values)
    if case["op"] == "attend":
        keys = sum(p + n for p, n in lengths)
        pairs = sum(n * p + n * (n + 1) // 2 for p, n in lengths)
        blocks = sum(-(-(p + n) // PAGE) for p, n in lengths)
        return dict(bytes=2 * keys * row + 4 * blocks + 2 * 2 * T * H * D + 4 * T * H + 8 * B, flops=4 * pairs * H * D)
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        return dict(bytes=2 * T * (H + Hk) * D * size + 8 * D + 8 * B, flops=10 * T * (H + Hk) * D)
    return dict(bytes=2 * T * H * D * size + 2 * T * Hk * D * (size + 2) + 2 * T * row + 8 * D + 8 * B,
                flops=10 * T * (H + 2 * Hk) * D)


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits, one sequence at a time

def _exact_heads(x, gamma, first, rope):
    """x [n][heads][dim] at positions first, first + 1, ...: each head over its root mean square, then turned as complex numbers."""
    x = x.double()
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * gamma.double()
    if rope:
        pos = torch.arange(first, first + x.shape[0], dtype=torch.float64, device=x.device)
        freq = torch.exp(torch.arange(0, rope, 2, dtype=torch.float64, device=x.device) * (-math.log(BASE) / rope))
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), torch.outer(pos, freq))
        z = torch.view_as_complex(x[..., x.shape[-1] - rope:].reshape(*x.shape[:-1], rope // 2, 2).contiguous())
        x = torch.cat([x[..., :x.shape[-1] - rope], torch.view_as_real(z * turn[:, None]).flatten(-2)], -1)
    return x


def _exact_round4(x):
    """x [..., dim] in 64 bits -> the nearest of the 4-bit values of its blocks, ties to the even code."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    b = x.reshape(-1, BLOCK)
    k = torch.full((b.shape[0],), K_MIN, dtype=torch.float64, device=x.device)
    top = b.abs().max(-1).values
    for e in range(K_MIN, K_MAX):
        k += (top > 6.0 * 2.0 ** e).double()
    step = torch.where(top > 0, torch.exp2(k), torch.ones_like(k))[:, None]
    a = (b.abs() / step).clamp(max=6.0)
    up = torch.searchsorted(grid, a.contiguous()).clamp(1, 7)
    down = up - 1
    over, under = grid[up] - a, a - grid[down]
    pick = torch.where((over < under) | ((over == under) & (up % 2 == 0)), up, down)
    return (torch.sign(b) * grid[pick] * step).reshape(x.shape)


def _exact_values(codes, scales):
    low, high = codes & 15, codes >> 4
    c = torch.stack([low, high], -1).flatten(-2).long()
    e, m = (c >> 1) & 3, (c & 1).double()
    size = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
    size = torch.where(c >= 8, -size, size)
    return size * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    s = prepare(case, seed)
    lengths = _lengths(case)
    if case["op"] != "attend":
        rows, at = [], 0
        for first, n in lengths:
            part = slice(at, at + n)
            q = _exact_heads(s["q"][part], s["gamma_q"], first, case["rope"]) if case["heads"] else None
            k = _exact_heads(s["k"][part], s["gamma_k"], first, case["rope"])
            if case["op"] == "append":
                rows.append((q, _exact_round4(k), _exact_round4(s["v"][part].double())))
            else:
                rows.append((q, k))
            at += n
        return {w: torch.cat(x) if x[0] is not None else None for w, x in zip("qkv", zip(*rows))}
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    G = H // Hk
    out = torch.empty(s["tokens"], H, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["tokens"], H, dtype=torch.float64, device="cuda")
    at = 0
    for b, (first, n) in enumerate(lengths):
        pages = s["table"][b, :-(-(first + n) // PAGE)].long()
        for h in range(Hk):
            k, v = (_exact_values(s[w + "_codes"][pages, h].flatten(0, 1)[:first + n],
                                  s[w + "_scales"][pages, h].flatten(0, 1)[:first + n]) for w in "kv")
            for i in range(0, n, 512):
                m = min(512, n - i)
                q = s["q"][at + i:at + i + m, h * G:(h + 1) * G].double()
                seen = first + i + m
                x = torch.einsum("igd,jd->igj", q, k[:seen]) / math.sqrt(D)
                j = torch.arange(seen, device=x.device)
                late = j[None, :] > first + i + torch.arange(m, device=x.device)[:, None]
                x = x.masked_fill(late[:, None], -math.inf)
                z = torch.logsumexp(x, -1)
                lse[at + i:at + i + m, h * G:(h + 1) * G] = z
                out[at + i:at + i + m, h * G:(h + 1) * G] = torch.einsum("igj,jd->igd", torch.exp(x - z[..., None]), v[:seen])
        at += n
    return dict(out=out, lse=lse)
