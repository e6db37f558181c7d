"""8-bit paged KV cache: append with rotation, decode attention, prompt
attention, against plain definitions in 64 bits; refusals; streams, captured
graphs, masked garbage; and a run of the three together."""
import itertools
import math
import subprocess
import sys
from pathlib import Path

import pytest
import torch

import compressed_decode_attention_quantize_b200 as tq

FP8 = torch.float8_e4m3fn
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


# ---------------------------------------------------------------- plain forms
def rotated(x, rope, interleaved):
    """x [rows, heads, d], rope [rows, rot], in 64 bits."""
    half = rope.shape[1] // 2
    c, s = rope[:, None, :half].double(), rope[:, None, half:].double()
    y = x.double().clone()
    ia = torch.arange(0, 2 * half, 2) if interleaved else torch.arange(half)
    ib = ia + (1 if interleaved else half)
    a, b = x[..., ia].double(), x[..., ib].double()
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return y


def spans(cu, lens):
    """(b, first row, rows, first position) of each sequence."""
    for b, n in enumerate(lens):
        yield b, cu[b], cu[b + 1] - cu[b], n - (cu[b + 1] - cu[b])


def plain_attention(cache, q, table, cu, lens, scale, window):
    """Output in 64 bits, and the bound of the kernels' error before the
    output's own rounding.  The scores are fp32 sums of d products (an error
    of at most d 2^-24 of the products' magnitudes, twice: numerator and
    denominator) and a few fp32 roundings of numbers up to their size; the
    weights of the value product are rounded to binary16, half a step of
    2^-11, or of 2^-25 of the largest below 2^-14."""
    n, hq, d = q.shape
    nb, hkv, bs, _ = cache["kcodes"].shape
    k, v = ((cache[x + "codes"].cpu().double() * cache[x + "scale"].cpu().double()[..., None, None]) for x in "kv")
    q, table = q.cpu().double(), table.cpu().long()
    out, tol = torch.zeros_like(q), torch.zeros_like(q)
    cap = table.shape[1] * bs
    for b, r0, rows, start in spans(cu, lens):
        for i in range(rows):
            p = start + i
            t = torch.arange(max(0, p - window + 1 if window else 0), max(0, min(p + 1, cap)))
            page = table[b, t // bs]
            keep = (page >= 0) & (page < nb)
            t, page = t[keep], page[keep]
            if not len(t):
                continue
            for h in range(hq):
                g = h * hkv // hq
                kk, vv = k[page, g, t % bs], v[page, g, t % bs]
                qq = q[r0 + i, h]
                w = torch.softmax(kk @ qq * scale, 0)
                out[r0 + i, h] = w @ vv
                size = (kk.abs() @ qq.abs() * scale).max()
                top = (w * cache["vscale"].cpu().double()[page, g]).max() * 448
                tol[r0 + i, h] = ((2.0 ** -11 + 2 * (d + 8) * 2.0 ** -24 * size + 2.0 ** -20) * (w @ vv.abs())
                                  + len(t) * 2.0 ** -25 * top)
    return out, tol


def check_attention(got, ref, tol):
    got = got.cpu()
    err = (got.double() - ref).abs()
    allowed = tol * (1 + 1e-6) + HALF_STEP[got.dtype] * (ref.abs() + tol) + 1e-30
    worst = (err / allowed).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"error {worst:.3f} times its bound"


# ---------------------------------------------------------------- inputs
def pages_for(lens, bs, g, spare=2, extra=0):
    """A block table of distinct pages in random order; behind a sequence's
    pages stand ids that are no pages.  -> table [B, mb], pages"""
    need = [max(1, -(-n // bs)) for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need) + extra), -7, dtype=torch.int32)
    at = 0
    for b, p in enumerate(need):
        table[b, :p] = order[at:at + p]
        at += p
    return table, total


def random_cache(total, hkv, bs, d, g, dev, spread=1.0):
    """Codes and scales of normal values; the scales vary by e^spread."""
    out = {}
    for x in "kv":
        y = torch.randn(total, hkv, bs, d, generator=g) * torch.exp(spread * torch.randn(total, hkv, 1, 1, generator=g))
        s = y.abs().amax((-2, -1)) / 448
        out[x + "codes"], out[x + "scale"] = (y / s[..., None, None]).to(FP8).to(dev), s.to(dev)
    return out


def hide_garbage(cache, table, lens, bs):
    """NaN codes wherever no token is, and NaN scales of unused pages."""
    used = torch.zeros(cache["kcodes"].shape[0], bs, dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            used[table[b, t // bs], t % bs] = True
    for x in "kv":
        raw = cache[x + "codes"].view(torch.uint8)
        raw.copy_(torch.where(used.to(raw.device)[:, None, :, None], raw, torch.full_like(raw, 0x7F)))
        cache[x + "scale"][(~used.any(1)).to(raw.device)] = float("nan")


def ints(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


# ---------------------------------------------------------------- decode
DECODE = [
    # B lens, Hq, Hkv, d, bs, dtype, window
    ([1], 1, 1, 64, 16, torch.float16, 0),
    ([1, 0, 2, 15, 16, 17], 4, 2, 128, 16, torch.bfloat16, 0),
    ([33, 300, 1, 0, 64, 65], 8, 1, 128, 32, torch.float16, 0),
    ([257, 31], 14, 2, 64, 48, torch.bfloat16, 0),
    ([100, 1000, 513], 32, 2, 128, 64, torch.bfloat16, 0),
    ([700, 3], 9, 1, 128, 256, torch.float16, 0),
    ([129, 40, 7], 12, 3, 64, 112, torch.float16, 33),
    ([400, 77, 1], 16, 1, 64, 16, torch.bfloat16, 1),
    ([400, 90, 0], 6, 6, 128, 16, torch.float16, 100),
    ([2500], 8, 8, 128, 16, torch.bfloat16, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,hq,hkv,d,bs,dtype,window", DECODE)
def test_decode_matches_definition(cuda, lens, hq, hkv, d, bs, dtype, window):
    g = torch.Generator().manual_seed(hash((tuple(lens), hq, d)) & 0xFFFF)
    table, total = pages_for(lens, bs, g, extra=1)
    cache = random_cache(total, hkv, bs, d, g, cuda)
    hide_garbage(cache, table, lens, bs)
    q = torch.randn(len(lens), hq, d, generator=g).to(dtype)
    scale = 1 / math.sqrt(d)
    got = tq.kv8_attn_decode(cache, q.to(cuda), table.to(cuda), ints(lens, cuda), window=window)
    ref, tol = plain_attention(cache, q, table, list(range(len(lens) + 1)), lens, scale, window)
    check_attention(got, ref, tol)


@pytest.mark.gpu
def test_decode_pages_that_are_none_are_masked(cuda):
    g = torch.Generator().manual_seed(5)
    lens, bs = [100, 64, 40], 16
    table, total = pages_for(lens, bs, g)
    table[0, 2], table[0, 6], table[1, :] = -1, total, 2 ** 31 - 1   # none at all in sequence 1
    cache = random_cache(total, 2, bs, 128, g, cuda)
    q = torch.randn(3, 8, 128, generator=g).to(torch.bfloat16)
    got = tq.kv8_attn_decode(cache, q.to(cuda), table.to(cuda), ints(lens, cuda))
    assert not got[1].any()
    ref, tol = plain_attention(cache, q, table, [0, 1, 2, 3], lens, 1 / math.sqrt(128), 0)
    check_attention(got, ref, tol)
    rows = tq.kv8_attn_prefill(cache, q.to(cuda), table.to(cuda), ints([0, 1, 2, 3], cuda), ints(lens, cuda))
    assert not rows[1].any()
    check_attention(rows, ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_scales_far_apart_and_zero(cuda, dtype):
    """Pages whose scales differ by 2^40, pages of zeros, tiny and large queries."""
    g = torch.Generator().manual_seed(6)
    lens, bs = [160, 96], 16
    table, total = pages_for(lens, bs, g)
    cache = random_cache(total, 1, bs, 64, g, cuda)
    cache["vscale"] *= torch.exp2(torch.randint(-20, 21, (total, 1), generator=g).float()).to(cuda)
    zero = table[0, 3].item()
    cache["kcodes"].view(torch.uint8)[zero] = 0
    cache["vcodes"].view(torch.uint8)[zero] = 0
    cache["kscale"][zero] = cache["vscale"][zero] = 0.0
    q = torch.randn(2, 4, 64, generator=g)
    q[0, 1] *= 1e-4
    q[1, 2] = 0
    q = q.to(dtype)
    ref, tol = plain_attention(cache, q, table, [0, 1, 2], lens, 0.125, 0)
    args = (table.to(cuda), ints([0, 1, 2], cuda), ints(lens, cuda))
    check_attention(tq.kv8_attn_decode(cache, q.to(cuda), args[0], args[2]), ref, tol)
    check_attention(tq.kv8_attn_prefill(cache, q.to(cuda), *args), ref, tol)
    if dtype == torch.bfloat16:   # queries far outside binary16's range, exactly
        for f in (2.0 ** 60, 2.0 ** -60):
            moved = dict(cache, kscale=cache["kscale"] / f)
            check_attention(tq.kv8_attn_decode(moved, (q * f).to(cuda), args[0], args[2]), ref, tol)
            check_attention(tq.kv8_attn_prefill(moved, (q * f).to(cuda), *args), ref, tol)


# ---------------------------------------------------------------- prompts
PREFILL = [
    # new rows, past, Hq, Hkv, d, bs, dtype, window
    ([1], [0], 1, 1, 128, 16, torch.float16, 0),
    ([5, 0, 1, 17], [0, 9, 200, 3], 4, 2, 64, 16, torch.bfloat16, 0),
    ([130, 64], [0, 77], 8, 2, 128, 32, torch.float16, 0),
    ([200], [0], 3, 1, 64, 48, torch.bfloat16, 0),
    ([33, 127, 2], [500, 0, 130], 5, 1, 128, 64, torch.bfloat16, 0),
    ([70, 41], [0, 300], 12, 4, 64, 112, torch.float16, 0),
    ([4, 4, 4], [1000, 37, 511], 16, 2, 128, 64, torch.bfloat16, 0),
    ([150], [40], 16, 1, 128, 256, torch.float16, 0),
    ([129, 30], [200, 0], 6, 2, 64, 32, torch.bfloat16, 50),
    ([140, 9], [0, 400], 4, 1, 128, 16, torch.float16, 1),
    ([300], [130], 2, 1, 128, 128, torch.float16, 129),
    ([90], [0], 13, 1, 128, 80, torch.bfloat16, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("new,past,hq,hkv,d,bs,dtype,window", PREFILL)
def test_prefill_matches_definition(cuda, new, past, hq, hkv, d, bs, dtype, window):
    g = torch.Generator().manual_seed(hash((tuple(new), hq, d)) & 0xFFFF)
    lens = [a + b for a, b in zip(new, past)]
    cu = [0] + list(itertools.accumulate(new))
    table, total = pages_for(lens, bs, g, extra=1)
    cache = random_cache(total, hkv, bs, d, g, cuda)
    hide_garbage(cache, table, lens, bs)
    n = cu[-1] + 3                                   # three rows of no sequence
    q = torch.randn(n, hq, d, generator=g).to(dtype)
    out = torch.full((n, hq, d), 7.0, dtype=dtype, device=cuda)
    got = tq.kv8_attn_prefill(cache, q.to(cuda), table.to(cuda), ints(cu, cuda), ints(lens, cuda), window=window,
                              out=out)
    assert got is out and (got[cu[-1]:] == 7.0).all()
    ref, tol = plain_attention(cache, q[:cu[-1]], table, cu, lens, 1 / math.sqrt(d), window)
    check_attention(got[:cu[-1]], ref, tol)


@pytest.mark.gpu
def test_prefill_rows_before_the_first_token_and_past_the_table_are_handled(cuda):
    """Lengths smaller than the rows (rows at negative positions are empty) and
    larger than the table (tokens past it have no weight)."""
    g = torch.Generator().manual_seed(8)
    lens, bs = [3, 32], 16
    table, total = pages_for(lens, bs, g)
    cache = random_cache(total, 1, bs, 64, g, cuda)
    q = torch.randn(13, 2, 64, generator=g).to(torch.float16)
    cu, said = [0, 5, 13], [3, 36]                   # 36 tokens claimed, 32 in the table
    got = tq.kv8_attn_prefill(cache, q.to(cuda), table.to(cuda), ints(cu, cuda), ints(said, cuda))
    assert not got[:2].any()
    ref, tol = plain_attention(cache, q, table, cu, said, 0.125, 0)
    check_attention(got, ref, tol)


# ---------------------------------------------------------------- append
def plain_append(cache, k, v, table, cu, lens, rope, interleaved):
    """The cache after the append, as (codes before rounding / their bound of
    error, scales), in 64 bits: name -> (wanted [.., d] in code units, scale)."""
    nb, hkv, bs, d = cache["kcodes"].shape
    cap = table.shape[1] * bs
    want = {x: cache[x + "codes"].cpu().double() for x in "kv"}
    exact = {x: torch.ones(want[x].shape[:3], dtype=torch.bool) for x in "kv"}   # codes that must stay as they are
    scale = {x: cache[x + "scale"].cpu().double() for x in "kv"}
    for b, r0, rows, start in spans(cu, lens):
        pos = [p for p in range(max(0, start), min(start + rows, cap))]
        for j in sorted({p // bs for p in pos}):
            page = int(table[b, j])
            if not 0 <= page < nb:
                continue
            mine = [p for p in pos if p // bs == j]
            sl, r = [p % bs for p in mine], [r0 + p - start for p in mine]
            for x, src in (("k", k), ("v", v)):
                y = src[r].double()
                if x == "k" and rope is not None:
                    y = rotated(src[r], rope[mine], interleaved)
                y = y.transpose(0, 1)                                             # [hkv, tokens, d]
                old = scale[x][page].clone() if sl[0] else torch.zeros(hkv, dtype=torch.float64)
                new = torch.maximum(old, y.abs().amax((-2, -1)) / 448)
                div = torch.where(new > 0, new, torch.ones_like(new))
                older = torch.arange(bs) < sl[0]
                grew = (new > old)[:, None] & older
                want[x][page] = torch.where(grew[..., None], want[x][page] * (old / div)[:, None, None], want[x][page])
                exact[x][page] &= ~grew
                want[x][page][:, sl] = y / div[:, None, None]
                exact[x][page][:, sl] = False
                scale[x][page] = new
    return want, exact, scale


def check_append(cache, want, exact, scale):
    for x in "kv":
        got = cache[x + "codes"].cpu().float().double()
        s = cache[x + "scale"].cpu().double()
        # Three fp32 roundings of the rotation, one of the division by 448.
        assert ((s - scale[x]).abs() <= scale[x] * 2.0 ** -21).all(), x
        same = exact[x][..., None].expand_as(got)
        assert torch.equal(got[same], want[x][same]), x
        y = want[x][~same]
        # Half a step of e4m3 (2^-4 of the value, 2^-10 below 2^-6), and the
        # fp32 roundings of rotation, scale and quotient.
        allowed = torch.maximum(y.abs() * 2.0 ** -4, torch.full_like(y, 2.0 ** -10)) + 448 * 2.0 ** -20
        assert ((got[~same] - y).abs() <= allowed).all(), x


APPEND = [
    # new rows, past, Hq, Hkv, d, bs, dtype, rot, interleaved
    ([1], [0], 1, 1, 64, 16, torch.bfloat16, 64, False),
    ([1, 1, 0, 1], [15, 16, 7, 100], 8, 2, 128, 16, torch.bfloat16, 128, False),
    ([40, 1, 0, 17], [3, 31, 5, 0], 4, 4, 128, 32, torch.float16, 64, False),
    ([100, 33], [0, 50], 6, 3, 64, 48, torch.float32, 32, True),
    ([300, 5], [10, 250], 2, 1, 128, 256, torch.bfloat16, 128, True),
    ([513], [0], 3, 1, 128, 256, torch.float32, 16, False),
    ([70], [200], 5, 5, 64, 128, torch.float16, 0, False),
    ([2, 2, 2], [14, 15, 16], 16, 8, 128, 16, torch.float16, 128, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("new,past,hq,hkv,d,bs,dtype,rot,interleaved", APPEND)
def test_append_matches_definition(cuda, new, past, hq, hkv, d, bs, dtype, rot, interleaved, strided):
    g = torch.Generator().manual_seed(hash((tuple(new), hq, d, rot)) & 0xFFFF)
    lens = [a + b for a, b in zip(new, past)]
    cu = [0] + list(itertools.accumulate(new))
    table, total = pages_for(lens, bs, g, extra=1)
    cache = random_cache(total, hkv, bs, d, g, cuda)
    n = cu[-1] + 2
    qkv = torch.randn(n, hq + 2 * hkv + 1, d, generator=g).to(dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:hq + 2 * hkv]
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    rope = tq.rope_table(table.shape[1] * bs, rot, device="cpu") if rot else None
    want, exact, scale = plain_append(cache, k, v, table, cu, lens, rope, interleaved)
    whole = qkv.to(cuda)
    dq, dk, dv = ((whole[:, :hq], whole[:, hq:hq + hkv], whole[:, hq + hkv:hq + 2 * hkv]) if strided
                  else (q.to(cuda), k.to(cuda), v.to(cuda)))
    args = (table.to(cuda), ints(cu, cuda), ints(lens, cuda))
    rope_d = rope.to(cuda) if rot else None
    if strided:                                    # in place, in the projection's output
        out = tq.kv8_append(cache, dk, dv, *args, q=dq, rope=rope_d, interleaved=interleaved, q_out=dq)
        assert out is dq and torch.equal(whole[:, hq:].cpu(), qkv[:, hq:])
    else:
        buf = torch.full((n, hq, d), 7.0, dtype=dtype, device=cuda)
        out = tq.kv8_append(cache, dk, dv, *args, q=dq, rope=rope_d, interleaved=interleaved, q_out=buf)
        assert (out[cu[-1]:] == 7.0).all()
    check_append(cache, want, exact, scale)
    for b, r0, rows, start in spans(cu, lens):
        if rows:
            x = q[r0:r0 + rows]
            ref = rotated(x, rope[start:start + rows], interleaved) if rot else x.double()
            size = x.double().abs().amax(-1, keepdim=True) * 2
            err = (out[r0:r0 + rows].cpu().double() - ref).abs()
            assert (err <= HALF_STEP[dtype] * ref.abs() + 4 * 2.0 ** -24 * size).all()


@pytest.mark.gpu
def test_append_values_are_the_fp32_formula_bit_for_bit(cuda):
    """Values are not rotated: maximum, quotient and rounding are single IEEE
    operations, so the codes are those of torch's tensor quotients (torch
    divides by a number as a product with its reciprocal, which is not one)."""
    g = torch.Generator().manual_seed(11)
    x = torch.randn(48, 3, 128, generator=g).to(torch.bfloat16).to(cuda)
    cache = tq.kv8_empty(3, 3, 16, 128)
    table, cu = ints([[2, 0, 1]], cuda), ints([0, 48], cuda)
    tq.kv8_append(cache, x, x, table, cu, ints([48], cuda))
    y = x.float().view(3, 16, 3, 128).transpose(1, 2)
    s = y.abs().amax((-2, -1))
    s = s / torch.full_like(s, 448.0)
    c = (y / s[..., None, None]).to(FP8)
    order = [2, 0, 1]
    for name in ("k", "v"):
        assert torch.equal(cache[name + "scale"][order], s)
        assert torch.equal(cache[name + "codes"][order].view(torch.uint8), c.view(torch.uint8))


@pytest.mark.gpu
def test_append_grows_a_page_token_by_token(cuda):
    """One token a call: the scale follows the largest magnitude, older codes
    are coded again, and a page that is begun anew forgets its scale."""
    g = torch.Generator().manual_seed(12)
    bs, d = 16, 64
    cache = tq.kv8_empty(2, 1, bs, d)
    cache["vscale"][1] = 1e6                        # of an earlier life of the page
    table, cu = ints([[1]], cuda), ints([0, 1], cuda)
    host = {k: v.cpu() for k, v in cache.items()}
    for t in range(bs):
        x = (torch.randn(1, 1, d, generator=g) * 2.0 ** (t // 3)).half()
        want, exact, scale = plain_append(host, x, x, table.cpu(), [0, 1], [t + 1], None, False)
        tq.kv8_append(cache, x.to(cuda), x.to(cuda), table, cu, ints([t + 1], cuda))
        check_append(cache, want, exact, scale)
        host = {k: v.cpu() for k, v in cache.items()}
    assert not cache["vcodes"][0].view(torch.uint8).any() and cache["vscale"][0].item() == 0


@pytest.mark.gpu
def test_append_skips_what_has_no_place(cuda):
    """Rows past the table or at negative positions, pages that are none, zero
    rows, sequences without rows."""
    g = torch.Generator().manual_seed(13)
    bs, d, total = 16, 64, 4
    cache = random_cache(total, 2, bs, d, g, cuda)
    table = ints([[0, 1], [2, -1], [3, 9], [5, 5]], cuda)
    cu, lens = [0, 6, 26, 26, 30], [34, 20, 20, 2]
    k = torch.randn(31, 2, d, generator=g).to(torch.bfloat16)
    k[7] = 0
    q = torch.randn(31, 3, d, generator=g).to(torch.bfloat16)
    rope = tq.rope_table(32, 64, device="cpu")
    before = {a: b.clone() for a, b in cache.items()}
    want, exact, scale = plain_append(cache, k, k, table.cpu(), cu, lens, rope, False)
    out = tq.kv8_append(cache, k.to(cuda), k.to(cuda), table, ints(cu, cuda), ints(lens, cuda), q=q.to(cuda),
                        rope=rope.to(cuda), q_out=torch.full_like(q, 7.0, device=cuda))
    check_append(cache, want, exact, scale)
    assert torch.equal(cache["kcodes"][3].view(torch.uint8), before["kcodes"][3].view(torch.uint8))
    assert not out[4:6].any() and not out[26:28].any() and (out[30] == 7.0).all()
    zeros = torch.zeros(1, 2, d, dtype=torch.bfloat16, device=cuda)
    tq.kv8_append(cache, zeros, zeros, ints([[1]], cuda), ints([0, 1], cuda), ints([1], cuda))
    assert not cache["kscale"][1].any() and not cache["kcodes"][1, :, 0].view(torch.uint8).any()


# ---------------------------------------------------------------- together
def _model_rows(n, hq, hkv, d, g, dtype, dev):
    return torch.randn(n, hq + 2 * hkv, d, generator=g).to(dtype).to(dev)


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,hkv,bs,dtype", [(128, 8, 2, 32, torch.bfloat16), (64, 6, 2, 16, torch.float16)])
def test_prompt_then_steps_then_drafts(cuda, d, hq, hkv, bs, dtype):
    """A server's run: two prompts, decode steps, a chunk of drafted tokens
    with a roll back; every attention against the cache as it then is."""
    g = torch.Generator().manual_seed(d)
    cap = 8
    table = torch.randperm(2 * cap, generator=g).to(torch.int32).view(2, cap).to(cuda)
    cache = tq.kv8_empty(2 * cap, hkv, bs, d)
    rope = tq.rope_table(cap * bs, d)
    scale, lens = 1 / math.sqrt(d), [0, 0]

    def turn(new, decode):
        cu = [0] + list(itertools.accumulate(new))
        for i, c in enumerate(new):
            lens[i] += c
        x = _model_rows(cu[-1], hq, hkv, d, g, dtype, cuda)
        q = tq.kv8_append(cache, x[:, hq:hq + hkv], x[:, hq + hkv:], table, ints(cu, cuda), ints(lens, cuda),
                          q=x[:, :hq], rope=rope)
        if decode:
            got = tq.kv8_attn_decode(cache, q, table, ints(lens, cuda))
        else:
            got = tq.kv8_attn_prefill(cache, q, table, ints(cu, cuda), ints(lens, cuda))
        ref, tol = plain_attention(cache, q, table, cu, lens, scale, 0)
        check_attention(got, ref, tol)

    turn([37, 70], False)
    for _ in range(3):
        turn([1, 1], True)
    turn([4, 3], False)
    lens[0] -= 2                                     # two drafts refused
    turn([1, 1], True)


@pytest.mark.gpu
def test_captured_graph_and_other_stream(cuda):
    """The same step captured once and replayed on new contents, next to one
    on a side stream; both give the eager results bit for bit."""
    g = torch.Generator().manual_seed(21)
    B, hq, hkv, d, bs, cap = 3, 8, 2, 128, 16, 6
    table = torch.randperm(B * cap, generator=g).to(torch.int32).view(B, cap).to(cuda)
    rope = tq.rope_table(cap * bs, d)
    start = random_cache(B * cap, hkv, bs, d, g, cuda)
    x, lens, cu = _model_rows(B, hq, hkv, d, g, torch.bfloat16, cuda), ints([50, 17, 80], cuda), ints([0, 1, 2, 3], cuda)
    ws = torch.empty(max(tq.kv8_decode_workspace_bytes(B, hq, hkv, d), tq.kv8_prefill_workspace_bytes(B, B, hq, hkv, d)),
                     dtype=torch.uint8, device=cuda)

    def step(cache, workspace, stream=None):
        q = tq.kv8_append(cache, x[:, hq:hq + hkv], x[:, hq + hkv:], table, cu, lens, q=x[:, :hq], rope=rope,
                          stream=stream)
        a = tq.kv8_attn_decode(cache, q, table, lens, workspace=workspace, stream=stream)
        b = tq.kv8_attn_prefill(cache, q, table, cu, lens, workspace=workspace, stream=stream)
        return a, b

    held = {k: v.clone() for k, v in start.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(held, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(held, ws)
    for turn in range(2):
        x.copy_(_model_rows(B, hq, hkv, d, g, torch.bfloat16, cuda))
        lens.add_(turn)
        for k in held:
            held[k].copy_(start[k])
        eager = {k: v.clone() for k, v in start.items()}
        other = {k: v.clone() for k, v in start.items()}
        want = step(eager, None)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            beside = step(other, None)
        explicit = {k: v.clone() for k, v in start.items()}
        torch.cuda.synchronize()
        third = step(explicit, None, stream=side)
        torch.cuda.synchronize()
        for got, cache in ((outs, held), (beside, other), (third, explicit)):
            for a, b in zip(got, want):
                assert torch.equal(a, b)
            for k in eager:
                assert torch.equal(cache[k].view(torch.uint8), eager[k].view(torch.uint8))


@pytest.mark.gpu
def test_many_sequences(cuda):
    """More sequences than a block has threads; every third one empty."""
    g = torch.Generator().manual_seed(22)
    B, hq, hkv, d, bs = 900, 2, 1, 64, 16
    lens = [0 if b % 3 == 2 else 1 + (b * 7) % 40 for b in range(B)]
    new = [0 if n == 0 else 1 + b % min(3, n) for b, n in enumerate(lens)]
    new = [min(a, n) for a, n in zip(new, lens)]
    cu = [0] + list(itertools.accumulate(new))
    table, total = pages_for(lens, bs, g)
    cache = random_cache(total, hkv, bs, d, g, cuda)
    x = torch.randn(cu[-1], hkv, d, generator=g).to(torch.float16)
    want, exact, scale = plain_append(cache, x, x, table, cu, lens, None, False)
    tq.kv8_append(cache, x.to(cuda), x.to(cuda), table.to(cuda), ints(cu, cuda), ints(lens, cuda))
    check_append(cache, want, exact, scale)
    q = torch.randn(B, hq, d, generator=g).to(torch.float16)
    got = tq.kv8_attn_decode(cache, q.to(cuda), table.to(cuda), ints(lens, cuda))
    ref, tol = plain_attention(cache, q, table, list(range(B + 1)), lens, 0.125, 0)
    check_attention(got, ref, tol)
    q = torch.randn(cu[-1], hq, d, generator=g).to(torch.float16)
    got = tq.kv8_attn_prefill(cache, q.to(cuda), table.to(cuda), ints(cu, cuda), ints(lens, cuda))
    ref, tol = plain_attention(cache, q, table, cu, lens, 0.125, 0)
    check_attention(got, ref, tol)


# ---------------------------------------------------------------- larger shapes
def gpu_attention(cache, q, table, cu, lens, scale, window, only=None):
    """plain_attention on the GPU, a sequence and head at a time (`only`: these
    heads); the bound takes the largest weights of the whole sequence."""
    n, hq, d = q.shape
    nb, hkv, bs, _ = cache["kcodes"].shape
    out, tol = torch.zeros(q.shape, dtype=torch.float64, device=q.device), torch.zeros_like(q, dtype=torch.float64)
    for b, r0, rows, start in spans(cu, lens):
        if not rows or lens[b] <= 0:
            continue
        pages = table[b, :-(-lens[b] // bs)].long()
        t = torch.arange(lens[b], device=q.device)
        for h in range(hq) if only is None else only:
            g = h * hkv // hq
            k, v = ((cache[x + "codes"][pages, g].double() * cache[x + "scale"][pages, g].double()[:, None, None])
                    .reshape(-1, d)[:lens[b]] for x in "kv")
            w = cache["vscale"][pages, g].double().repeat_interleave(bs)[:lens[b]]
            x = q[r0:r0 + rows, h].double()
            p = (start + torch.arange(rows, device=q.device))[:, None]
            hidden = (t > p) | (t <= p - window if window else t < 0)
            s = (x @ k.T * scale).masked_fill(hidden, -math.inf)
            pr = torch.softmax(s, -1)
            out[r0:r0 + rows, h] = pr @ v
            size = (x.abs() @ k.abs().T * scale).masked_fill(hidden, 0).amax(-1, keepdim=True)
            top = (pr * w).amax(-1, keepdim=True) * 448
            tol[r0:r0 + rows, h] = ((2.0 ** -11 + 2 * (d + 8) * 2.0 ** -24 * size + 2.0 ** -20) * (pr @ v.abs())
                                    + lens[b] * 2.0 ** -25 * top)
    return out, tol


LARGE = [
    # new rows, past, Hq, Hkv, d, bs, dtype, window; the decode kernel's narrow blocks, the tensor-core kernel's items
    ([4] * 40, [37 * i % 900 for i in range(40)], 8, 2, 128, 64, torch.bfloat16, 0),
    ([1] * 63 + [100], [13 * i % 500 for i in range(64)], 8, 2, 64, 16, torch.float16, 0),
    ([2, 3, 1, 0, 4], [20000, 3, 9000, 50, 0], 6, 2, 128, 128, torch.float16, 0),
    ([5, 2, 7], [3000, 100, 5000], 2, 2, 64, 48, torch.bfloat16, 1000),
    ([1, 1], [30000, 12345], 32, 2, 128, 64, torch.bfloat16, 0),
    ([700, 1, 300], [0, 900, 2500], 8, 2, 128, 64, torch.bfloat16, 0),
    ([3000], [500], 4, 1, 64, 256, torch.float16, 0),
    ([520, 33], [0, 4100], 16, 1, 128, 16, torch.bfloat16, 0),
    ([1500, 640], [0, 77], 3, 3, 128, 112, torch.float16, 0),
    ([900, 900], [2000, 0], 10, 2, 64, 80, torch.bfloat16, 300),
    ([40], [40000], 4, 1, 128, 128, torch.bfloat16, 0),
    ([64, 64, 64], [1000, 0, 500], 1, 1, 128, 32, torch.float16, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("new,past,hq,hkv,d,bs,dtype,window", LARGE)
def test_larger_prompts_match_definition(cuda, new, past, hq, hkv, d, bs, dtype, window):
    """Items split over CTAs and joined, several items a CTA, blocks of every kind."""
    g = torch.Generator().manual_seed(len(new) * 1000 + d)
    lens = [a + b for a, b in zip(new, past)]
    cu = [0] + list(itertools.accumulate(new))
    table, total = pages_for(lens, bs, g)
    cache = random_cache(total, hkv, bs, d, g, cuda)
    q = torch.randn(cu[-1], hq, d, generator=g).to(dtype).to(cuda)
    got = tq.kv8_attn_prefill(cache, q, table.to(cuda), ints(cu, cuda), ints(lens, cuda), window=window)
    ref, tol = gpu_attention(cache, q, table.to(cuda), cu, lens, 1 / math.sqrt(d), window)
    check_attention(got, ref.cpu(), tol.cpu())
    last = torch.tensor([c - 1 for c, n in zip(cu[1:], new) if n], device=cuda)   # the newest rows, as a decode
    some = torch.tensor([b for b, n in enumerate(new) if n], device=cuda)
    one = tq.kv8_attn_decode(cache, q[last].contiguous(), table.to(cuda)[some].contiguous(), ints(lens, cuda)[some],
                             window=window)
    check_attention(one, ref[last].cpu(), tol[last].cpu())
    assert tq.tq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [2, 150])
@pytest.mark.parametrize("up", [1.0, -1.0])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_climb_or_fall_far(cuda, rows, up, d):
    """Scores that move by hundreds (in log2) along the sequence, in jumps: the
    running reference has to follow, and nothing may overflow on the way."""
    g = torch.Generator().manual_seed(31)
    bs, n = 16, 700
    table, total = pages_for([n], bs, g)
    cache = random_cache(total, 1, bs, d, g, cuda, spread=0.0)
    jump = torch.linspace(-1, 1, -(-n // bs)) * up            # a page after a page
    host = torch.randn(total, 1, bs, d, generator=g) * 0.3
    for j in range(len(jump)):
        host[table[0, j], 0] += 40 * jump[j] * (1 + (j % 7 == 3))
    s = host.abs().amax((-2, -1)) / 448
    cache["kcodes"], cache["kscale"] = (host / s[..., None, None]).to(FP8).to(cuda), s.to(cuda)
    q = (torch.randn(rows, 2, d, generator=g) * 0.1 + 1).to(torch.bfloat16).to(cuda)
    cu, lens = [0, rows], [n]
    ref, tol = gpu_attention(cache, q, table.to(cuda), cu, lens, 1 / math.sqrt(d), 0)
    got = tq.kv8_attn_prefill(cache, q, table.to(cuda), ints(cu, cuda), ints(lens, cuda))
    check_attention(got, ref.cpu(), tol.cpu())
    one = tq.kv8_attn_decode(cache, q[-1:].contiguous(), table.to(cuda), ints(lens, cuda))
    check_attention(one, ref[-1:].cpu(), tol[-1:].cpu())


@pytest.mark.gpu
def test_windows_larger_than_any_table(cuda):
    g = torch.Generator().manual_seed(32)
    lens, cu = [90, 5], [0, 20, 25]
    table, total = pages_for(lens, 16, g)
    cache = random_cache(total, 1, 16, 64, g, cuda)
    q = torch.randn(25, 2, 64, generator=g).half().to(cuda)
    args = (table.to(cuda), ints(cu, cuda), ints(lens, cuda))
    want = tq.kv8_attn_prefill(cache, q, *args)
    for w in (90, 1 << 30, (1 << 31) - 1):
        assert torch.equal(tq.kv8_attn_prefill(cache, q, *args, window=w), want)


@pytest.mark.gpu
def test_calls_on_two_streams_at_once(cuda):
    """Each with its own workspace; results as one after the other."""
    g = torch.Generator().manual_seed(33)
    new, past = [600, 3], [100, 5000]
    lens, cu = [700, 5003], [0, 600, 603]
    table, total = pages_for(lens, 64, g)
    cache = random_cache(total, 2, 64, 128, g, cuda)
    table = table.to(cuda)
    q = torch.randn(603, 8, 128, generator=g).to(torch.bfloat16).to(cuda)
    lens_d, cu_d = ints(lens, cuda), ints(cu, cuda)
    one = q[[599, 602]].contiguous()
    want = tq.kv8_attn_prefill(cache, q, table, cu_d, lens_d), tq.kv8_attn_decode(cache, one, table, lens_d)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for i, s in enumerate(streams):
            got.append((i % 2, tq.kv8_attn_decode(cache, one, table, lens_d, stream=s) if i % 2
                        else tq.kv8_attn_prefill(cache, q, table, cu_d, lens_d, stream=s)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i, x in got)


@pytest.mark.gpu
@pytest.mark.parametrize("new,said,window", [([16, 0], 72, 1), ([16, 0], 74, 4), ([8, 8], 71, 3)])
def test_blocks_of_rows_past_a_window_are_written(cuda, new, said, window):
    """Rows whose window lies behind the table's end see nothing, although
    earlier rows of their sequence see tokens: their output is 0."""
    g = torch.Generator().manual_seed(41)
    table, total = pages_for([64, 64], 16, g)
    cache = random_cache(total, 1, 16, 64, g, cuda)
    cu, lens = [0] + list(itertools.accumulate(new)), [said, said]
    q = torch.randn(16, 1, 64, generator=g).half()
    out = torch.full((16, 1, 64), 7.0, dtype=torch.float16, device=cuda)
    tq.kv8_attn_prefill(cache, q.to(cuda), table.to(cuda), ints(cu, cuda), ints(lens, cuda), window=window, out=out)
    for b, r0, rows, start in spans(cu, lens):
        some = min(rows, 64 + window - 1 - start)        # rows whose window reaches into the table
        ref, tol = plain_attention(cache, q[r0:r0 + some], table[b:b + 1], [0, some], [start + some], 0.125, window)
        check_attention(out[r0:r0 + some], ref, tol)
        assert not out[r0 + some:r0 + rows].any()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gone", [64, 128, 320, 700])
def test_prompts_whose_first_pages_are_none(cuda, gone, d):
    """The first tokens (700: all) have no page: no weight, and no reference
    for the softmax yet."""
    g = torch.Generator().manual_seed(42)
    n, rows, bs = 700, 150, 32
    table, total = pages_for([n], bs, g)
    table[0, :gone // bs] = -1
    if gone == n:
        table[:] = total
    cache = random_cache(total, 1, bs, d, g, cuda)
    q = torch.randn(rows, 2, d, generator=g).to(torch.bfloat16)
    got = tq.kv8_attn_prefill(cache, q.to(cuda), table.to(cuda), ints([0, rows], cuda), ints([n], cuda))
    ref, tol = plain_attention(cache, q, table, [0, rows], [n], 1 / math.sqrt(d), 0)
    assert got.isfinite().all()
    check_attention(got, ref, tol)


@pytest.mark.gpu
def test_windows_past_32_bits(cuda):
    """A window that no C int holds is one that holds everything, or refused."""
    g = torch.Generator().manual_seed(43)
    table, total = pages_for([90], 16, g)
    cache = random_cache(total, 1, 16, 64, g, cuda)
    q = torch.randn(40, 2, 64, generator=g).half().to(cuda)
    table, cu, lens = table.to(cuda), ints([0, 40], cuda), ints([90], cuda)
    want, one = tq.kv8_attn_prefill(cache, q, table, cu, lens), q[-1:].contiguous()
    for w in (1 << 31, (1 << 32) + 5):
        assert torch.equal(tq.kv8_attn_prefill(cache, q, table, cu, lens, window=w), want)
        assert torch.equal(tq.kv8_attn_decode(cache, one, table, lens, window=w),
                           tq.kv8_attn_decode(cache, one, table, lens))
    with pytest.raises(tq.TQError):
        tq.kv8_attn_decode(cache, one, table, lens, window=-(1 << 32))


@pytest.mark.gpu
@pytest.mark.parametrize("new,past", [([1, 1], [3000, 7]), ([3, 2], [2500, 0]), ([300, 70], [900, 0])])
def test_output_over_the_queries(cuda, new, past):
    g = torch.Generator().manual_seed(44)
    lens, cu = [a + b for a, b in zip(new, past)], [0] + list(itertools.accumulate(new))
    table, total = pages_for(lens, 64, g)
    cache = random_cache(total, 2, 64, 128, g, cuda)
    q = torch.randn(cu[-1], 8, 128, generator=g).to(torch.bfloat16).to(cuda)
    args = (table.to(cuda), ints(cu, cuda), ints(lens, cuda))
    want, mine = tq.kv8_attn_prefill(cache, q, *args), q.clone()
    assert tq.kv8_attn_prefill(cache, mine, *args, out=mine) is mine and torch.equal(mine, want)
    if new == [1, 1]:
        want, mine = tq.kv8_attn_decode(cache, q, args[0], args[2]), q.clone()
        tq.kv8_attn_decode(cache, mine, args[0], args[2], out=mine)
        assert torch.equal(mine, want)


WIDE_COPIES = [
    # new rows, past, Hq, Hkv, bs, dtype, window: d = 64 in pages that hold whole copies of 32 tokens, and that do not
    ([1, 1, 1, 1, 1], [0, 15, 16, 31, 32], 4, 2, 32, torch.float16, 0),
    ([1, 1, 1], [33, 4000, 47], 14, 2, 64, torch.bfloat16, 0),
    ([1, 1], [20011, 700], 9, 1, 32, torch.float16, 0),
    ([1, 1, 1], [5000, 64, 20], 7, 1, 256, torch.bfloat16, 17),
    ([1, 1], [9000, 333], 32, 2, 96, torch.bfloat16, 4097),
    ([4, 3, 0, 2], [2000, 17, 9, 0], 8, 2, 32, torch.float16, 0),
    ([4, 4], [3000, 45], 12, 3, 160, torch.bfloat16, 49),
    ([2, 2], [12000, 30], 6, 3, 48, torch.float16, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("new,past,hq,hkv,bs,dtype,window", WIDE_COPIES)
def test_pages_of_32_tokens_and_others(cuda, new, past, hq, hkv, bs, dtype, window):
    g = torch.Generator().manual_seed(bs * 10 + len(new))
    lens, cu = [a + b for a, b in zip(new, past)], [0] + list(itertools.accumulate(new))
    table, total = pages_for(lens, bs, g, extra=1)
    cache = random_cache(total, hkv, bs, 64, g, cuda)
    hide_garbage(cache, table, lens, bs)
    for b, n in enumerate(lens):                     # a page in the middle that is none
        if n > 6 * bs:
            table[b, 3] = -1 if b % 2 else total
    q = torch.randn(cu[-1], hq, 64, generator=g).to(dtype)
    args = (table.to(cuda), ints(cu, cuda), ints(lens, cuda))
    ref, tol = plain_attention(cache, q, table, cu, lens, 0.125, window)
    check_attention(tq.kv8_attn_prefill(cache, q.to(cuda), *args, window=window), ref, tol)
    some = [b for b, n in enumerate(new) if n]
    last = [cu[b + 1] - 1 for b in some]
    got = tq.kv8_attn_decode(cache, q[last].to(cuda), args[0][some].contiguous(), args[2][some].contiguous(), window=window)
    check_attention(got, ref[last], tol[last])
    assert tq.tq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d,bs", [(128, 128), (64, 32)])
def test_pages_past_4_gib(cuda, d, bs):
    """Pages at the end of a cache whose codes pass 2^32 bytes: the results of
    the same pages in a small cache, bit for bit."""
    g = torch.Generator().manual_seed(51)
    hkv, hq, new, past = 8, 16, [200, 1, 3], [300, 700, 0]
    total = (1 << 32) // (hkv * bs * d) + 64
    lens, cu = [a + b for a, b in zip(new, past)], [0] + list(itertools.accumulate(new))
    table, small = pages_for(lens, bs, g)
    far = torch.where(table >= 0, total - small + table, table)
    near = random_cache(small, hkv, bs, d, g, cuda)
    big = {x: torch.empty((total,) + y.shape[1:], dtype=y.dtype, device=cuda) for x, y in near.items()}
    for x in near:
        big[x][total - small:] = near[x]
    rows = torch.randn(cu[-1], hq + 2 * hkv, d, generator=g).to(torch.bfloat16).to(cuda)
    rope, at = tq.rope_table(table.shape[1] * bs, d), (ints(cu, cuda), ints(lens, cuda))
    got = []
    for cache, pages in ((near, table.to(cuda)), (big, far.to(cuda))):
        q = tq.kv8_append(cache, rows[:, hq:hq + hkv], rows[:, hq + hkv:], pages, *at, q=rows[:, :hq], rope=rope)
        few = q[200:].contiguous()
        got.append((q, tq.kv8_attn_prefill(cache, q, pages, *at), tq.kv8_attn_decode(cache, q[[199, 200, 203]], pages, at[1]),
                    tq.kv8_attn_prefill(cache, few, pages[1:].contiguous(), ints([0, 1, 4], cuda), at[1][1:].contiguous())))
    for a, b in zip(*got):
        assert a.isfinite().all() and torch.equal(a, b)
    for x in near:
        assert torch.equal(near[x].view(torch.uint8), big[x][total - small:].view(torch.uint8))


# ---------------------------------------------------------------- refusals
_FAKE = 1 << 20   # a pointer that is aligned and never read: every case is refused before a launch


def _c_append(**over):
    a = dict(q=_FAKE, ldq=256, q_out=_FAKE, ldqo=256, k=_FAKE, ldk=128, v=_FAKE, ldv=128, dtype=tq.TQ_BF16, n=4, B=2,
             Hq=2, Hkv=1, d=128, cu_q=_FAKE, seq_lens=_FAKE, rope=_FAKE, rope_rows=64, rot=128, interleaved=0,
             kcodes=_FAKE, kscale=_FAKE, vcodes=_FAKE, vscale=_FAKE, table=_FAKE, max_blocks=4, block_size=16,
             num_blocks=9, stream=None)
    a.update(over)
    return tq._lib.tq_kv8_append(*a.values())


def _c_attn(prefill, **over):
    a = dict(q=_FAKE, dtype=tq.TQ_BF16, n=4, B=4, Hq=2, Hkv=1, d=128, kcodes=_FAKE, kscale=_FAKE, vcodes=_FAKE,
             vscale=_FAKE, table=_FAKE, max_blocks=4, block_size=16, num_blocks=9, cu_q=_FAKE, seq_lens=_FAKE, window=0,
             scale=0.1, out=_FAKE, ws=None, ws_bytes=0, stream=None)
    a.update(over)
    if not prefill:
        del a["n"], a["cu_q"]
    fn = tq._lib.tq_kv8_attn_prefill if prefill else tq._lib.tq_kv8_attn_decode
    return fn(*a.values())


CACHE_REFUSALS = [
    (dict(d=96), tq.TQ_ERR_UNSUPPORTED), (dict(block_size=24), tq.TQ_ERR_UNSUPPORTED),
    (dict(block_size=272), tq.TQ_ERR_UNSUPPORTED), (dict(block_size=0), tq.TQ_ERR_UNSUPPORTED),
    (dict(max_blocks=0), tq.TQ_ERR_ARG), (dict(num_blocks=0), tq.TQ_ERR_ARG), (dict(Hkv=0), tq.TQ_ERR_ARG),
    (dict(Hkv=65, Hq=65), tq.TQ_ERR_UNSUPPORTED), (dict(max_blocks=1 << 27), tq.TQ_ERR_UNSUPPORTED),
    (dict(num_blocks=1 << 27), tq.TQ_ERR_UNSUPPORTED),
    (dict(kcodes=None), tq.TQ_ERR_ARG), (dict(vscale=None), tq.TQ_ERR_ARG), (dict(table=None), tq.TQ_ERR_ARG),
    (dict(vcodes=_FAKE + 8), tq.TQ_ERR_ARG), (dict(kscale=_FAKE + 2), tq.TQ_ERR_ARG),
    (dict(seq_lens=None), tq.TQ_ERR_ARG), (dict(B=-1), tq.TQ_ERR_ARG),
]


@pytest.mark.parametrize("over,status", CACHE_REFUSALS + [
    (dict(dtype=7), tq.TQ_ERR_ARG), (dict(n=-1), tq.TQ_ERR_ARG), (dict(k=None), tq.TQ_ERR_ARG),
    (dict(k=_FAKE + 2), tq.TQ_ERR_ARG), (dict(ldk=127), tq.TQ_ERR_ARG), (dict(ldv=132), tq.TQ_ERR_ARG),
    (dict(q_out=None), tq.TQ_ERR_ARG), (dict(ldqo=128), tq.TQ_ERR_ARG), (dict(Hq=0), tq.TQ_ERR_ARG),
    (dict(rot=8), tq.TQ_ERR_UNSUPPORTED), (dict(rot=144), tq.TQ_ERR_UNSUPPORTED), (dict(rope=None), tq.TQ_ERR_ARG),
    (dict(rope_rows=63), tq.TQ_ERR_ARG), (dict(ldqo=384), tq.TQ_ERR_ARG), (dict(cu_q=None), tq.TQ_ERR_ARG), (dict(n=1 << 31), tq.TQ_ERR_UNSUPPORTED)])
def test_append_refuses(over, status):
    assert _c_append(**over) == status
    assert b"tq_kv8_append" in tq._lib.tq_last_error()


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("over,status", CACHE_REFUSALS + [
    (dict(dtype=tq.TQ_F32), tq.TQ_ERR_UNSUPPORTED), (dict(Hq=3, Hkv=2), tq.TQ_ERR_ARG),
    (dict(Hq=17), tq.TQ_ERR_UNSUPPORTED), (dict(window=-1), tq.TQ_ERR_ARG), (dict(scale=0.0), tq.TQ_ERR_ARG),
    (dict(scale=float("nan")), tq.TQ_ERR_ARG), (dict(scale=float("inf")), tq.TQ_ERR_ARG), (dict(q=None), tq.TQ_ERR_ARG),
    (dict(out=_FAKE + 4), tq.TQ_ERR_ARG), (dict(), tq.TQ_ERR_WORKSPACE), (dict(B=4097), tq.TQ_ERR_UNSUPPORTED)])
def test_attention_refuses(over, status, prefill):
    assert _c_attn(prefill, **over) == status
    assert b"tq_kv8_attn" in tq._lib.tq_last_error()


def test_prefill_refuses_its_own():
    assert _c_attn(True, cu_q=None) == tq.TQ_ERR_ARG
    assert _c_attn(True, n=-1) == tq.TQ_ERR_ARG
    assert _c_attn(True, n=1 << 26) == tq.TQ_ERR_UNSUPPORTED


def test_nothing_to_do_is_fine():
    assert _c_append(n=0) == tq.TQ_OK and _c_append(B=0) == tq.TQ_OK
    assert _c_attn(False, B=0) == tq.TQ_OK and _c_attn(True, n=0) == tq.TQ_OK


def test_exports_and_tables():
    assert {"tq_kv8_append", "tq_kv8_attn_decode", "tq_kv8_attn_prefill"} <= set(tq.EXPORTED)
    t = tq.rope_table(70000, 32, device="cpu").double()
    i = torch.arange(16, dtype=torch.float64)
    angle = 69999 * 10000.0 ** (-2 * i / 32)
    assert (t[69999] - torch.cat([angle.cos(), angle.sin()])).abs().max() <= 2.0 ** -24
    c = tq.kv8_empty(3, 2, 16, 64, device="cpu")
    assert c["kcodes"].dtype == FP8 and c["vscale"].shape == (3, 2)


def test_tensors_off_the_gpu_are_refused():
    c = tq.kv8_empty(3, 2, 16, 64, device="cpu")
    i = ints([[0, 1]], "cpu")
    x = torch.zeros(1, 2, 64, dtype=torch.float16)
    with pytest.raises(tq.TQError, match="current CUDA device"):
        tq.kv8_append(c, x, x, i, ints([0, 1], "cpu"), ints([1], "cpu"))
    with pytest.raises(tq.TQError, match="current CUDA device"):
        tq.kv8_attn_decode(c, x, i, ints([1], "cpu"))


@pytest.mark.gpu
def test_binding_refuses_mismatched_tensors(cuda):
    c = tq.kv8_empty(3, 2, 16, 64)
    t, cu, lens = ints([[0, 1]], cuda), ints([0, 1], cuda), ints([1], cuda)
    x = torch.zeros(1, 2, 64, dtype=torch.float16, device=cuda)
    for bad in (dict(c, kcodes=c["kcodes"].view(torch.uint8)), dict(c, kscale=c["kscale"].double()),
                dict(c, vcodes=c["vcodes"][:2]), dict(c, kscale=c["kscale"].t().contiguous().t()),
                dict(c, vscale=c["vscale"].cpu())):
        with pytest.raises(tq.TQError):
            tq.kv8_append(bad, x, x, t, cu, lens)
        with pytest.raises(tq.TQError):
            tq.kv8_attn_decode(bad, x, t, lens)
    for call in (lambda: tq.kv8_append(c, x, x.float(), t, cu, lens),
                 lambda: tq.kv8_append(c, x[:, :1], x, t, cu, lens),
                 lambda: tq.kv8_append(c, x.transpose(1, 2).contiguous().transpose(1, 2), x, t, cu, lens),
                 lambda: tq.kv8_append(c, x, x, t.long(), cu, lens),
                 lambda: tq.kv8_append(c, x, x, t, ints([0], cuda), lens),
                 lambda: tq.kv8_append(c, x, x, t, cu, lens.cpu()),
                 lambda: tq.kv8_append(c, x, x, t, cu, lens, q_out=x),
                 lambda: tq.kv8_append(c, x, x, t, cu, lens, q=x, rope=torch.zeros(31, 64, device=cuda)),
                 lambda: tq.kv8_attn_decode(c, x.float(), t, lens),
                 lambda: tq.kv8_attn_decode(c, x.repeat(2, 1, 1), t, lens),
                 lambda: tq.kv8_attn_decode(c, x[:, :1], t, lens),
                 lambda: tq.kv8_attn_decode(c, x, t, lens, out=torch.empty_like(x).bfloat16()),
                 lambda: tq.kv8_attn_decode(c, x, t, lens, workspace=torch.empty(8, dtype=torch.uint8, device=cuda)),
                 lambda: tq.kv8_attn_prefill(c, x, t, cu, lens, window=-2),
                 lambda: tq.kv8_attn_prefill(c, x, t, cu[:1], lens)):
        with pytest.raises(tq.TQError):
            call()
    if torch.cuda.device_count() > 1:
        with torch.cuda.device(1), pytest.raises(tq.TQError, match="current CUDA device"):
            tq.kv8_attn_decode(c, x, t, lens)


# ---------------------------------------------------------------- weights beside one another
def page_of(cache, x, page, rows):
    """Codes and scales of a page from rows [hkv, bs, d] (a scale of 0 where they are 0)."""
    s = rows.abs().amax((-2, -1)) / 448
    code = torch.where(s[:, None, None] > 0, rows / s[:, None, None].clamp(min=1e-38), torch.zeros_like(rows)).to(FP8)
    cache[x + "codes"][page], cache[x + "scale"][page] = code.to(cache[x + "codes"].device), s.to(cache[x + "scale"].device)


@pytest.mark.gpu
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 32), (64, 16)])
@pytest.mark.parametrize("bits", [13, 20, 30])
@pytest.mark.parametrize("at", [0, 5, 30])
@pytest.mark.parametrize("nats", [0.0, 10.0])
def test_pages_without_values_take_no_range_from_the_others(cuda, d, bs, bits, at, nats):
    """One page of zero values among pages of small ones, its keys like the
    others' or `nats` above: it adds to the weights' sum and to nothing else."""
    g = torch.Generator().manual_seed(1000 * bits + at)
    n = 32 * bs + 7
    table, total = pages_for([n], bs, g)
    cache = random_cache(total, 1, bs, d, g, cuda, spread=0.0)
    cache["vscale"] = cache["vscale"] / cache["vscale"] * 2.0 ** -bits / 448
    sign = torch.randint(0, 2, (d,), generator=g).float() * 2 - 1
    zero = table[0, at].item()
    page_of(cache, "v", zero, torch.zeros(1, bs, d))
    if nats:
        page_of(cache, "k", zero, (sign * nats / math.sqrt(d)).expand(1, bs, d))
    q = (sign + 0.2 * torch.randn(150, 2, d, generator=g)).to(torch.bfloat16)
    for rows in (1, 4, 150):
        x = q[-rows:].contiguous()
        ref, tol = plain_attention(cache, x, table, [0, rows], [n], 1 / math.sqrt(d), 0)
        args = (table.to(cuda), ints([0, rows], cuda), ints([n], cuda))
        check_attention(tq.kv8_attn_prefill(cache, x.to(cuda), *args), ref, tol)
        if rows == 1:
            check_attention(tq.kv8_attn_decode(cache, x.to(cuda), args[0], args[2]), ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_pages_without_values_only(cuda, d):
    g = torch.Generator().manual_seed(61)
    table, total = pages_for([300], 16, g)
    cache = random_cache(total, 1, 16, d, g, cuda)
    cache["vcodes"].view(torch.uint8).zero_()
    for scale in (0.0, 1e-31, 1e-38):
        cache["vscale"].fill_(scale)
        q = torch.randn(150, 2, d, generator=g).to(torch.bfloat16).to(cuda)
        args = (table.to(cuda), ints([0, 150], cuda), ints([300], cuda))
        assert not tq.kv8_attn_prefill(cache, q, *args).any()
        assert not tq.kv8_attn_decode(cache, q[:1].contiguous(), args[0], args[2]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -110])
def test_append_keeps_the_sign_of_zeros(cuda, dtype, size):
    """-0 / scale is -0, whichever way the quotient is taken (scales near the
    ends of the range are divided by)."""
    if dtype == torch.float16 and size < 1:
        size = 2.0 ** -14
    g = torch.Generator().manual_seed(63)
    x = torch.randn(40, 2, 64, generator=g) * size
    x[torch.rand(x.shape, generator=g) < 0.3] = -0.0
    x[torch.rand(x.shape, generator=g) < 0.3] = 0.0
    x = x.to(dtype).to(cuda)
    cache = tq.kv8_empty(3, 2, 16, 64)
    tq.kv8_append(cache, x, x, ints([[0, 1, 2]], cuda), ints([0, 40], cuda), ints([40], cuda))
    y = torch.cat([x.float(), torch.zeros(8, 2, 64, device=cuda)]).view(3, 16, 2, 64).transpose(1, 2)
    s = y.abs().amax((-2, -1))
    s = s / torch.full_like(s, 448.0)
    c = (y / s[..., None, None]).to(FP8).view(torch.uint8)
    for name in ("k", "v"):
        assert torch.equal(cache[name + "scale"], s)
        assert torch.equal(cache[name + "codes"].view(torch.uint8), c)


def test_prefill_takes_the_rows_that_it_documents():
    """2^25 rows reach the check of the workspace, one more does not."""
    assert _c_attn(True, n=1 << 25) == tq.TQ_ERR_WORKSPACE
    assert _c_attn(True, n=(1 << 25) + 1) == tq.TQ_ERR_UNSUPPORTED


def test_import_without_cuda_in_torch():
    """A torch build without CUDA has none of its private entry points: the
    package imports for its host side, and the calls refuse tensors off the GPU."""
    code = """
import torch
for x in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, x):
        delattr(torch._C, x)
import compressed_decode_attention_quantize_b200 as tq
c = tq.kv8_empty(2, 1, 16, 64, device="cpu")
i = lambda *x: torch.tensor(x, dtype=torch.int32)
try:
    tq.kv8_attn_decode(c, torch.zeros(1, 1, 64, dtype=torch.float16), i(0)[None], i(1))
except tq.TQError as e:
    print("refused:", e)
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=Path(__file__).resolve().parent.parent, capture_output=True,
                          text=True, timeout=300)
    assert done.returncode == 0 and "refused:" in done.stdout, done.stderr[-2000:]


@pytest.mark.gpu
@pytest.mark.parametrize("d,bs", [(64, 256), (128, 256), (64, 48)])
def test_tails_far_below_the_largest_weight(cuda, d, bs):
    """The first token of each page outweighs every other by 2^26 and has no
    value: what is read out are the others.  The largest weight is 2^6 at least
    (in the decode kernel 2^8), so binary16, whose least half step is 2^-25, is
    off by 2^-31 (2^-33) of it."""
    g = torch.Generator().manual_seed(62)
    pages, rows, B, hkv = 4096 // bs, 150, 64, 8
    n = pages * bs
    sign = torch.randint(0, 2, (d,), generator=g).float() * 2 - 1
    keys = torch.zeros(pages, hkv, bs, d)
    keys[:, :, 0] = 448 * sign
    values = torch.rand(pages, hkv, bs, d, generator=g) + 1
    values[:, :, 0] = 0
    bits = 26 * math.log(2) / (448 * math.sqrt(d))            # scale of the keys
    cache = {"kcodes": keys.to(FP8).to(cuda), "kscale": torch.full((pages, hkv), bits, device=cuda),
             "vcodes": values.to(FP8).to(cuda), "vscale": torch.ones(pages, hkv, device=cuda)}
    table = torch.arange(pages, dtype=torch.int32, device=cuda).repeat(B, 1)
    q = sign.to(torch.bfloat16).to(cuda).expand(rows, hkv, d).contiguous()
    k, v = (cache[x + "codes"].double().transpose(0, 1).reshape(hkv, n, d) for x in "kv")
    s = torch.einsum("rhd,htd->hrt", q.double(), k) * cache["kscale"][0, 0].double() / math.sqrt(d)
    t = torch.arange(n, device=cuda)
    s = s.masked_fill(t > n - rows + torch.arange(rows, device=cuda)[:, None], -math.inf)
    p = torch.softmax(s, -1)
    ref = (p @ v).transpose(0, 1)
    least = p.amax(-1, keepdim=True) * 2.0 ** -33 * (v.abs().sum(1, keepdim=True))
    tol = (2.0 ** -11 + 2 * (d + 8) * 2.0 ** -24 * 26 * math.log(2) + 2.0 ** -20) * (p @ v.abs())
    wide, tol = (tol + 4 * least).transpose(0, 1), (tol + least).transpose(0, 1)
    got = tq.kv8_attn_prefill(cache, q, table[:1].contiguous(), ints([0, rows], cuda), ints([n], cuda))
    check_attention(got, ref.cpu(), wide.cpu())
    got = tq.kv8_attn_decode(cache, q[-1:].expand(B, -1, -1).contiguous(), table, ints([n] * B, cuda))
    for b in range(B):
        check_attention(got[b:b + 1], ref[-1:].cpu(), tol[-1:].cpu())
    x = q[-4:].repeat(16, 1, 1)                               # few rows of each sequence
    got = tq.kv8_attn_prefill(cache, x, table[:16].contiguous(), ints(list(range(0, 65, 4)), cuda), ints([n] * 16, cuda))
    for b in range(16):
        check_attention(got[4 * b:4 * b + 4], ref[-4:].cpu(), tol[-4:].cpu())


# ---------------------------------------------------------------- single rows beside prompts
MIXED = [
    # new rows, past, Hq, Hkv, d, bs, dtype, window: sequences of few and of many rows in one call
    ([1] * 20 + [300], [37 * i % 700 for i in range(21)], 8, 2, 128, 64, torch.bfloat16, 0),
    ([200] + [1, 4, 5, 0, 16, 17, 3] * 3, [11 * i % 300 for i in range(22)], 4, 4, 64, 32, torch.float16, 0),
    ([1, 2, 1, 90, 1, 0, 1, 1, 70, 2], [900, 3, 0, 50, 16, 8, 2000, 31, 400, 640], 16, 1, 128, 16, torch.bfloat16, 0),
    ([1] * 9 + [257], [200 + 13 * i for i in range(10)], 12, 1, 64, 48, torch.float16, 70),
    ([3] * 40 + [500, 2], [5000] + [17 * i % 400 for i in range(41)], 3, 3, 64, 64, torch.bfloat16, 0),
    ([0] * 30 + [400] + [0] * 9, [0] * 40, 8, 2, 128, 128, torch.float16, 0),
    ([150, 80, 120, 40, 33, 60, 71, 90], [0, 300, 10, 0, 999, 0, 5, 64], 8, 2, 64, 32, torch.bfloat16, 0),
    ([4] * 30, [101 * i % 1500 for i in range(30)], 8, 2, 128, 64, torch.float16, 100),
]


@pytest.mark.gpu
@pytest.mark.parametrize("new,past,hq,hkv,d,bs,dtype,window", MIXED)
def test_few_and_many_rows_in_one_call(cuda, new, past, hq, hkv, d, bs, dtype, window):
    """Whatever the workspace held; rows behind the last sequence stay."""
    g = torch.Generator().manual_seed(len(new) * 100 + hq)
    lens, cu = [a + b for a, b in zip(new, past)], [0] + list(itertools.accumulate(new))
    table, total = pages_for(lens, bs, g, extra=1)
    cache = random_cache(total, hkv, bs, d, g, cuda)
    hide_garbage(cache, table, lens, bs)
    n = cu[-1] + 5
    q = torch.randn(n, hq, d, generator=g).to(dtype).to(cuda)
    ws = torch.full((tq.kv8_prefill_workspace_bytes(n, len(new), hq, hkv, d),), 255, dtype=torch.uint8, device=cuda)
    out = torch.full((n, hq, d), 7.0, dtype=dtype, device=cuda)
    tq.kv8_attn_prefill(cache, q, table.to(cuda), ints(cu, cuda), ints(lens, cuda), window=window, out=out, workspace=ws)
    assert (out[cu[-1]:] == 7.0).all()
    for b, r0, rows, start in spans(cu, lens):
        if rows:
            part = slice(r0, r0 + rows)
            ref, tol = gpu_attention(cache, q[part], table[b:b + 1].to(cuda), [0, rows], [lens[b]], 1 / math.sqrt(d), window)
            check_attention(out[part], ref.cpu(), tol.cpu())
    assert tq.tq_device_fault() == 0


@pytest.mark.gpu
def test_captured_batch_whose_rows_move_between_sequences(cuda):
    """One graph, replayed with the rows dealt out anew: what was a prompt is a
    single row, and the other way round."""
    g = torch.Generator().manual_seed(71)
    B, n, hq, hkv, d, bs, cap = 12, 400, 8, 2, 128, 64, 16
    table = torch.randperm(B * cap, generator=g).to(torch.int32).view(B, cap).to(cuda)
    cache = random_cache(B * cap, hkv, bs, d, g, cuda)
    q = torch.randn(n, hq, d, generator=g).to(torch.bfloat16).to(cuda)
    cu, lens = torch.zeros(B + 1, dtype=torch.int32, device=cuda), torch.zeros(B, dtype=torch.int32, device=cuda)
    ws = torch.empty(tq.kv8_prefill_workspace_bytes(n, B, hq, hkv, d), dtype=torch.uint8, device=cuda)
    out = torch.empty_like(q)
    call = lambda: tq.kv8_attn_prefill(cache, q, table, cu, lens, out=out, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ([1] * 11 + [389], [300, 1, 0, 4, 95] + [0] * 7, [33] * 12, [1] * 12, [0] * 12, [0] * 11 + [400]):
        at, said = [0] + list(itertools.accumulate(new)), [c + 7 * i % 50 + 300 for i, c in enumerate(new)]
        cu.copy_(ints(at, cuda)), lens.copy_(ints(said, cuda))
        out.fill_(7.0)
        graph.replay()
        assert (out[at[-1]:] == 7.0).all()
        for b, r0, rows, start in spans(at, said):
            if rows:
                part = slice(r0, r0 + rows)
                ref, tol = gpu_attention(cache, q[part], table[b:b + 1], [0, rows], [said[b]], 1 / math.sqrt(d), 0)
                check_attention(out[part], ref.cpu(), tol.cpu())
    assert tq.tq_device_fault() == 0


def _shortest(call, turns=10):
    """Device time of a call in microseconds, the shortest of a few."""
    call(), call()
    best = math.inf
    for _ in range(turns):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record(), call(), b.record()
        torch.cuda.synchronize()
        best = min(best, 1000 * a.elapsed_time(b))
    return best


@pytest.mark.gpu
@pytest.mark.parametrize("others", [0, 1])
def test_a_prompt_among_many_sequences_costs_about_itself(cuda, others):
    """1024 rows among 255 sequences of no row or one: the prompt's own call,
    the other rows' decode and launches (the whole took 38 and 5 times that
    where the average rows chose one kernel for all)."""
    g = torch.Generator().manual_seed(72)
    B, hq, hkv, d, bs, rows, past = 256, 32, 8, 128, 64, 1024, 500
    new = [others] * 100 + [rows] + [others] * 155
    lens, cu = [c + (past if c == 1 else 0) for c in new], [0] + list(itertools.accumulate(new))
    table, total = pages_for(lens, bs, g)
    cache, table = random_cache(total, hkv, bs, d, g, cuda), table.to(cuda)
    q = torch.randn(cu[-1], hq, d, generator=g).to(torch.bfloat16).to(cuda)
    cu_d, lens_d = ints(cu, cuda), ints(lens, cuda)
    whole = _shortest(lambda: tq.kv8_attn_prefill(cache, q, table, cu_d, lens_d))
    mine = q[cu[100]:cu[101]].contiguous()
    prompt = _shortest(lambda: tq.kv8_attn_prefill(cache, mine, table[100:101], ints([0, rows], cuda), lens_d[100:101]))
    rest = [b for b in range(B) if b != 100]
    one = q[[cu[b] for b in rest]].contiguous() if others else None
    table2, lens2 = table[rest].contiguous(), lens_d[rest].contiguous()
    decode = _shortest(lambda: tq.kv8_attn_decode(cache, one, table2, lens2)) if others else 0.0
    assert whole <= 1.6 * (prompt + decode) + 30, (whole, prompt, decode)


# ---------------------------------------------------------------- waits that run out
def test_wait_limit_is_exported():
    assert "tq_kv8_set_wait_limit" in tq.EXPORTED and tq._lib.tq_kv8_set_wait_limit(-1) == tq.TQ_OK


@pytest.mark.gpu
@pytest.mark.parametrize("new,past,code", [
    ([1, 1, 1], [3000, 70, 9000], 8), ([4, 2, 3], [2000, 17, 900], 8),       # decode, few rows
    ([700, 300], [100, 2500], 4), ([40], [20000], 4),                        # prompts, one of them split over CTAs
    ([1] * 30 + [600], [2000] * 31, 4),                                      # too little to split: the prompt kernel
    ([1] * 60 + [600], [4000] * 61, 12),                                     # both kernels
])
@pytest.mark.parametrize("d", [64, 128])
def test_waits_that_run_out_are_reported(cuda, new, past, code, d):
    """With waits that give up without looking each kernel returns, having
    waited for its copies and products, and sets its bit of tq_device_fault; the
    bit is cleared by reading it, and the next call is right."""
    g = torch.Generator().manual_seed(81)
    lens, cu = [a + b for a, b in zip(new, past)], [0] + list(itertools.accumulate(new))
    table, total = pages_for(lens, 32, g)
    cache = random_cache(total, 2, 32, d, g, cuda)
    q = torch.randn(cu[-1], 8, d, generator=g).to(torch.bfloat16).to(cuda)
    args = (cache, q, table.to(cuda), ints(cu, cuda), ints(lens, cuda))
    want = tq.kv8_attn_prefill(*args)
    one = (cache, q, args[2], args[4])
    single = tq.kv8_attn_decode(*one) if max(new) == 1 else None
    assert tq.tq_device_fault() == 0
    try:
        tq.kv8_set_wait_limit(0)
        tq.kv8_attn_prefill(*args)
        if single is not None:
            tq.kv8_attn_decode(*one)
    finally:
        tq.kv8_set_wait_limit(-1)
    assert tq.tq_device_fault() == code
    assert tq.tq_device_fault() == 0
    assert torch.equal(tq.kv8_attn_prefill(*args), want)
    if single is not None:
        assert torch.equal(tq.kv8_attn_decode(*one), single)
    assert tq.tq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d,bs", [(64, 16), (64, 32), (128, 48), (128, 256)])
@pytest.mark.parametrize("new,past,window", [([1, 1], [700, 90], 33), ([4, 2], [600, 70], 100), ([150, 60], [500, 900], 77),
                                             ([1] * 9 + [130], [300 + 41 * i for i in range(10)], 64)])
def test_nan_that_no_row_sees(cuda, d, bs, new, past, window):
    """NaN codes before the first row's window and behind the last token, NaN
    scales of pages that nobody sees at all."""
    g = torch.Generator().manual_seed(91)
    lens, cu = [a + b for a, b in zip(new, past)], [0] + list(itertools.accumulate(new))
    table, total = pages_for(lens, bs, g, extra=1)
    cache = random_cache(total, 2, bs, d, g, cuda)
    hide_garbage(cache, table, lens, bs)
    for b, r0, rows, start in spans(cu, lens):
        for j in range(-(-lens[b] // bs)):
            unseen = [t for t in range(j * bs, min((j + 1) * bs, lens[b])) if t < start - window + 1]
            for x in "kv" if unseen else "":
                cache[x + "codes"].view(torch.uint8)[table[b, j], :, [t % bs for t in unseen]] = 0x7F
                if unseen[-1] == min((j + 1) * bs, lens[b]) - 1:
                    cache[x + "scale"][table[b, j]] = float("nan")
    q = torch.randn(cu[-1], 4, d, generator=g).to(torch.bfloat16).to(cuda)
    args = (table.to(cuda), ints(cu, cuda), ints(lens, cuda))
    clean = {x: torch.where(torch.isnan(y.float()), torch.zeros_like(y.float()), y.float()).to(y.dtype) for x, y in cache.items()}
    ref, tol = plain_attention(clean, q, table, cu, lens, 1 / math.sqrt(d), window)
    check_attention(tq.kv8_attn_prefill(cache, q, *args, window=window), ref, tol)
    last = [c - 1 for c in cu[1:]]
    check_attention(tq.kv8_attn_decode(cache, q[last], args[0], args[2], window=window), ref[last], tol[last])


@pytest.mark.gpu
@pytest.mark.parametrize("new,past,hq,hkv,d,bs,rot,interleaved", [
    ([3000, 1], [100, 4000], 8, 4, 128, 64, 128, False),
    ([700, 900, 1300], [0, 31, 5], 6, 2, 64, 32, 32, True),
    ([1] * 200, [29 * i % 500 for i in range(200)], 16, 8, 128, 16, 64, False),
])
def test_larger_appends_of_fp32_rows(cuda, new, past, hq, hkv, d, bs, rot, interleaved):
    g = torch.Generator().manual_seed(92)
    lens, cu = [a + b for a, b in zip(new, past)], [0] + list(itertools.accumulate(new))
    table, total = pages_for(lens, bs, g)
    cache = random_cache(total, hkv, bs, d, g, cuda)
    rows = torch.randn(cu[-1], hq + 2 * hkv, d, generator=g)
    k, v, rope = rows[:, hq:hq + hkv], rows[:, hq + hkv:], tq.rope_table(table.shape[1] * bs, rot, device="cpu")
    want, exact, scale = plain_append(cache, k, v, table, cu, lens, rope, interleaved)
    x = rows.to(cuda)
    out = tq.kv8_append(cache, x[:, hq:hq + hkv], x[:, hq + hkv:], table.to(cuda), ints(cu, cuda), ints(lens, cuda),
                        q=x[:, :hq], rope=rope.to(cuda), interleaved=interleaved)
    check_append(cache, want, exact, scale)
    for b, r0, n, start in spans(cu, lens):
        part = rows[r0:r0 + n, :hq]
        ref = rotated(part, rope[start:start + n], interleaved)
        size = part.double().abs().amax(-1, keepdim=True) * 2
        assert ((out[r0:r0 + n].cpu().double() - ref).abs() <= HALF_STEP[torch.float32] * ref.abs() + 4 * 2.0 ** -24 * size).all()


@pytest.mark.gpu
def test_mixed_batches_on_two_streams_and_over_the_queries(cuda):
    """Calls that run both kernels, at once on four streams with a workspace
    each, and with the output over the queries."""
    g = torch.Generator().manual_seed(95)
    new = [1] * 50 + [400, 3, 16, 33]
    lens, cu = [c + 3000 for c in new], [0] + list(itertools.accumulate(new))
    table, total = pages_for(lens, 64, g)
    cache = random_cache(total, 4, 64, 128, g, cuda)
    q = torch.randn(cu[-1], 16, 128, generator=g).to(torch.bfloat16).to(cuda)
    args = (table.to(cuda), ints(cu, cuda), ints(lens, cuda))
    want = tq.kv8_attn_prefill(cache, q, *args)
    ref, tol = gpu_attention(cache, q, args[0], cu, lens, 1 / math.sqrt(128), 0, only=[5])
    check_attention(want[:, 5], ref[:, 5].cpu(), tol[:, 5].cpu())
    streams = [torch.cuda.Stream() for _ in range(4)]
    mine = [q.clone() for _ in streams]
    torch.cuda.synchronize()
    got = [tq.kv8_attn_prefill(cache, q, *args, stream=s) for _ in range(3) for s in streams]
    for x, s in zip(mine, streams):
        tq.kv8_attn_prefill(cache, x, *args, out=x, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got + mine)
    assert tq.tq_device_fault() == 0
