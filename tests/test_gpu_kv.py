"""The key/value cache (hqq_kv_append, hqq_kv_read, hqq_kv_attention, hqq_kv_prefix_attention)
against plain implementations in 64 bits on the host.

Append and read are defined operation by operation in binary32, so their results are compared bit
for bit.  Attention is compared with the softmax in 64 bits of the rows (code - zero) * scale.  Its
tolerance counts the roundings of the kernel, u = 2^-11 being half a step of fp16:
  * the weights p_t * scale_tg are rounded to fp16 once: an output element is off by at most
    u * sum_t p_t |v_td| / sum_t p_t;
  * a score (in powers of two) is a binary32 sum: its error is at most (D + 8) 2^-23 times
    sum_g scale_tg (sum_d |q_d| a_td + |zero_tg| |sum_d q_d|), and what the exponential (2^-22 relative)
    and the sums over n tokens add is below (n + 16) 2^-23 relative, taken on sum_t p_t |v_td|, with
    the codes and zero points summed apart: |v_td| is replaced by scale_tg (c_td + |zero_tg|);
  * the output is rounded to its type: half a step relative to itself;
  * behind a prefix with more than 64 rows on a key head, the values too are rounded to fp16 once, after a
    zero point that is off by at most 2^-17 of a step (2^-9 of one of 255): another u * |v_td| and that
    share of scale_tg.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def hqq():
    from free_weight_quantization_b200 import build
    build.build()
    assert torch.cuda.is_available(), "this test needs a CUDA device"
    from free_weight_quantization_b200 import hqq as h
    return h


F16, BF16 = torch.float16, torch.bfloat16


def element_places(D, g, pieces):
    """place[d]: the number of element d among a row's stored codes."""
    d = np.arange(D)
    run = g // pieces
    return d % g // run * (D // pieces) + d // g * run + d % run


def quantize_rows(x, nbits, g):
    """Codes (element order), scale and zero of float32 rows [.., D], step by step in binary32."""
    top = np.float32(2 ** nbits - 1)
    x = np.clip(np.where(np.isnan(x), np.float32(-65504), x), np.float32(-65504), np.float32(65504))
    x = x.reshape(*x.shape[:-1], -1, g)
    lo, hi = x.min(-1), x.max(-1)
    step = (hi - lo).astype(np.float32) / top
    least = np.maximum(np.abs(lo), np.abs(hi)) * np.float32(2.0 ** -10)
    scale = np.maximum(np.maximum(step, least), np.float32(2.0 ** -24)).astype(np.float16)
    inv = np.float32(1) / scale.astype(np.float32)
    zero = (-lo * inv).astype(np.float32).astype(np.float16)
    t = (x * inv[..., None]).astype(np.float32) + zero.astype(np.float32)[..., None]
    code = np.clip(np.rint(t), 0, top).astype(np.int64)
    return code.reshape(*code.shape[:-2], -1), scale, zero


def pack_rows(code, nbits, g, pieces):
    D = code.shape[-1]
    stored = np.empty_like(code)
    stored[..., element_places(D, g, pieces)] = code
    per = 8 // nbits
    stored = stored.reshape(*code.shape[:-1], D // per, per)
    return (stored << (nbits * np.arange(per))).sum(-1).astype(np.uint8)


def unpack_rows(data, nbits, g, pieces):
    per = 8 // nbits
    codes = (data[..., None].astype(np.int64) >> (nbits * np.arange(per))) & (2 ** nbits - 1)
    return codes.reshape(*data.shape[:-1], -1)[..., element_places(data.shape[-1] * per, g, pieces)]


def values_of(code, meta, g, dtype):
    """(code - zero) * scale in binary32, rounded to dtype."""
    m = np.repeat(meta.astype(np.float32), g, -2)
    y = (code.astype(np.float32) - m[..., 1]) * m[..., 0]
    return torch.from_numpy(y).to(dtype)


def bits(t):
    return t.cpu().view(torch.int16)


LAYOUTS = [(D, nb, g) for D in (64, 128, 256) for nb in (2, 4, 8) for g in (32, 64, 128) if g <= D]


def rows(rng, n, h, D, dtype):
    x = rng.standard_normal((n, h, D)) * np.exp(rng.standard_normal((1, h, D))) + rng.standard_normal((1, h, D))
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("D,nb,g", LAYOUTS)
def test_append_and_read_bit_exact(hqq, D, nb, g, dtype):
    rng = np.random.default_rng(D + nb + g)
    n, h, ps = 37, 3, 16
    cache = hqq.hqq_kv_cache(6, h, D, ps, nb, g)
    k, v = rows(rng, n, h, D, dtype), rows(rng, n, h, D, dtype)
    k[3] = 0.0                         # a constant group, and one far from zero with a small spread
    v[4] = 100.0 + 0.01 * torch.arange(D)
    k[5, 0, :5] = torch.tensor([math.inf, -math.inf, 60000.0, -60000.0, 0.0])
    v[6] = 2.0 ** -24 * torch.arange(D)
    v[10, 1, 3], k[11, 2, D - 1] = math.nan, math.nan
    slots = rng.permutation(6 * ps)[:n]
    slots[7], slots[8], slots[9] = -1, 6 * ps, -(2 ** 40)   # padding, and past the pool
    s = torch.from_numpy(slots).cuda()
    kv = hqq.hqq_kv_append(cache, k.cuda(), v.cuda(), s, return_values=True)
    back = hqq.hqq_kv_read(cache, s, dtype)
    there = (slots >= 0) & (slots < 6 * ps)
    for x, codes, meta, pieces, got, again in ((k, cache.k_codes, cache.k_meta, 4, kv[0], back[0]),
                                               (v, cache.v_codes, cache.v_meta, 8, kv[1], back[1])):
        code, scale, zero = quantize_rows(x.float().numpy(), nb, g)
        m = np.stack((scale, zero), -1)
        want_codes = np.zeros(tuple(codes.shape), np.uint8)
        want_meta = np.zeros(tuple(meta.shape), np.float16)
        packed = pack_rows(code, nb, g, pieces)
        for t in np.nonzero(there)[0]:
            want_codes[slots[t] // ps, :, slots[t] % ps] = packed[t]
            want_meta[slots[t] // ps, :, slots[t] % ps] = m[t]
        assert np.array_equal(codes.cpu().numpy(), want_codes)
        assert np.array_equal(meta.cpu().numpy().view(np.uint16), want_meta.view(np.uint16))
        want = values_of(code, m, g, dtype)
        want[torch.from_numpy(~there)] = 0
        assert torch.equal(bits(got), bits(want)) and torch.equal(bits(again), bits(want))


# ---------------------------------------------------------------- attention

def random_cache(hqq, rng, pages, h, D, ps, nb, g):
    cache = hqq.hqq_kv_cache(pages, h, D, ps, nb, g)
    for codes, meta in ((cache.k_codes, cache.k_meta), (cache.v_codes, cache.v_meta)):
        codes.copy_(torch.from_numpy(rng.integers(0, 256, tuple(codes.shape)).astype(np.uint8)))
        m = np.empty(tuple(meta.shape), np.float16)
        m[..., 0] = np.exp(rng.standard_normal(m.shape[:-1])) / 2 ** nb
        m[..., 1] = rng.random(m.shape[:-1]) * 2 ** nb
        meta.copy_(torch.from_numpy(m))
    return cache


def context(cache, table, count):
    """keys and values [heads, count, D] in 64 bits and, for the tolerance, scale * (code + |zero|)."""
    ps, out = cache.page_size, []
    for codes, meta, pieces in ((cache.k_codes, cache.k_meta, 4), (cache.v_codes, cache.v_meta, 8)):
        c = unpack_rows(codes.cpu().numpy(), cache.nbits, cache.group_size, pieces).astype(np.float64)
        m = np.repeat(meta.cpu().numpy().astype(np.float64), cache.group_size, -2)
        x = [(c - m[..., 1]) * m[..., 0], (c + np.abs(m[..., 1])) * m[..., 0]]
        x += [m[..., 0]] if pieces == 8 else []
        n = -(-count // ps)
        out += [np.concatenate([y[p] for p in table[:n]] or [np.zeros((cache.kv_heads, 0, cache.head_dim))], 1)[:, :count] for y in x]
    return out


def attend(cache, q, tables, lens, window=0, prefix=(None, 0), scale=None, hidden=None):
    """out, lse and the error bound of out before its rounding, all in 64 bits.  hidden[b]: tokens of
    sequence b that are not seen whatever their place."""
    rounded = prefix[1] > 0 and q.shape[0] * q.shape[1] * q.shape[2] // cache.kv_heads > 64
    step = 2.0 ** -9 if cache.nbits == 8 else 2.0 ** -17
    B, nq, H, D = q.shape
    share = H // cache.kv_heads
    scale = D ** -0.5 if scale is None else scale
    out, lse, tol = np.zeros((B, nq, H, D)), np.full((B, nq, H), -np.inf), np.zeros((B, nq, H, D))
    head = context(cache, *prefix) if prefix[1] else None
    for b in range(B):
        own = max(int(lens[b]), 0)
        ctx = context(cache, tables[b], own)
        if head is not None:
            ctx = [np.concatenate((x, y), 1) for x, y in zip(head, ctx)]
        k, ka, v, va, vs = ctx
        n = k.shape[1]
        for i in range(nq):
            at = n - nq + i
            seen = np.arange(n) <= at
            if window:
                seen &= np.arange(n) > at - window
            if hidden is not None:
                seen &= ~hidden[b][:n]
            if not seen.any():
                continue
            for h in range(H):
                kv = h // share
                qv = q[b, i, h].astype(np.float64)
                s = scale * (k[kv][seen] @ qv)
                es = scale * (ka[kv][seen] @ np.abs(qv)) * (D + 8) * 2.0 ** -23  # error of a score
                m = s.max()
                p = np.exp(s - m)
                lse[b, i, h] = m + np.log(p.sum())
                p /= p.sum()
                out[b, i, h] = p @ v[kv][seen]
                mag = p @ np.abs(v[kv][seen])
                both = p @ va[kv][seen]
                tol[b, i, h] = 2.0 ** -11 * mag + (p * 2 * es) @ va[kv][seen] + 2 * (p @ es) * both \
                    + (seen.sum() + 32) * 2.0 ** -23 * both
                if rounded:
                    tol[b, i, h] += 2.0 ** -11 * mag + p @ vs[kv][seen] * step
    return out, lse, tol


def check(got, lse_got, want, label=""):
    out, lse, tol = want
    half = torch.finfo(got.dtype).eps / 2
    y = got.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(y).all(), label
    bound = tol * (1 + half) + half * np.abs(out) + 2.0 ** -25
    bad = np.abs(y - out) / bound
    assert (bad <= 1).all(), (label, float(bad.max()))
    z = lse_got.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isinf(z), np.isinf(lse)) and (z[np.isinf(z)] < 0).all(), label
    fine = np.isfinite(lse)
    assert (np.abs(z[fine] - lse[fine]) <= 2e-5 * np.maximum(1, np.abs(lse[fine]))).all(), label


def tables_of(rng, pages, lens, ps, wide):
    order = rng.permutation(pages)
    t, at = np.zeros((len(lens), wide), np.int32), 0
    for b, n in enumerate(lens):
        used = -(-max(n, 0) // ps)
        t[b, :used] = order[at:at + used]
        at += used
    assert at <= pages
    return t


@pytest.mark.parametrize("D,nb,g", LAYOUTS)
def test_attention_layouts(hqq, D, nb, g):
    # every layout, both types, rows of one and of several query heads, lengths around a step of 16
    rng = np.random.default_rng(D * nb + g)
    lens, ps, h = [33, 1, 16, 0, 130], 16, 2
    cache = random_cache(hqq, rng, 16, h, D, ps, nb, g)
    t = tables_of(rng, 16, lens, ps, 9)
    for dtype, heads in ((F16, 2), (BF16, 6)):
        q = torch.from_numpy(rng.standard_normal((len(lens), 1, heads, D)).astype(np.float32)).to(dtype)
        out, lse = hqq.hqq_kv_attention(cache, q.cuda(), torch.from_numpy(t).cuda(),
                                        torch.tensor(lens, dtype=torch.int32).cuda(), return_lse=True)
        check(out, lse, attend(cache, q.float().numpy(), t, lens), (dtype, heads))


# (batch lengths, queries, heads, key heads, page size, window)
CASES = [([1], 1, 1, 1, 16, 0), ([700, 3], 1, 8, 1, 64, 0), ([257, 64, 65, 31], 3, 10, 2, 32, 0),
         ([5, 2, 0, 4], 4, 4, 4, 16, 0), ([2, 300, 90], 5, 15, 3, 64, 0), ([2000], 1, 20, 1, 128, 0),
         ([1, 40, 333, 600], 1, 4, 1, 16, 37), ([1200, 16, 17], 7, 6, 2, 32, 100), ([129], 33, 4, 2, 16, 0),
         ([520], 1, 2, 2, 1024, 1), ([900], 2, 4, 4, 256, 5000)]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("lens,nq,heads,kv,ps,window", CASES)
def test_attention_cases(hqq, lens, nq, heads, kv, ps, window, dtype):
    rng = np.random.default_rng(sum(lens) + nq)
    wide = -(-max(lens) // ps) + 1
    pages = sum(-(-n // ps) for n in lens) + 2
    cache = random_cache(hqq, rng, pages, kv, 128, ps, 4, 64)
    t = tables_of(rng, pages, lens, ps, wide)
    q = torch.from_numpy(2 * rng.standard_normal((len(lens), nq, heads, 128)).astype(np.float32)).to(dtype)
    out, lse = hqq.hqq_kv_attention(cache, q.cuda(), torch.from_numpy(t).cuda(),
                                    torch.tensor(lens, dtype=torch.int32).cuda(), window=window, return_lse=True)
    check(out, lse, attend(cache, q.float().numpy(), t, lens, window))


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("prefix,lens,nq,heads,kv,D", [
    (100, [1, 40, 7], 1, 8, 2, 128), (1, [3, 1], 1, 2, 2, 128), (64, [0, 5, 200], 1, 4, 1, 64),
    (1000, [2, 30, 17, 9, 64], 2, 20, 4, 128), (333, [0, 1, 2, 50], 3, 6, 3, 128), (700, [20] * 9, 1, 5, 1, 256),
    (515, [9] * 40, 1, 8, 1, 128)])
def test_prefix_attention(hqq, prefix, lens, nq, heads, kv, D, dtype):
    rng = np.random.default_rng(prefix + nq)
    ps = 32
    shared = -(-prefix // ps)
    pages = shared + sum(-(-n // ps) for n in lens) + 1
    cache = random_cache(hqq, rng, pages, kv, D, ps, 4, 64)
    t = tables_of(rng, pages - shared, lens, ps, -(-max(lens) // ps)) + shared
    pt = rng.permutation(shared).astype(np.int32)
    q = torch.from_numpy(2 * rng.standard_normal((len(lens), nq, heads, D)).astype(np.float32)).to(dtype)
    out, lse = hqq.hqq_kv_prefix_attention(cache, q.cuda(), torch.from_numpy(pt).cuda(), prefix,
                                           torch.from_numpy(t).cuda(),
                                           torch.tensor(lens, dtype=torch.int32).cuda(), return_lse=True)
    check(out, lse, attend(cache, q.float().numpy(), t, lens, prefix=(pt, prefix)))


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("D,g", [(128, 64), (128, 128), (64, 64), (64, 32), (128, 32)])
@pytest.mark.parametrize("nb", [2, 4, 8])
def test_prefix_of_many_rows(hqq, D, g, nb, dtype):
    # two tiles of 128 rows, the second ragged; the prefix ends inside a tile of 64 tokens and a page;
    # some sequences shorter than their queries, some without tokens; a page that is not there
    rng = np.random.default_rng(D + g + nb)
    B, nq, heads, kv, ps, prefix = 23, 2, 6, 1, 16, 333
    lens = [int(n) for n in rng.integers(0, 40, B)]
    shared = -(-prefix // ps)
    pages = shared + sum(-(-n // ps) for n in lens) + 1
    cache = random_cache(hqq, rng, pages, kv, D, ps, nb, g)
    t = tables_of(rng, pages - shared, lens, ps, 3) + shared
    pt = rng.permutation(shared).astype(np.int32)
    q = torch.from_numpy(2 * rng.standard_normal((B, nq, heads, D)).astype(np.float32)).to(dtype)
    args = (q.cuda(), torch.from_numpy(pt).cuda(), prefix, torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    out, lse = hqq.hqq_kv_prefix_attention(cache, *args, return_lse=True)
    check(out, lse, attend(cache, q.float().numpy(), t, lens, prefix=(pt, prefix)))
    gone = pt.copy()
    gone[3], gone[-1] = -1, pages
    out, lse = hqq.hqq_kv_prefix_attention(cache, args[0], torch.from_numpy(gone).cuda(), *args[2:], return_lse=True)
    hidden = [np.zeros(prefix + max(n, 0), bool) for n in lens]
    for x in hidden:
        x[3 * ps:4 * ps] = x[(shared - 1) * ps:prefix] = True
    check(out, lse, attend(cache, q.float().numpy(), t, lens, prefix=(pt, prefix), hidden=hidden))


def test_prefix_equals_one_long_sequence(hqq):
    # the same tokens by both calls: the prefix's pages in front of each sequence's own
    rng = np.random.default_rng(3)
    B, ps, prefix, kv, heads, D = 12, 32, 320, 2, 8, 128
    lens = [int(n) for n in rng.integers(1, 100, B)]
    pages = prefix // ps + sum(-(-n // ps) for n in lens)
    cache = random_cache(hqq, rng, pages, kv, D, ps, 4, 64)
    pt = rng.permutation(prefix // ps).astype(np.int32)
    t = tables_of(rng, pages - len(pt), lens, ps, 4) + len(pt)
    whole = np.concatenate((np.repeat(pt[None], B, 0), t), 1).astype(np.int32)
    q = torch.randn(B, 1, heads, D, device="cuda").half()
    a, la = hqq.hqq_kv_prefix_attention(cache, q, torch.from_numpy(pt).cuda(), prefix, torch.from_numpy(t.astype(np.int32)).cuda(),
                                        torch.tensor(lens, dtype=torch.int32).cuda(), return_lse=True)
    b, lb = hqq.hqq_kv_attention(cache, q, torch.from_numpy(whole).cuda(),
                                 torch.tensor([n + prefix for n in lens], dtype=torch.int32).cuda(), return_lse=True)
    want = attend(cache, q.float().cpu().numpy(), t, lens, prefix=(pt, prefix))
    check(a, la, want)
    check(b, lb, want)


def test_many_ragged_sequences(hqq):
    # more sequences than threads of a CTA, lengths that share CTAs and that span several
    rng = np.random.default_rng(4)
    B, ps, kv, heads, D = 300, 16, 1, 2, 64
    lens = [int(n) for n in rng.integers(0, 60, B)]
    lens[7], lens[150], lens[299] = 3000, 0, 1111
    pages = sum(-(-n // ps) for n in lens)
    cache = random_cache(hqq, rng, pages, kv, D, ps, 4, 32)
    t = tables_of(rng, pages, lens, ps, -(-3000 // ps))
    q = torch.randn(B, 1, heads, D, device="cuda").to(BF16)
    run = lambda: hqq.hqq_kv_attention(cache, q, torch.from_numpy(t).cuda(),  # noqa: E731
                                       torch.tensor(lens, dtype=torch.int32).cuda(), return_lse=True)
    out, lse = run()
    check(out, lse, attend(cache, q.float().cpu().numpy(), t, lens))
    for _ in range(3):   # joined in a fixed order: the same bits again
        again, lse2 = run()
        assert torch.equal(bits(again), bits(out)) and torch.equal(lse2, lse)


def test_what_is_not_seen_does_not_matter(hqq):
    # rows behind the last token, pages before the window and pages of nobody hold NaN and garbage;
    # page numbers outside the pool are not seen; lengths are cut to the table and to max_len
    rng = np.random.default_rng(5)
    D, ps, kv, heads, window = 128, 16, 2, 4, 40
    lens = [100, 17, 700]
    cache = random_cache(hqq, rng, 80, kv, D, ps, 4, 64)
    t = tables_of(rng, 80, lens, ps, 44)
    used = np.zeros((80, ps), bool)
    for b, n in enumerate(lens):
        for tok in range(max(0, n - window), n):
            used[t[b, tok // ps], tok % ps] = True
    q = torch.randn(3, 1, heads, D, device="cuda").half()
    tc, lc = torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    want = hqq.hqq_kv_attention(cache, q, tc, lc, window=window, return_lse=True)
    keep = torch.from_numpy(used).cuda()[:, None, :, None, None]
    for meta in (cache.k_meta, cache.v_meta):
        meta.copy_(torch.where(keep, meta, torch.full_like(meta, math.nan)))
    got = hqq.hqq_kv_attention(cache, q, tc, lc, window=window, return_lse=True)
    assert torch.equal(bits(got[0]), bits(want[0])) and torch.equal(got[1], want[1])

    cache = random_cache(hqq, rng, 80, kv, D, ps, 4, 64)
    bad = t.copy()
    bad[0, 2], bad[2, 0], bad[2, 9] = -5, 80, 2 ** 31 - 1
    hidden = [np.zeros(n, bool) for n in lens]
    hidden[0][2 * ps:3 * ps] = hidden[2][:ps] = hidden[2][9 * ps:10 * ps] = True
    out, lse = hqq.hqq_kv_attention(cache, q, torch.from_numpy(bad).cuda(), lc, return_lse=True)
    check(out, lse, attend(cache, q.float().cpu().numpy(), t, lens, hidden=hidden))
    # past max_len, and below zero
    cut = torch.tensor([2 ** 31 - 1, -3, 120], dtype=torch.int32).cuda()
    out, lse = hqq.hqq_kv_attention(cache, q, tc, cut, max_len=96, return_lse=True)
    check(out, lse, attend(cache, q.float().cpu().numpy(), t, [96, 0, 96]))


def test_strided_and_unaligned_inputs(hqq):
    # queries, keys and values as slices of one fused product; then shifted by one value
    rng = np.random.default_rng(6)
    B, heads, kv, D, ps = 3, 4, 2, 128, 16
    fused = torch.randn(B, 1, heads + 2 * kv, D, device="cuda").to(BF16)
    for shift in (0, 1):
        if shift:
            flat = torch.empty(fused.numel() + 1, dtype=BF16, device="cuda")
            flat[1:] = fused.flatten()
            f = flat[1:].view_as(fused)
        else:
            f = fused
        q, k, v = f[:, :, :heads], f[:, 0, heads:heads + kv], f[:, 0, heads + kv:]
        cache = hqq.hqq_kv_cache(8, kv, D, ps, 4, 64)
        slots = torch.tensor([5, 40, 99], device="cuda")
        hqq.hqq_kv_append(cache, k, v, slots)
        kr, vr = hqq.hqq_kv_read(cache, slots, BF16)
        other = hqq.hqq_kv_cache(8, kv, D, ps, 4, 64)
        kc, vc = hqq.hqq_kv_append(other, k.contiguous(), v.contiguous(), slots, return_values=True)
        assert torch.equal(bits(kr), bits(kc)) and torch.equal(bits(vr), bits(vc))
        assert torch.equal(cache.k_codes, other.k_codes) and torch.equal(cache.v_codes, other.v_codes)
        table = torch.tensor([[0, 9, 9], [2, 1, 9], [6, 2, 9]], dtype=torch.int32, device="cuda")[:, :2]  # rows 3 apart
        lens = torch.tensor([6, 25, 20], dtype=torch.int32, device="cuda")
        a = hqq.hqq_kv_attention(cache, q, table, lens)
        b = hqq.hqq_kv_attention(cache, q.contiguous(), table.contiguous(), lens)
        assert torch.equal(bits(a), bits(b))
        pa = hqq.hqq_kv_prefix_attention(cache, q.expand(B, 40, heads, D), table[0].contiguous(), 9, table, lens)
        pb = hqq.hqq_kv_prefix_attention(cache, q.expand(B, 40, heads, D).contiguous(), table[0].contiguous(), 9, table, lens)
        assert torch.equal(bits(pa), bits(pb))


def test_decoding_as_a_run(hqq):
    # a prompt appended at once, then token by token: append and attend, against plain attention of the
    # values that the appends returned
    rng = np.random.default_rng(7)
    B, heads, kv, D, ps, prompt, steps = 2, 8, 2, 128, 16, 30, 5
    cache = hqq.hqq_kv_cache(16, kv, D, ps, 8, 64)
    table = torch.from_numpy(rng.permutation(16)[:B * 4].reshape(B, 4).astype(np.int32)).cuda()
    slots_of = lambda b, t: int(table[b, t // ps]) * ps + t % ps  # noqa: E731
    ks, vs = [[] for _ in range(B)], [[] for _ in range(B)]
    for step in range(-1, steps):
        toks = range(prompt) if step < 0 else [prompt + step]
        k, v = (torch.randn(B * len(toks), kv, D, device="cuda").to(BF16) for _ in range(2))
        s = torch.tensor([slots_of(b, t) for b in range(B) for t in toks], device="cuda")
        kh, vh = hqq.hqq_kv_append(cache, k, v, s, return_values=True)
        for b in range(B):
            ks[b] += list(kh[b * len(toks):(b + 1) * len(toks)].double())
            vs[b] += list(vh[b * len(toks):(b + 1) * len(toks)].double())
        if step < 0:
            continue
        n = prompt + step + 1
        q = torch.randn(B, 1, heads, D, device="cuda").to(BF16)
        out, lse = hqq.hqq_kv_attention(cache, q, table, torch.full((B,), n, dtype=torch.int32, device="cuda"), return_lse=True)
        for b in range(B):
            K, V = torch.stack(ks[b]).repeat_interleave(heads // kv, 1), torch.stack(vs[b]).repeat_interleave(heads // kv, 1)
            sc = torch.einsum("hd,thd->ht", q[b, 0].double(), K) * D ** -0.5
            want = torch.einsum("ht,thd->hd", sc.softmax(-1), V)
            # the returned values are rounded to bf16: a relative 2^-8 on each key and value beside the output's own
            es = torch.einsum("hd,thd->ht", q[b, 0].double().abs(), K.abs()).amax(-1)[:, None] * D ** -0.5 * 2.0 ** -8
            tol = torch.einsum("ht,thd->hd", sc.softmax(-1), V.abs()) * (2.0 ** -8 + 2 * es + 2.0 ** -10) + want.abs() * 2.0 ** -8
            assert ((out[b, 0].double() - want).abs() <= tol).all()
            assert ((lse[b, 0].double() - torch.logsumexp(sc, -1)).abs() <= es[:, 0] + 1e-5).all()


def test_graphs_streams_and_empty_calls(hqq):
    rng = np.random.default_rng(8)
    D, ps, kv, heads, B = 128, 16, 2, 8, 4
    cache = random_cache(hqq, rng, 400, kv, D, ps, 4, 64)
    t = torch.from_numpy(rng.permutation(400)[:B * 90].reshape(B, 90).astype(np.int32)).cuda()
    lens = torch.tensor([1400, 3, 900, 64], dtype=torch.int32, device="cuda")
    q = torch.randn(B, 1, heads, D, device="cuda").half()
    pt = t[0, :7].contiguous()
    calls = [lambda **k: hqq.hqq_kv_attention(cache, q, t, lens, return_lse=True, **k),
             lambda **k: hqq.hqq_kv_prefix_attention(cache, q, pt, 101, t, lens, return_lse=True, **k),
             lambda **k: hqq.hqq_kv_prefix_attention(cache, q.expand(B, 1, heads, D).repeat(1, 9, 1, 1), pt, 101, t, lens, return_lse=True, **k)]
    for call in calls:
        want = call()
        graphs, results = [], []
        for _ in range(2):  # two graphs live at once, each with its own workspace
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                results.append(call())
            graphs.append(g)
        lens.copy_(torch.tensor([64, 1300, 0, 5], dtype=torch.int32))   # lengths are read when it runs
        other = call()
        for g in graphs:
            g.replay()
        for r in results:
            assert torch.equal(bits(r[0]), bits(other[0])) and torch.equal(r[1], other[1])
        lens.copy_(torch.tensor([1400, 3, 900, 64], dtype=torch.int32))
        graphs[0].replay()
        assert torch.equal(bits(results[0][0]), bits(want[0])) and torch.equal(results[0][1], want[1])
        # two streams at once
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        got = [call(stream=s) for s in streams for _ in range(3)]
        torch.cuda.synchronize()
        for r in got:
            assert torch.equal(bits(r[0]), bits(want[0])) and torch.equal(r[1], want[1])
        # a workspace and an output of the caller's
        ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(want[0])
        r = call(workspace=ws, out=out)
        assert r[0] is out and torch.equal(bits(out), bits(want[0]))
    with pytest.raises(hqq.HqqError, match="workspace"):
        hqq.hqq_kv_attention(cache, q, t, lens, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    # nothing to do
    none = hqq.hqq_kv_attention(cache, q[:0], t[:0], lens[:0])
    assert none.shape == (0, 1, heads, D)
    assert hqq.hqq_kv_attention(cache, q[:, :0], t, lens).shape == (B, 0, heads, D)
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    assert hqq.hqq_kv_read(cache, slots)[0].shape == (0, kv, D)
    hqq.hqq_kv_append(cache, q[:0, 0, :kv], q[:0, 0, :kv], slots)
    # an empty prefix
    a = hqq.hqq_kv_prefix_attention(cache, q, pt[:0], 0, t, lens, return_lse=True)
    b = hqq.hqq_kv_attention(cache, q, t, lens, return_lse=True)
    assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(a[1], b[1])
    # an empty table: nothing is seen
    out, lse = hqq.hqq_kv_attention(cache, q, t[:, :0], lens, return_lse=True)
    assert not out.any() and torch.isinf(lse).all()


def test_offsets_past_32_bits(hqq):
    # 5.2 GB of codes for keys and for values; everything in the last pages of the pool
    pages, kv, D, ps = 40000, 2, 256, 256
    cache = hqq.hqq_kv_cache(pages, kv, D, ps, 8, 128)
    assert cache.k_codes.numel() > 2 ** 32
    n = 300
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    slots = torch.cat([int(p) * ps + torch.arange(ps) for p in table[0].tolist()])[:n].cuda()
    k, v = (torch.randn(n, kv, D, device="cuda").to(BF16) for _ in range(2))
    hqq.hqq_kv_append(cache, k, v, slots)
    small = hqq.hqq_kv_cache(2, kv, D, ps, 8, 128)
    hqq.hqq_kv_append(small, k, v, torch.arange(n, device="cuda"))
    a, b = hqq.hqq_kv_read(cache, slots, BF16), hqq.hqq_kv_read(small, torch.arange(n, device="cuda"), BF16)
    assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(bits(a[1]), bits(b[1]))
    q = torch.randn(1, 1, 4, D, device="cuda").to(BF16)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    x = hqq.hqq_kv_attention(cache, q, table, lens)
    y = hqq.hqq_kv_attention(small, q, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), lens)
    assert torch.equal(bits(x), bits(y))


def test_binding_refuses(hqq):
    cache = hqq.hqq_kv_cache(4, 2, 128)
    q = torch.randn(2, 1, 4, 128, device="cuda").half()
    t = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    k = torch.randn(2, 2, 128, device="cuda").half()
    bad = [lambda: hqq.hqq_kv_attention(cache, q.float(), t, lens), lambda: hqq.hqq_kv_attention(cache, q.cpu(), t, lens),
           lambda: hqq.hqq_kv_attention(cache, q[:, :, :3], t, lens), lambda: hqq.hqq_kv_attention(cache, q[..., :64], t, lens),
           lambda: hqq.hqq_kv_attention(cache, q, t.long(), lens), lambda: hqq.hqq_kv_attention(cache, q, t[:1], lens),
           lambda: hqq.hqq_kv_attention(cache, q, t, lens.long()), lambda: hqq.hqq_kv_attention(cache, q, t, lens[:1]),
           lambda: hqq.hqq_kv_attention(cache, q, t, lens, max_len=129), lambda: hqq.hqq_kv_attention(cache, q, t, lens, window=-1),
           lambda: hqq.hqq_kv_attention(cache, q, t, lens, scale=0.0), lambda: hqq.hqq_kv_attention(cache, q, t, lens, out=q[:1]),
           lambda: hqq.hqq_kv_attention(cache, q.transpose(2, 3).contiguous().transpose(2, 3), t, lens),
           lambda: hqq.hqq_kv_prefix_attention(cache, q, t[0], 129, t, lens), lambda: hqq.hqq_kv_prefix_attention(cache, q, t, 1, t, lens),
           lambda: hqq.hqq_kv_append(cache, k, k.to(BF16), slots), lambda: hqq.hqq_kv_append(cache, k[:1], k, slots),
           lambda: hqq.hqq_kv_append(cache, k, k, slots.int()), lambda: hqq.hqq_kv_append(cache, k.cpu(), k, slots),
           lambda: hqq.hqq_kv_read(cache, slots, torch.float32), lambda: hqq.hqq_kv_read(cache, slots, out=(k[:1], k))]
    for call in bad:
        with pytest.raises(hqq.HqqError):
            call()
