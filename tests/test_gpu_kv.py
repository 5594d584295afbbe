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
  * the output is rounded to its type: half a step relative to itself.
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
        n = -(-count // ps)
        out += [np.concatenate([y[p] for p in table[:n]] or [np.zeros((cache.kv_heads, 0, cache.head_dim))], 1)[:, :count] for y in x]
    return out


def attend(cache, q, tables, lens, window=0, prefix=(None, 0), scale=None, hidden=None):
    """out, lse and the error bound of out before its rounding, all in 64 bits."""
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
        k, ka, v, va = ctx
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
