"""The key/value cache's calls at the ends of their ranges, against the 64-bit forms and the tolerances
of test_gpu_kv.py."""
import sys
from types import SimpleNamespace

import numpy as np
import pytest

from test_gpu_kv import BF16, F16, LAYOUTS, attend, bits, check, context, hqq, random_cache, tables_of  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def attend_prefix(cache, q, table, count):
    """What test_gpu_kv's attend() computes, for rows that all see `count` tokens of one table: many rows
    at once, in 64 bits on the GPU."""
    B, nq, H, D = q.shape
    kv, share = cache.kv_heads, H // cache.kv_heads
    k, ka, v, va, vs = (torch.from_numpy(x).cuda() for x in context(cache, table, count))
    rows = q.double().view(B, nq, kv, share, D).permute(2, 0, 1, 3, 4).reshape(kv, -1, D) * D ** -0.5
    s = rows @ k.transpose(1, 2)
    es = (rows.abs() @ ka.transpose(1, 2)) * (D + 8) * 2.0 ** -23
    lse = s.logsumexp(-1)
    p = (s - lse[..., None]).exp()
    out, mag, both = p @ v, p @ v.abs(), p @ va
    step = 2.0 ** -9 if cache.nbits == 8 else 2.0 ** -17
    tol = 2.0 ** -11 * mag + (p * 2 * es) @ va + 2 * (p * es).sum(-1, keepdim=True) * both + (count + 32) * 2.0 ** -23 * both
    tol += 2.0 ** -11 * mag + (p @ vs) * step

    def back(x):
        return x.view(kv, B, nq, share, -1).permute(1, 2, 0, 3, 4).reshape(B, nq, H, -1).cpu().numpy()
    return back(out), back(lse[..., None])[..., 0], back(tol)


@pytest.mark.parametrize("D,g", [(128, 64), (128, 128), (64, 64)])
@pytest.mark.parametrize("nb", [2, 4, 8])
def test_prefix_value_scales_grow(hqq, D, g, nb):  # noqa: F811
    # each tile of 64 tokens has value scales about twice those of the one before, so that every tile of a
    # chunk has a unit of its own: a producer warp that took another tile's would be wrong by that factor
    rng = np.random.default_rng(D + g + nb)
    B, heads, kv, ps, prefix = 40, 160, 8, 64, 3000
    pages = -(-prefix // ps)
    cache = random_cache(hqq, rng, pages, kv, D, ps, nb, g)
    pt = rng.permutation(pages).astype(np.int32)
    grow = np.empty(pages, np.float32)
    grow[pt] = 2.0 ** (np.arange(pages) % 12 - 6)       # a page is a tile
    cache.v_meta[..., 0] *= torch.from_numpy(grow).cuda()[:, None, None, None].half()
    q = torch.from_numpy((0.5 * rng.standard_normal((B, 1, heads, D))).astype(np.float32)).cuda().to(F16)
    table = torch.zeros(B, 0, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")

    def run():
        return hqq.hqq_kv_prefix_attention(cache, q, torch.from_numpy(pt).cuda(), prefix, table, lens, return_lse=True)
    out, lse = run()
    check(out, lse, attend_prefix(cache, q, pt, prefix))
    for _ in range(20):
        again, lse2 = run()
        assert torch.equal(bits(again), bits(out)) and torch.equal(lse2, lse)


@pytest.mark.parametrize("lens", [[4000, 3, 700], [600, 1]])
def test_windows_that_hide_nothing(hqq, lens):  # noqa: F811
    # one plan with shared CTAs, one with a CTA a pair; "no limit" as a number, up to the largest
    rng = np.random.default_rng(len(lens))
    ps, kv, heads, D = 64, 2, 8, 128
    wide = -(-max(lens) // ps)
    pages = sum(-(-n // ps) for n in lens)
    cache = random_cache(hqq, rng, pages, kv, D, ps, 4, 64)
    t = tables_of(rng, pages, lens, ps, wide)
    q = torch.from_numpy(rng.standard_normal((len(lens), 3, heads, D)).astype(np.float32)).cuda().to(F16)
    tc, lc = torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    want = hqq.hqq_kv_attention(cache, q, tc, lc, return_lse=True)
    check(*want, attend(cache, q.float().cpu().numpy(), t, lens))
    for window in (wide * ps, 2 ** 31 - 1, 2 ** 31, sys.maxsize - 20, sys.maxsize, 2 ** 64 + 5):
        got = hqq.hqq_kv_attention(cache, q, tc, lc, window=window, return_lse=True)
        assert torch.equal(bits(got[0]), bits(want[0])) and torch.equal(got[1], want[1]), window
    for window in (wide * ps - 1, max(lens) - 1):   # the largest that hide something, or might
        got = hqq.hqq_kv_attention(cache, q, tc, lc, window=window, return_lse=True)
        check(*got, attend(cache, q.float().cpu().numpy(), t, lens, window))


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("path", ["own", "shared", "prefix", "many rows"])
def test_a_row_that_is_not_finite_is_nan(hqq, path, dtype):  # noqa: F811
    # on every path (one CTA a pair, cut pairs, a prefix of few rows, of many): such a row is NaN where it
    # sees a token, and the other rows are what they are beside finite rows.  Without zero points an infinity in q makes every
    # score the same infinity, which must not look like a hidden token
    rng = np.random.default_rng(5)
    D, ps, kv, heads = 128, 16, 2, 8
    lens = {"shared": [2500, 1, 700, 40], "own": [500, 1, 30, 40]}.get(path, [30, 1, 70, 4])
    B, nq = len(lens), 10 if path == "many rows" else 3
    shared = -(-333 // ps) if path not in ("own", "shared") else 0
    pages = shared + sum(-(-n // ps) for n in lens)
    cache = random_cache(hqq, rng, pages, kv, D, ps, 8, 64)
    cache.k_meta[..., 1] = 0
    t = tables_of(rng, pages - shared, lens, ps, -(-max(lens) // ps)) + shared
    tc, lc = torch.from_numpy(t.astype(np.int32)).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    pt = torch.from_numpy(rng.permutation(shared).astype(np.int32)).cuda()

    def run(x):
        if shared:
            return hqq.hqq_kv_prefix_attention(cache, x, pt, 333, tc, lc, return_lse=True)
        return hqq.hqq_kv_attention(cache, x, tc, lc, return_lse=True)
    q = torch.from_numpy(rng.standard_normal((B, nq, heads, D)).astype(np.float32)).cuda().to(dtype)
    want, lse = run(q)
    assert torch.isfinite(want).all()
    bad, x = torch.zeros(B, nq, heads, dtype=torch.bool, device="cuda"), q.clone()
    # rows (0, 0) of the sequence of one token see nothing of their own (and all but 2 of a prefix)
    for (b, i, h), d, what in (((0, 0, 0), 3, np.nan), ((0, nq - 1, 5), 127, np.inf), ((2, 1, 2), 64, -np.inf), ((3, 2, 7), 0, np.nan),
                               ((3, 0, 4), 1, -np.inf), ((1, nq - 1, 3), 9, np.inf), ((1, 0, 1), 70, np.nan), ((2, 2, 6), 0, np.inf)):
        x[b, i, h, d] = what
        bad[b, i, h] = True
    x[2, 2, 6, 1] = -np.inf      # both infinities
    x[0, 0, 1], bad[0, 0, 1] = np.nan, True
    got, lse2 = run(x)
    sees = ~torch.isinf(lse)
    assert (bad & ~sees).any() == (not shared)
    assert torch.isnan(got[bad & sees]).all() and torch.isnan(lse2[bad & sees]).all()
    # The others to their tolerance, not to the bit: the rows of a block move their running maxima together,
    # when any of them asks for it, and a weight exp(s - m) is rounded to fp16 whatever m is, so that a
    # row's last bit depends on when the rows beside it asked.  A NaN asks for nothing.
    got[bad & sees], lse2[bad & sees] = want[bad & sees], lse[bad & sees]
    check(got, lse2, attend(cache, q.float().cpu().numpy(), t, lens, prefix=(pt.cpu().numpy(), 333) if shared else (None, 0)))


@pytest.mark.parametrize("apart", [14, 20])
@pytest.mark.parametrize("path", ["own", "shared", "prefix", "many rows"])
@pytest.mark.parametrize("D,nb,g", [(128, 4, 64), (128, 2, 32), (256, 8, 32), (64, 4, 32)])
def test_groups_of_far_apart_value_scales(hqq, D, nb, g, path, apart):  # noqa: F811
    # the groups of a value keep their accuracy beside one whose scales are 2^14 or 2^20 larger, for tokens
    # of small weight too (scores spread over some 2^20): each group has a unit of its own
    rng = np.random.default_rng(D + nb + apart)
    ps, kv, heads = 16, 2, 8
    lens = {"shared": [2500, 700], "own": [500, 30]}.get(path, [30, 1, 70, 4])
    B, nq = len(lens), 10 if path == "many rows" else 1
    prefix = 700 if path not in ("own", "shared") else 0
    shared = -(-prefix // ps)
    pages = shared + sum(-(-n // ps) for n in lens)
    cache = random_cache(hqq, rng, pages, kv, D, ps, nb, g)
    up = torch.arange(D // g, device="cuda") % 2 * apart - apart + 9.0
    cache.v_meta[..., 0] = (cache.v_meta[..., 0].float() * 2.0 ** up).clamp(2.0 ** -24, 2.0 ** 15).half()
    t = tables_of(rng, pages - shared, lens, ps, -(-max(lens) // ps)) + shared
    tc, lc = torch.from_numpy(t.astype(np.int32)).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    pt = rng.permutation(shared).astype(np.int32)
    q = torch.from_numpy((3 * rng.standard_normal((B, nq, heads, D))).astype(np.float32)).cuda().to(BF16)
    if shared:
        out, lse = hqq.hqq_kv_prefix_attention(cache, q, torch.from_numpy(pt).cuda(), prefix, tc, lc, return_lse=True)
    else:
        out, lse = hqq.hqq_kv_attention(cache, q, tc, lc, return_lse=True)
    check(out, lse, attend(cache, q.float().cpu().numpy(), t, lens, prefix=(pt, prefix) if shared else (None, 0)))


@pytest.mark.parametrize("path", ["own", "shared", "prefix", "many rows"])
@pytest.mark.parametrize("big,scale,nan", [
    (2.0 ** 99, 2.0 ** -97, False), (2.0 ** 13, 1.0, False), (2.0 ** 40, 1.0, True), (2.0 ** 60, 1.0, True), (2.0 ** 101, 2.0 ** -99, True), (2.0 ** 90, 1.0, True),
    (2.0 ** 110, 0.1, True), (1e-20, 1e-30, False), (2.0 ** -120, 2.0 ** -140, False), (1e-30, 2e33, False)])
def test_range_of_queries_and_scales(hqq, path, big, scale, nan):  # noqa: F811
    # rows as large and as small as bf16 has them, with scales that bring the scores to some units, to
    # one-sided extremes or to nothing.  Rows out of range are NaN, never "sees nothing"
    rng = np.random.default_rng(6)
    D, ps, kv, heads = 64, 16, 2, 4
    lens = {"shared": [1500, 1, 700], "own": [500, 1, 30]}.get(path, [30, 1, 70])
    B, nq = len(lens), 14 if path == "many rows" else 3
    prefix = 200 if path not in ("own", "shared") else 0
    shared = -(-prefix // ps)
    pages = shared + sum(-(-n // ps) for n in lens)
    cache = random_cache(hqq, rng, pages, kv, D, ps, 4, 64)
    cache.k_meta[..., 1] = 0        # keys of one sign: the scores of a row have one too
    t = tables_of(rng, pages - shared, lens, ps, -(-max(lens) // ps)) + shared
    tc, lc = torch.from_numpy(t.astype(np.int32)).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    pt = rng.permutation(shared).astype(np.int32)
    q = np.abs(rng.standard_normal((B, nq, heads, D))) / 4
    q[:, :, 1::2] *= -1
    q[..., 5] = np.sign(q[..., 5])  # the largest magnitude
    q = np.clip(q, -1, 1)
    x = torch.from_numpy((q * big).astype(np.float32)).cuda().to(BF16)
    if shared:
        out, lse = hqq.hqq_kv_prefix_attention(cache, x, torch.from_numpy(pt).cuda(), prefix, tc, lc, scale=scale, return_lse=True)
    else:
        out, lse = hqq.hqq_kv_attention(cache, x, tc, lc, scale=scale, return_lse=True)
    want = attend(cache, x.float().cpu().numpy(), t, lens, prefix=(pt, prefix) if shared else (None, 0), scale=float(np.float32(scale)))
    if nan:
        sees = torch.from_numpy(np.isfinite(want[1])).cuda()
        assert torch.isnan(out[sees]).all() and torch.isnan(lse[sees]).all()
        assert not out[~sees].any() and torch.isneginf(lse[~sees]).all()
    else:
        check(out, lse, want)


@pytest.mark.parametrize("dtype,heads", [(F16, 2), (BF16, 6)], ids=["fp16", "bf16"])
@pytest.mark.parametrize("D,nb,g", LAYOUTS)
def test_layouts_on_shared_ctas(hqq, D, nb, g, dtype, heads):  # noqa: F811
    # every layout where CTAs share the tokens: stages used again, the page table fetched again after 32
    # blocks of a warp, pairs cut between CTAs, beside short and empty sequences
    rng = np.random.default_rng(D * nb + g)
    lens, ps, kv = [2200, 1, 16, 0, 130, 1025], 16, 2
    pages = sum(-(-n // ps) for n in lens)
    cache = random_cache(hqq, rng, pages, kv, D, ps, nb, g)
    t = tables_of(rng, pages, lens, ps, -(-2200 // ps) + 1)
    q = torch.from_numpy(rng.standard_normal((len(lens), 1, heads, D)).astype(np.float32)).cuda().to(dtype)
    out, lse = hqq.hqq_kv_attention(cache, q, torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), return_lse=True)
    check(out, lse, attend(cache, q.float().cpu().numpy(), t, lens))


@pytest.mark.parametrize("D,nb,g", [(128, 2, 64), (64, 8, 64), (256, 4, 64), (128, 4, 32)])
def test_long_own_tokens_few_ctas(hqq, D, nb, g):  # noqa: F811
    # many pairs of many units: each CTA has more than 32 blocks a warp of one pair
    rng = np.random.default_rng(D + nb)
    lens, ps, kv, heads = [int(n) for n in rng.integers(4500, 5000, 48)], 64, 8, 8
    pages = sum(-(-n // ps) for n in lens)
    cache = random_cache(hqq, rng, pages, kv, D, ps, nb, g)
    t = tables_of(rng, pages, lens, ps, -(-5000 // ps))
    q = torch.from_numpy(rng.standard_normal((len(lens), 1, heads, D)).astype(np.float32)).cuda().to(F16)
    out, lse = hqq.hqq_kv_attention(cache, q, torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), return_lse=True)
    for b in (0, 17, 47):
        one, own = slice(b, b + 1), torch.from_numpy(t[b, :-(-lens[b] // ps)]).long().cuda()
        part = SimpleNamespace(**{x: getattr(cache, x) for x in ("page_size", "nbits", "group_size", "kv_heads", "head_dim")},
                               **{x: getattr(cache, x)[own] for x in ("k_codes", "v_codes", "k_meta", "v_meta")})
        check(out[one], lse[one], attend(part, q[one].float().cpu().numpy(), np.arange(len(own))[None], lens[one]), b)


@pytest.mark.parametrize("nb", [2, 4, 8])
@pytest.mark.parametrize("B,nq,heads,kv,D,g", [(3, 2, 8, 2, 128, 64), (20, 2, 8, 1, 128, 64), (18, 1, 4, 1, 64, 64),
                                               (20, 2, 8, 1, 256, 128), (20, 2, 8, 1, 128, 32)])
def test_prefix_and_long_own_tokens(hqq, B, nq, heads, kv, D, g, nb):  # noqa: F811
    # the join finds the parts of pairs that are cut between CTAs and the prefix's, for both prefix kernels
    rng = np.random.default_rng(B + D + nb)
    ps, prefix = 32, 777
    lens = [int(n) for n in rng.integers(0, 200, B)]
    lens[1], lens[-1] = 1700, 1100
    shared = -(-prefix // ps)
    pages = shared + sum(-(-n // ps) for n in lens)
    cache = random_cache(hqq, rng, pages, kv, D, ps, nb, g)
    t = tables_of(rng, pages - shared, lens, ps, -(-1700 // ps)) + shared
    pt = rng.permutation(shared).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((B, nq, heads, D)).astype(np.float32)).cuda().to(BF16)
    out, lse = hqq.hqq_kv_prefix_attention(cache, q, torch.from_numpy(pt).cuda(), prefix, torch.from_numpy(t.astype(np.int32)).cuda(),
                                           torch.tensor(lens, dtype=torch.int32).cuda(), return_lse=True)
    check(out, lse, attend(cache, q.float().cpu().numpy(), t, lens, prefix=(pt, prefix)))


@pytest.mark.parametrize("nb,D,g", [(4, 128, 64), (2, 64, 32), (8, 256, 64)])
def test_what_is_not_seen_does_not_matter_on_shared_ctas(hqq, nb, D, g):  # noqa: F811
    # pages outside the pool, lengths that are cut, NaN behind the last token and before a window, with
    # pairs that are cut between CTAs
    rng = np.random.default_rng(nb)
    ps, kv, heads, lens, window = 16, 2, 4, [2100, 17, 1300], 1200
    pages = sum(-(-n // ps) for n in lens) + 5
    t = tables_of(rng, pages, lens, ps, 140)
    tc, lc = torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    q = torch.randn(3, 1, heads, D, device="cuda").half()
    for w in (0, window):
        cache = random_cache(hqq, rng, pages, kv, D, ps, nb, g)
        used = np.zeros((pages, ps), bool)
        for b, n in enumerate(lens):
            for tok in range(max(0, n - w) if w else 0, n):
                used[t[b, tok // ps], tok % ps] = True
        want = hqq.hqq_kv_attention(cache, q, tc, lc, window=w, return_lse=True)
        check(*want, attend(cache, q.float().cpu().numpy(), t, lens, w))
        keep = torch.from_numpy(used).cuda()[:, None, :, None, None]
        for meta in (cache.k_meta, cache.v_meta):
            meta.copy_(torch.where(keep, meta, torch.full_like(meta, np.nan)))
        got = hqq.hqq_kv_attention(cache, q, tc, lc, window=w, return_lse=True)
        assert torch.equal(bits(got[0]), bits(want[0])) and torch.equal(got[1], want[1])
    cache = random_cache(hqq, rng, pages, kv, D, ps, nb, g)
    bad = t.copy()
    bad[0, 2], bad[0, 100], bad[2, 0], bad[2, 9], bad[1, :] = -5, pages, -2 ** 31, 2 ** 31 - 1, -1
    hidden = [np.zeros(n, bool) for n in lens]
    for b, p in ((0, 2), (0, 100), (2, 0), (2, 9)):
        hidden[b][p * ps:(p + 1) * ps] = True
    hidden[1][:] = True
    out, lse = hqq.hqq_kv_attention(cache, q, torch.from_numpy(bad).cuda(), lc, return_lse=True)
    check(out, lse, attend(cache, q.float().cpu().numpy(), t, lens, hidden=hidden))
    cut = torch.tensor([2 ** 31 - 1, -3, 1250], dtype=torch.int32).cuda()
    out, lse = hqq.hqq_kv_attention(cache, q, tc, cut, max_len=1205, return_lse=True)
    check(out, lse, attend(cache, q.float().cpu().numpy(), t, [1205, 0, 1205]))


@pytest.mark.parametrize("D,nb,g,window", [(128, 4, 64, 0), (64, 2, 32, 700), (256, 8, 128, 0)])
def test_a_piece_of_a_prompt(hqq, D, nb, g, window):  # noqa: F811
    # a hundred queries a sequence over a cached context, more queries than tokens among them
    rng = np.random.default_rng(D)
    lens, ps, kv, heads, nq = [1500, 100, 37], 32, 2, 6, 100
    pages = sum(-(-n // ps) for n in lens)
    cache = random_cache(hqq, rng, pages, kv, D, ps, nb, g)
    t = tables_of(rng, pages, lens, ps, -(-1500 // ps))
    q = torch.from_numpy(rng.standard_normal((3, nq, heads, D)).astype(np.float32)).cuda().to(F16)
    out, lse = hqq.hqq_kv_attention(cache, q, torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                    window=window, return_lse=True)
    check(out, lse, attend(cache, q.float().cpu().numpy(), t, lens, window))


@pytest.mark.parametrize("nb", [2, 4, 8])
def test_rows_at_the_end_of_the_range(hqq, nb):  # noqa: F811
    # infinities, NaN and the largest numbers: finite metadata, finite as bf16 and in attention; as fp16
    # what lies beyond 65504 is infinite, as the conversion makes it
    D, ps, n = 128, 16, 6
    for dtype in (F16, BF16):
        cache = hqq.hqq_kv_cache(1, 1, D, ps, nb, 64)
        k = torch.randn(n, 1, D, device="cuda").to(dtype)
        k[0, 0, :2] = torch.tensor([np.inf, -np.inf])
        k[1, 0, 3], k[2], k[3, 0, 70] = np.nan, np.inf, -65504.0
        k[4, 0, ::2], k[4, 0, 1::2] = 65504.0, -65504.0
        v = k.flip(0).contiguous()
        slots = torch.arange(n, device="cuda")
        hqq.hqq_kv_append(cache, k, v, slots)
        assert torch.isfinite(cache.k_meta).all() and torch.isfinite(cache.v_meta).all()
        as_bf, as_half = hqq.hqq_kv_read(cache, slots, BF16), hqq.hqq_kv_read(cache, slots, F16)
        table = np.zeros((1, 1), np.int32)
        values = [torch.from_numpy(x).cuda().transpose(0, 1) for x in context(cache, table[0], n)[::2][:2]]
        for bf, half, x in zip(as_bf, as_half, values):
            assert torch.isfinite(bf).all() and x.abs().max() < 65504 * (1 + 2.0 ** -8)
            assert torch.equal(torch.isinf(half), x.abs() >= 65520)
        q = torch.randn(1, 1, 2, D, device="cuda").to(BF16)
        out, lse = hqq.hqq_kv_attention(cache, q, torch.from_numpy(table).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"),
                                        return_lse=True)
        check(out, lse, attend(cache, q.float().cpu().numpy(), table, [n]))


def test_results_require_no_grad(hqq):  # noqa: F811
    cache = hqq.hqq_kv_cache(2, 1, 64, 16, 4, 32)
    k = torch.randn(4, 1, 64, device="cuda").to(BF16).requires_grad_()
    slots = torch.arange(4, device="cuda")
    assert not any(x.requires_grad for x in hqq.hqq_kv_append(cache, k, k, slots, return_values=True))
    q = torch.randn(1, 1, 2, 64, device="cuda").to(BF16).requires_grad_()
    t, n = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([4], dtype=torch.int32, device="cuda")
    assert not any(x.requires_grad for x in hqq.hqq_kv_attention(cache, q, t, n, return_lse=True))
    assert not any(x.requires_grad for x in hqq.hqq_kv_prefix_attention(cache, q, t[0], 4, t, n - 4, return_lse=True))


@pytest.mark.parametrize("path", ["own", "shared", "prefix", "many rows"])
def test_scores_far_apart_are_right_or_nan(hqq, path):  # noqa: F811
    # some tokens' scores lie at -2^19 to -2^30 and beyond, the others near zero: rows with scores below 2^22
    # are right, the others right or NaN; nothing is silently wrong
    rng = np.random.default_rng(8)
    D, ps, kv, heads = 128, 16, 2, 4
    lens = {"shared": [1500, 64, 700], "own": [500, 64, 300]}.get(path, [30, 1, 70])
    B, nq = len(lens), 14 if path == "many rows" else 3
    prefix = 600 if path not in ("own", "shared") else 0
    shared = -(-prefix // ps)
    pages = shared + sum(-(-n // ps) for n in lens)
    t = tables_of(rng, pages - shared, lens, ps, -(-max(lens) // ps)) + shared
    tc, lc = torch.from_numpy(t.astype(np.int32)).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    pt = rng.permutation(shared).astype(np.int32)
    q = torch.from_numpy(-np.abs(rng.standard_normal((B, nq, heads, D))).astype(np.float32)).cuda().to(BF16)
    for low, high, size in ((9, 11, (pages, kv, ps, 1)), (13, 15, (pages, kv, ps, 1)), (13, 15, (pages, 1, 1, 1))):
        cache = random_cache(hqq, rng, pages, kv, D, ps, 4, 64)
        cache.k_meta[..., 1] = 0
        up = 2.0 ** torch.from_numpy(rng.uniform(low, high, (pages, kv, ps, 1))).cuda()
        up[torch.from_numpy(rng.random(size) < 0.6).cuda().expand(up.shape)] = 1   # some tokens, or whole blocks
        cache.k_meta[..., 0] = (cache.k_meta[..., 0].double() * up).clamp(max=2.0 ** 15).half()
        for scale in (1.0, 16.0, 1024.0):
            if shared:
                out, lse = hqq.hqq_kv_prefix_attention(cache, q, torch.from_numpy(pt).cuda(), prefix, tc, lc, scale=scale, return_lse=True)
            else:
                out, lse = hqq.hqq_kv_attention(cache, q, tc, lc, scale=scale, return_lse=True)
            want = attend(cache, q.float().cpu().numpy(), t, lens, prefix=(pt, prefix) if shared else (None, 0), scale=scale)
            bad = torch.isnan(lse)
            k = np.concatenate([context(cache, x, len(x) * ps)[0] for y in (pt[None], t) for x in y if len(x)], 1)
            rows = np.abs(q.float().cpu().numpy().astype(np.float64)).sum(-1).max()
            if scale * np.log2(np.e) * rows * np.abs(k).max() < 2.0 ** 22:
                assert not bad.any()
            assert torch.isnan(out[bad]).all()
            out[bad], lse[bad] = torch.from_numpy(want[0]).cuda().to(out)[bad], torch.from_numpy(want[1]).cuda().to(lse)[bad]
            check(out, lse, want, (low, scale))
