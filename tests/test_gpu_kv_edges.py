"""The key/value cache's calls at the ends of their ranges, against the 64-bit forms and the tolerances
of test_gpu_kv.py."""
import sys

import numpy as np
import pytest

from test_gpu_kv import F16, attend, bits, check, context, hqq, random_cache, tables_of  # noqa: F401

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
