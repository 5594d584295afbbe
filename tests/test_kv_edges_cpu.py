"""The key/value cache's plans and refusals at the ends of their ranges.  No GPU is needed."""
import ctypes

import pytest

from free_weight_quantization_b200 import hqq
from test_kv_cpu import ARG, FAKE, UNSUPPORTED, WORKSPACE, L, append, attend, cache, read  # noqa: F401

pytest.importorskip("torch")


@pytest.mark.parametrize("batch,nq,max_len", [(4, 1, 8192), (1, 1, 100000), (64, 7, 2048), (3, 2, 600), (1, 65535, 5000),
                                              (1, 1, 2 ** 31 - 1)])
def test_a_window_that_hides_nothing_is_planned_as_none(L, batch, nq, max_len):  # noqa: F811
    c = cache(heads=8)
    ws = lambda window: L.hqq_kv_attention_workspace_bytes(ctypes.byref(c), batch, nq, 32, max_len, window, 0)  # noqa: E731
    none = ws(0)
    assert none > 0 or max_len <= 1024
    for window in (max_len, max_len + 1, 2 ** 31 - 1, 2 ** 31, 2 ** 63 - 17 - nq, 2 ** 63 - 17, 2 ** 63 - 16, 2 ** 63 - 2, 2 ** 63 - 1):
        assert ws(window) == none, window


@pytest.mark.parametrize("what", [dict(kv_heads=-1), dict(kv_heads=0), dict(page_size=-16), dict(page_size=0), dict(page_size=48),
                                  dict(page_size=1 << 40), dict(head_dim=-64), dict(head_dim=0), dict(head_dim=1 << 40),
                                  dict(num_pages=-1)])
def test_a_cache_of_impossible_sizes_is_refused_before_it_is_allocated(what):
    sizes = dict(dict(num_pages=2, kv_heads=1, head_dim=128, page_size=16), **what)
    with pytest.raises(hqq.HqqError, match="hqq_kv_cache"):
        hqq.hqq_kv_cache(**sizes, device="cpu")


def test_scales_out_of_range_are_refused(L):  # noqa: F811
    c = cache()
    for scale in (3e38, 2.4e38, 1e39, -1.0, 0.0, 1e-50):
        assert attend(L, c, scale=scale) == ARG
        assert attend(L, c, prefix=(FAKE, 64), scale=scale) == ARG


def test_limits_of_the_attention_calls(L):  # noqa: F811
    c = cache(heads=1, dim=128)
    assert attend(L, c, batch=65535, heads=8, wide=1 << 26, max_len=1 << 30) == UNSUPPORTED     # pairs * units
    assert attend(L, c, batch=65535, nq=65535, heads=1) == UNSUPPORTED                           # rows
    c = cache(heads=1, dim=256, group=128)
    assert attend(L, c, prefix=(FAKE, 64), batch=65535, nq=9, heads=1) == UNSUPPORTED            # blocks of the prefix's rows
    assert append(L, cache(heads=65535), tokens=32769) == UNSUPPORTED
    assert append(L, cache(heads=65536)) == UNSUPPORTED
    assert read(L, cache(pages=(1 << 27) + 1, heads=2)) == UNSUPPORTED                           # 2^34 rows


@pytest.mark.parametrize("wide", [1 << 57, 1 << 58, 1 << 60, 2 ** 63 - 1])
def test_tables_wider_than_64_bits_of_tokens(L, wide):  # noqa: F811
    # the table's room in tokens is not counted, so that it cannot overflow: such a call comes as far as
    # its missing workspace
    for prefix in (None, (FAKE, 64)):
        assert attend(L, cache(), wide=wide, max_len=8192, ws=None, wsb=0, prefix=prefix) == WORKSPACE
        assert attend(L, cache(), wide=127, max_len=8192, ws=None, wsb=0, prefix=prefix) == ARG
        assert attend(L, cache(), wide=127, max_len=127 * 64, ws=None, wsb=0, prefix=prefix) == WORKSPACE
