"""The key/value cache's calls refuse bad arguments on the host, before anything reaches a GPU, and
plan their workspace; the binding's checks.  No GPU is needed."""
import ctypes

import pytest

from free_weight_quantization_b200 import build as fbuild
from free_weight_quantization_b200 import hqq

torch = pytest.importorskip("torch")

OK, ARG, ALIGN, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 5
FAKE = 0x10000  # never dereferenced: every call below fails its host-side checks, or launches nothing


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return hqq.lib()


def cache(**k):
    a = dict(dict(kc=FAKE, vc=FAKE, km=FAKE, vm=FAKE, pages=10, page=64, heads=2, dim=128, bits=4, group=64), **k)
    return hqq.HqqKvCache(a["kc"], a["vc"], a["km"], a["vm"], a["pages"], a["page"], a["heads"], a["dim"], a["bits"], a["group"])


BAD_CACHES = [(dict(pages=-1), ARG), (dict(heads=0), ARG), (dict(page=0), ARG), (dict(bits=0), ARG), (dict(bits=9), ARG),
              (dict(group=0), ARG), (dict(dim=0), ARG), (dict(group=48), ARG), (dict(kc=0), ARG), (dict(vm=0), ARG),
              (dict(bits=3), UNSUPPORTED), (dict(dim=96, group=32), UNSUPPORTED), (dict(group=16), UNSUPPORTED),
              (dict(dim=512), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=8), UNSUPPORTED),
              (dict(page=2048), UNSUPPORTED), (dict(pages=1 << 40), UNSUPPORTED), (dict(kc=FAKE + 8), ALIGN),
              (dict(km=FAKE + 4), ALIGN)]


def append(L, c, k=FAKE, v=FAKE, dtype=0, tokens=4, slots=FAKE, kv=0, vv=0):
    return L.hqq_kv_append(ctypes.byref(c) if c is not None else None, k, v, dtype, tokens, 256, 128, 256, 128, slots,
                           kv or None, vv or None, None)


def read(L, c, slots=FAKE, tokens=4, dtype=0, k=FAKE, v=FAKE):
    return L.hqq_kv_read(ctypes.byref(c), slots, tokens, dtype, k, v, None)


def attend(L, c, q=FAKE, dtype=0, batch=2, nq=1, heads=4, pages=FAKE, wide=8, lens=FAKE, max_len=512, window=0, scale=0.1,
           out=FAKE, lse=0, ws=FAKE, wsb=1 << 30, prefix=None):
    head = (ctypes.byref(c), q, dtype, batch, nq, heads, nq * heads * 128, heads * 128, 128)
    table = (pages, wide, wide, lens, max_len)
    tail = (scale, out, lse or None, ws, wsb, None)
    if prefix is None:
        return L.hqq_kv_attention(*head, *table, window, *tail)
    return L.hqq_kv_prefix_attention(*head, *prefix, *table, *tail)


@pytest.mark.parametrize("what,code", BAD_CACHES, ids=lambda v: str(v))
def test_a_bad_cache_is_refused_by_every_call(L, what, code):
    c = cache(**what)
    assert append(L, c) == code
    assert read(L, c) == code
    assert attend(L, c) == code
    assert attend(L, c, prefix=(FAKE, 64)) == code
    assert L.hqq_kv_attention_workspace_bytes(ctypes.byref(c), 2, 1, 4, 512, 0, 0) == 0


def test_append_and_read_refuse(L):
    c = cache()
    assert append(L, None) == ARG
    assert append(L, c, tokens=0, k=None, v=None, slots=None) == OK      # nothing to do
    assert append(L, c, tokens=-1) == ARG
    assert append(L, c, dtype=2) == ARG
    assert append(L, c, tokens=1 << 31) == UNSUPPORTED
    assert append(L, c, k=None) == ARG and append(L, c, v=None) == ARG and append(L, c, slots=None) == ARG
    assert append(L, c, k=FAKE + 1) == ALIGN
    assert append(L, c, slots=FAKE + 4) == ALIGN
    assert append(L, c, kv=FAKE + 8, vv=FAKE) == ALIGN
    assert read(L, c, tokens=0, slots=None, k=None, v=None) == OK
    assert read(L, c, k=None, v=None) == ARG
    assert read(L, c, dtype=-1) == ARG
    assert read(L, c, k=FAKE + 2) == ALIGN
    assert read(L, c, slots=None) == ARG


def test_attention_refuses(L):
    c = cache()
    for prefix in (None, (FAKE, 64)):
        call = lambda **k: attend(L, c, prefix=prefix, **k)  # noqa: E731, B023
        assert call(batch=0, q=None, out=None, ws=None, wsb=0) == OK
        assert call(nq=0, q=None, out=None, ws=None, wsb=0) == OK
        assert call(batch=-1) == ARG and call(nq=-1) == ARG
        assert call(heads=0) == ARG and call(heads=3) == ARG             # 3 query heads, 2 key heads
        assert call(max_len=-1) == ARG and call(max_len=513) == ARG      # the table has room for 512
        assert call(scale=0.0) == ARG and call(scale=-1.0) == ARG
        assert call(scale=float("inf")) == ARG and call(scale=float("nan")) == ARG
        assert call(dtype=3) == ARG
        assert call(q=None) == ARG and call(lens=None) == ARG and call(out=None) == ARG and call(pages=None) == ARG
        assert call(q=FAKE + 1) == ALIGN and call(out=FAKE + 8) == ALIGN and call(lens=FAKE + 2) == ALIGN
        assert call(batch=65536, wide=8) == UNSUPPORTED and call(nq=65536) == UNSUPPORTED
        assert call(wide=1 << 26, max_len=1 << 31) == UNSUPPORTED
    assert attend(L, c, window=-1) == ARG
    assert attend(L, c, prefix=(FAKE, -1)) == ARG
    assert attend(L, c, prefix=(None, 64)) == ARG
    assert attend(L, c, prefix=(FAKE + 2, 64)) == ALIGN
    # a workspace that is missing, too small or misaligned, where one is needed
    need = L.hqq_kv_attention_workspace_bytes(ctypes.byref(c), 2, 1, 4, 8192, 0, 0)
    assert need > 0
    assert attend(L, c, wide=128, max_len=8192, ws=None, wsb=need) == WORKSPACE
    assert attend(L, c, wide=128, max_len=8192, wsb=need - 1) == WORKSPACE
    assert attend(L, c, wide=128, max_len=8192, ws=FAKE + 8, wsb=need) == ALIGN


def test_workspace_plan(L):
    c = cache()
    ws = lambda *a: L.hqq_kv_attention_workspace_bytes(ctypes.byref(c), *a)  # noqa: E731
    assert ws(2, 1, 4, 512, 0, 0) == 0              # short: a CTA for each pair, no parts
    long = ws(1, 1, 4, 100000, 0, 0)
    assert 0 < long < 64 << 20
    assert ws(1, 1, 4, 100000, 100, 0) == 0         # a window makes it short
    assert ws(64, 1, 4, 100000, 0, 0) <= 64 << 20   # bounded by the GPU, not by batch or length
    assert ws(2, 1, 4, 512, 0, 1000) > 0            # a prefix's parts
    assert ws(2, 1, 3, 512, 0, 0) == 0              # invalid


def test_binding_refuses_without_a_gpu():
    codes = torch.zeros(2, 1, 16, 64, dtype=torch.uint8)
    meta = torch.zeros(2, 1, 16, 2, 2, dtype=torch.float16)
    with pytest.raises(hqq.HqqError, match="CUDA"):
        hqq.KVCache(codes, codes, meta, meta, 4, 64)
    with pytest.raises(hqq.HqqError, match="nbits"):
        hqq.KVCache(codes, codes, meta, meta, 3, 64)
    with pytest.raises(hqq.HqqError, match="group_size"):
        hqq.KVCache(codes, codes, meta, meta, 4, 48)
    with pytest.raises(hqq.HqqError, match="head_dim"):
        hqq.KVCache(codes[..., :40], codes, meta, meta, 4, 64)
    with pytest.raises(hqq.HqqError, match="page_size"):
        hqq.KVCache(codes[:, :, :12], codes[:, :, :12], meta[:, :, :12], meta[:, :, :12], 4, 64)
    with pytest.raises(hqq.HqqError, match="k_meta"):
        hqq.KVCache(codes, codes, meta[..., :1, :], meta, 4, 64)
    with pytest.raises(hqq.HqqError, match="v_codes"):
        hqq.KVCache(codes, codes.to(torch.int8), meta, meta, 4, 64)
    with pytest.raises(hqq.HqqError):
        hqq.hqq_kv_cache(4, 1, 128, nbits=5, device="cpu")
    with pytest.raises(hqq.HqqError):
        hqq.hqq_kv_cache(4, 1, 100, device="cpu")
