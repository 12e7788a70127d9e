"""Host checks of the paged-cache entry points: every refusal happens before any
CUDA call, so these need no GPU."""
import ctypes

import pytest

from bit_quantized_gemv_tq1_gb300 import _lib as L
from bit_quantized_gemv_tq1_gb300 import build as B

FAKE = 1 << 20  # an aligned address that is never dereferenced
NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.library()


def cache(**kw):
    f = dict(k=FAKE, v=FAKE, n_pages=10, n_kv=2, page_size=16, head_dim=64, page_stride=2048, head_stride=1024,
             slot_stride=64, dtype=L.TQ1_F16)
    return L.KvCache(**{**f, **kw})


def batch(**kw):
    return L.KvBatch(**{**dict(page_table=FAKE, q_start=FAKE, kv_len=FAKE, n_seqs=3, max_pages=4), **kw})


def pool(**kw):
    f = dict(base=FAKE, n_pools=2, pool_stride=640, page_bytes=64, n_pages=10, refs=FAKE, page_table=FAKE, kv_len=FAKE,
             n_seqs=3, max_pages=4, page_size=16)
    return L.PagePool(**{**f, **kw})


BAD_CACHES = [(dict(k=None), NULL), (dict(v=None), NULL), (dict(v=FAKE + 8), ALIGN), (dict(page_stride=2047), ALIGN),
              (dict(head_stride=12), ALIGN), (dict(slot_stride=68), ALIGN), (dict(slot_stride=56), SHAPE),
              (dict(n_kv=0), SHAPE), (dict(head_dim=0), SHAPE), (dict(head_dim=60), SHAPE), (dict(page_size=0), SHAPE),
              (dict(page_size=24), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED),
              (dict(dtype=L.TQ1_F32), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED), (dict(n_pages=-1), SHAPE)]
BAD_BATCHES = [(dict(page_table=None), NULL), (dict(q_start=None), NULL), (dict(kv_len=None), NULL), (dict(kv_len=FAKE + 2), ALIGN),
               (dict(n_seqs=0), SHAPE), (dict(max_pages=0), SHAPE), (dict(n_seqs=8193), UNSUPPORTED),
               (dict(max_pages=(1 << 20) + 1), UNSUPPORTED)]


def attn(lib, c=None, b=None, q=FAKE, ldq=512, t=5, n_q=8, scale=0.1, causal=1, window=0, out=FAKE, ldo=512, f32=0, ws=FAKE,
         ws_bytes=0):
    return lib.tq1_paged_attn(c or cache(), b or batch(), q, ldq, t, n_q, scale, causal, window, out, ldo, f32, ws, ws_bytes, None)


def rope(lib, c=None, b=None, q=FAKE, ldq=512, k=FAKE, ldk=128, v=FAKE, ldv=128, dtype=0, q_out=FAKE, t=5, n_q=8, f=FAKE,
         rot=64, pos=None):
    return lib.tq1_rope_append(c or cache(), b or batch(), q, ldq, k, ldk, v, ldv, dtype, q_out, t, n_q, f, rot, 0, 1.0, pos, None)


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_caches(lib, kw, code):
    assert attn(lib, c=cache(**kw)) == code
    assert rope(lib, c=cache(**kw)) == code
    assert L.tq1_paged_attn_workspace_size(cache(**kw), 5, 8, 3) == 0


@pytest.mark.parametrize("kw,code", BAD_BATCHES)
def test_batches(lib, kw, code):
    assert attn(lib, b=batch(**kw)) == code
    assert rope(lib, b=batch(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(t=-1), SHAPE), (dict(t=(1 << 24) + 1), UNSUPPORTED), (dict(n_q=0), SHAPE), (dict(n_q=7), SHAPE), (dict(n_q=258, ldq=1 << 20, ldo=1 << 20), UNSUPPORTED),
    (dict(n_q=1 << 40), UNSUPPORTED), (dict(ldq=504), SHAPE), (dict(ldo=504), SHAPE), (dict(ldq=516), ALIGN), (dict(ldo=516), ALIGN),
    (dict(t=1 << 24, n_q=256, ldq=1 << 20, ldo=1 << 20), UNSUPPORTED), (dict(window=-1), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=float("nan")), SHAPE),
    (dict(scale=float("inf")), SHAPE), (dict(q=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL),
    (dict(q=FAKE + 8), ALIGN), (dict(out=FAKE + 8), ALIGN), (dict(ws=FAKE + 8), ALIGN), (dict(t=0), 0),
])
def test_attention_arguments(lib, kw, code):
    assert attn(lib, **kw) == code


def test_attention_head_dims(lib):
    for d in (8, 32, 96, 256):
        c = cache(head_dim=d, slot_stride=256, head_stride=4096, page_stride=8192)
        assert attn(lib, c=c, ldq=8 * d, ldo=8 * d) == UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(t=-1), SHAPE), (dict(n_q=0), SHAPE), (dict(n_q=1 << 40), UNSUPPORTED), (dict(rot=-8), SHAPE), (dict(rot=72), SHAPE), (dict(rot=12), SHAPE),
    (dict(ldq=511), SHAPE), (dict(ldk=127), SHAPE), (dict(ldv=127), SHAPE), (dict(ldq=514), ALIGN), (dict(ldk=130), ALIGN),
    (dict(ldv=129), ALIGN), (dict(dtype=3), UNSUPPORTED), (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(q_out=None), NULL), (dict(f=None), NULL), (dict(q=FAKE + 8), ALIGN), (dict(k=FAKE + 4), ALIGN),
    (dict(v=FAKE + 2), ALIGN), (dict(q_out=FAKE + 8), ALIGN), (dict(f=FAKE + 1), ALIGN), (dict(pos=FAKE + 2), ALIGN), (dict(t=0), 0),
])
def test_rope_arguments(lib, kw, code):
    assert rope(lib, **kw) == code


def test_null_structs(lib):
    null_c, null_b = ctypes.POINTER(L.KvCache)(), ctypes.POINTER(L.KvBatch)()
    assert lib.tq1_paged_attn(null_c, batch(), FAKE, 512, 5, 8, 0.1, 1, 0, FAKE, 512, 0, FAKE, 0, None) == NULL
    assert lib.tq1_paged_attn(cache(), null_b, FAKE, 512, 5, 8, 0.1, 1, 0, FAKE, 512, 0, FAKE, 0, None) == NULL
    assert lib.tq1_pages_compact(ctypes.POINTER(L.PagePool)(), FAKE, 1 << 20, None) == NULL


@pytest.mark.parametrize("args,code", [
    ((FAKE, 0, 1e4, 1.0, 0, 1, 32), SHAPE), ((FAKE, 3, 1e4, 1.0, 0, 1, 32), SHAPE), ((FAKE, 64, 0.0, 1.0, 0, 1, 32), SHAPE),
    ((FAKE, 64, 1e4, 0.0, 0, 1, 32), SHAPE), ((FAKE, 64, 1e4, float("inf"), 0, 1, 32), SHAPE), ((FAKE, 64, 1e4, 2.0, float("nan"), 1, 32), SHAPE),
    ((None, 64, 1e4, 1.0, 0, 1, 32), NULL), ((FAKE + 2, 64, 1e4, 1.0, 0, 1, 32), ALIGN), ((FAKE, 258, 1e4, 1.0, 0, 1, 32), UNSUPPORTED),
])
def test_frequency_arguments(lib, args, code):
    assert lib.tq1_rope_freqs(*args, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(base=None), NULL), (dict(refs=None), NULL), (dict(page_table=None), NULL), (dict(kv_len=None), NULL),
    (dict(base=FAKE + 8), ALIGN), (dict(refs=FAKE + 4), ALIGN), (dict(kv_len=FAKE + 1), ALIGN), (dict(page_bytes=24), ALIGN),
    (dict(pool_stride=648), ALIGN), (dict(pool_stride=624), SHAPE), (dict(n_pages=0), SHAPE), (dict(page_size=0), SHAPE),
    (dict(n_seqs=0), SHAPE), (dict(max_pages=0), SHAPE), (dict(n_pools=-1), SHAPE), (dict(page_size=257), UNSUPPORTED),
    (dict(n_pages=(1 << 22) + 1), UNSUPPORTED), (dict(max_pages=(1 << 20) + 1), UNSUPPORTED),
])
def test_pools(lib, kw, code):
    p = pool(**kw)
    assert lib.tq1_pages_copy(p, FAKE, FAKE, 2, None) == code
    assert lib.tq1_pages_resize(p, FAKE, FAKE, 2, FAKE, 1 << 20, None) == code
    assert lib.tq1_pages_fork(p, FAKE, FAKE, 2, FAKE, 1 << 20, None) == code
    assert lib.tq1_pages_compact(p, FAKE, 1 << 20, None) == code
    assert L.tq1_pages_workspace_size(p) == 0


def test_page_calls(lib):
    need = L.tq1_pages_workspace_size(pool())
    assert need > 0 and need % 256 == 0
    for fn in (lib.tq1_pages_resize, lib.tq1_pages_fork):
        assert fn(pool(), FAKE, FAKE, 2, FAKE, need - 1, None) == WORKSPACE
        assert fn(pool(), FAKE, FAKE, 4, FAKE, need, None) == SHAPE  # more than there are sequences
        assert fn(pool(), FAKE, FAKE, -1, FAKE, need, None) == SHAPE
        assert fn(pool(), None, FAKE, 2, FAKE, need, None) == NULL
        assert fn(pool(), FAKE, None, 2, FAKE, need, None) == NULL
        assert fn(pool(), FAKE, FAKE, 2, None, need, None) == NULL
        assert fn(pool(), FAKE, FAKE, 2, FAKE + 8, need, None) == ALIGN
        assert fn(pool(), FAKE + 2, FAKE, 2, FAKE, need, None) == ALIGN
        assert fn(pool(), None, None, 0, None, 0, None) == 0
    assert lib.tq1_pages_compact(pool(), FAKE, need - 1, None) == WORKSPACE
    assert lib.tq1_pages_compact(pool(), None, need, None) == NULL
    assert lib.tq1_pages_copy(pool(), FAKE, FAKE, 11, None) == SHAPE
    assert lib.tq1_pages_copy(pool(), None, FAKE, 2, None) == NULL
    assert lib.tq1_pages_copy(pool(), FAKE, FAKE + 2, 2, None) == ALIGN
    assert lib.tq1_pages_copy(pool(), None, None, 0, None) == 0


def test_status_text(lib):
    assert L.STATUS[-9] == "TQ1_ERR_NO_PAGES" and b"page" in lib.tq1_status_string(-9)
