"""tq1_paged_attn at the edges of its numbers, masks, tables and workspaces."""
import math

import pytest
import torch

from . import kv_ref
from .gpu_util import lib
from .kv_ref import Batch, attention, rounded

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def attend(b, q, n_q, scale, out_dtype=None, window=0, causal=True, ws=None):
    L = lib()
    out = torch.full((b.t, n_q, b.d), 7.0, dtype=out_dtype or b.dtype, device="cuda")
    if ws is None:
        ws = torch.empty(L.tq1_paged_attn_workspace_size(b.cache, b.t, n_q, len(b.new)), dtype=torch.uint8, device="cuda")
    L.tq1_paged_attn(b.cache, b.batch, q, out, scale, causal=causal, window=window, ws=ws)
    return out


def queries(b, n_q):
    q = torch.randn(b.t, n_q, b.d, generator=b.g).to(b.dtype)
    return q, q.cuda()


@pytest.mark.parametrize("new,lift", [(1, 15), (5, 15), (40, 7), (200, 7)])
@pytest.mark.parametrize("d", [64, 128])
def test_many_small_weights_beside_large_ones(new, lift, d):
    # Sixteen keys with the largest weight and values of zero, one in every 16
    # of the first 256; 3744 others with weights of e^-17 to e^-20 of that,
    # below fp16's smallest number, whose values make up the output.  Weights
    # are formed times 2^lift: half the spacing of fp16's smallest numbers is
    # then 2^(-25-lift) of the largest weight.  As many heads and sequences as
    # let every CTA have long runs of keys behind the large ones.
    L, n, heads, seqs = lib(), 4000, 8, 20
    b = Batch([new], [n], 32, heads, d, F16, seed=new)
    pages = b.table[0, :n // 32].long()
    x = -17 - torch.randint(0, 193, (n,), generator=b.g) / 64
    x[5:256:16] = 0
    x = x.to(F16)
    b.kv[0] = 0
    b.kv[0, pages, :, :, 0] = x.view(-1, 1, 32)
    b.kv[1] = b.kv[1].abs() + 0.5
    for j in range(5, 256, 16):
        b.kv[1, pages[j // 32], :, j % 32] = 0
    b.to_gpu(L)
    b.t *= seqs
    b.new = [new] * seqs
    b.gtable, b.glen = b.gtable.repeat(seqs, 1), b.glen.repeat(seqs)  # all read the same pages
    b.gq = torch.arange(0, b.t + 1, new, dtype=torch.int32, device="cuda")
    b.batch = L.tq1_kv_batch(b.gtable, b.gq, b.glen)
    q = torch.zeros(b.t, heads, d, dtype=F16, device="cuda")
    q[..., 0] = 1
    out = attend(b, q, heads, 1.0, F32, causal=False).cpu().double()
    assert L.tq1_sync_status() == 0
    e, v = x.double().exp(), b.sequence(0, 1)
    want = (e[:, None, None] * v).sum(0) / e.sum()  # every term is positive
    tol = want * (kv_ref.UNIT[F16] + 2.0 ** -20 + 2 * n * 2.0 ** -24) + n * 2.0 ** (-25 - lift) * v.max() / e.sum()
    assert ((out - want).abs() <= tol).all(), float(((out - want).abs() / tol).max())


@pytest.mark.parametrize("window", [1, 16, 100, 333])
@pytest.mark.parametrize("new", [1, 3, 40, 260])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 64)])
def test_pages_before_the_window_may_be_gone(d, page, window, new):
    # A cache that frees what its window has passed: the table names no page
    # there (or one that is no page any more), and that is no error.
    length = [new + 399, new + 2001]
    b = Batch([new, new], length, page, 2, d, F16, seed=window).to_gpu(lib())
    q, gq = queries(b, 6)
    for i, ln in enumerate(length):
        gone = max(0, ln - new + 1 - window) // page
        b.gtable[i, :gone] = -1
        b.gtable[i, :gone:3] = b.n_pages + 7
    out = attend(b, gq, 6, 0.125, window=window)
    assert lib().tq1_sync_status() == 0
    want, tol = attention(b, q, 0.125, True, window)
    assert ((out.cpu().double() - want).abs() <= rounded(tol, want, F16)).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("new,length,n_q", [([4], [2], 2), ([9, 1, 5], [8, 3, 1], 2), ([50], [30], 2), ([150], [100], 4),
                                            ([700, 1], [600, 40], 4), ([2600], [2500], 6), ([12] * 40, [7] * 40, 2)])
def test_rows_that_see_nothing_are_zero_whatever_the_values_are(new, length, n_q, f32, bad):
    # More new tokens than slots: the first rows stand before the first slot.
    b = Batch(new, length, 16, 2, 64, F16)
    b.kv[1] = bad
    b.to_gpu(lib())
    _, gq = queries(b, n_q)
    out = attend(b, gq, n_q, 0.125, F32 if f32 else None).cpu()
    assert lib().tq1_sync_status() == 0
    at = 0
    for n, ln in zip(new, length):
        none = max(n - ln, 0)
        assert (out[at:at + none] == 0).all()
        assert not out[at + none:at + n].isfinite().any()
        at += n


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q,n_kv", [(8, 2), (1, 1), (96, 1)])
def test_a_workspace_for_the_largest_batch_serves_smaller_ones(d, n_q, n_kv):
    L = lib()
    most = Batch([1] * 64, [40] * 64, 16, n_kv, d, F16).to_gpu(L)
    ws = torch.empty(L.tq1_paged_attn_workspace_size(most.cache, 64, n_q, 64), dtype=torch.uint8, device="cuda")
    for new in ([64], [63, 1], [1] * 64, [7] * 9, [2], [33] + [0] * 40 + [31], [16, 16, 16, 16]):
        b = Batch(new, [n + 50 for n in new], 16, n_kv, d, F16, seed=len(new)).to_gpu(L)
        assert L.tq1_paged_attn_workspace_size(b.cache, b.t, n_q, len(new)) <= ws.numel()
        q, gq = queries(b, n_q)
        out = attend(b, gq, n_q, 0.125, ws=ws)
        assert L.tq1_sync_status() == 0
        want, tol = attention(b, q, 0.125, True, 0)
        assert ((out.cpu().double() - want).abs() <= rounded(tol, want, F16)).all()


@pytest.mark.parametrize("t,n_q", [(40, 2), (300, 2), (300, 12)])
def test_starts_that_do_not_ascend_are_refused_whole(t, n_q):
    # Sequences that count the same tokens several times over: nothing is done.
    L = lib()
    b = Batch([t, 0, 0, 0, 0], [t + 20, 30, 30, 30, 30], 16, 1, 64, F16).to_gpu(L)
    _, gq = queries(b, n_q)
    b.gq.copy_(torch.tensor([0, t, 0, t, 0, t], dtype=torch.int32))
    out = attend(b, gq, n_q, 0.125)
    assert L.tq1_sync_status() == -8
    assert (out == 7).all()
    b.gq.copy_(b.q_start)
    assert (attend(b, gq, n_q, 0.125) != 7).any(-1).all() and L.tq1_sync_status() == 0


def test_starts_that_hold_anything():
    L = lib()
    g = torch.Generator().manual_seed(3)
    for n_seqs, t in ((3, 20), (700, 100), (5, 700)):
        b = Batch([t] + [0] * (n_seqs - 1), [t + 9] + [5] * (n_seqs - 1), 16, 1, 64, F16).to_gpu(L)
        _, gq = queries(b, 4)
        for _ in range(8):
            b.gq.copy_(torch.randint(-2 ** 31, 2 ** 31 - 1, (n_seqs + 1,), generator=g, dtype=torch.int64).to(torch.int32))
            b.glen.copy_(torch.randint(-2 ** 31, 2 ** 31 - 1, (n_seqs,), generator=g, dtype=torch.int64).to(torch.int32))
            attend(b, gq, 4, 0.125)
            assert L.tq1_sync_status() in (0, -8)


@pytest.mark.parametrize("new", [[1, 1], [30], [200, 3]])
def test_heads_that_share_their_pages(new):
    # Head stride 0: all kv heads read the same keys and values.
    L = lib()
    b = Batch(new, [n + 150 for n in new], 16, 3, 128, BF16)
    b.kv[:] = b.kv[:, :, :1].clone()
    b.to_gpu(L)
    one = b.gkv[:, :, :1].contiguous().expand(-1, -1, 3, -1, -1)
    b.cache = L.tq1_kv_cache(one[0], one[1])
    assert b.cache.head_stride == 0
    q, gq = queries(b, 12)
    out = attend(b, gq, 12, 0.1)
    assert L.tq1_sync_status() == 0
    want, tol = attention(b, q, 0.1, True, 0)
    assert ((out.cpu().double() - want).abs() <= rounded(tol, want, BF16)).all()
