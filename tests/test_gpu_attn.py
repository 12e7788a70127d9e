"""tq1_paged_attn against attention in 64 bits, at the sizes and masks where it
can go wrong; the bound on the difference is derived in kv_ref.attention."""
import math

import pytest
import torch

from .gpu_util import lib
from .kv_ref import Batch, attention, rounded

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def queries(b, n_q, wide=False):
    q = torch.randn(b.t, n_q, b.d, generator=b.g).to(b.dtype)
    if not wide:
        return q, q.cuda()
    room = torch.zeros(b.t, n_q * b.d + 24, dtype=b.dtype, device="cuda")  # rows of a wider matrix
    room[:, 8:8 + n_q * b.d] = q.cuda().flatten(1)
    return q, room[:, 8:8 + n_q * b.d].unflatten(1, (n_q, b.d))


def run(b, q, n_q, causal=True, window=0, f32=False, stream=None, scale=None):
    L = lib()
    scale = 1 / math.sqrt(b.d) if scale is None else scale
    out = torch.full((b.t, n_q, b.d), 7.0, dtype=torch.float32 if f32 else b.dtype, device="cuda")
    ws = torch.full((L.tq1_paged_attn_workspace_size(b.cache, b.t, n_q, len(b.new)),), 0xFF, dtype=torch.uint8, device="cuda")
    L.tq1_paged_attn(b.cache, b.batch, q, out, scale, causal=causal, window=window, ws=ws, stream=stream)
    assert L.tq1_sync_status() == 0
    return out


def check(b, n_q, causal=True, window=0, f32=False, wide=False, scale=None):
    b.to_gpu(lib())
    q, gq = queries(b, n_q, wide)
    out = run(b, gq, n_q, causal, window, f32, scale=scale)
    ref, tol = attention(b, q, 1 / math.sqrt(b.d) if scale is None else scale, causal, window)
    tol = rounded(tol, ref, out.dtype)
    got = out.cpu().double()
    used = int(b.q_start[-1])
    assert torch.isfinite(got).all()
    worst = ((got - ref).abs() / tol.clamp(min=1e-300))[:used]
    assert (worst <= 1).all(), f"{(worst > 1).sum()} of {worst.numel()} outside, worst {worst.max():.3g}"
    assert (got[used:] == 7).all(), "rows of no sequence were written"
    return out


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,length", [
    ([1], [1]), ([1], [2]), ([1], [15]), ([1], [127]), ([1], [128]), ([1], [129]), ([1], [777]),
    ([1, 1, 1, 1, 1], [1, 16, 17, 600, 33]),
    ([3], [3]), ([17], [40]), ([65, 2], [65, 300]), ([130], [131]), ([300, 1, 7], [300, 257, 900]),
])
def test_lengths(dtype, d, new, length):
    check(Batch(new, length, 16, 2, d, dtype), 8)


@pytest.mark.parametrize("n_q,n_kv", [(1, 1), (4, 4), (3, 1), (5, 1), (14, 2), (16, 1), (17, 1), (48, 2), (128, 1)])
@pytest.mark.parametrize("new", [1, 9, 70])
def test_head_groups(n_q, n_kv, new):
    check(Batch([new, 1], [new + 100, 64], 32, n_kv, 64, F16, seed=n_q), n_q)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["hsd", "shd", "joint"])
def test_pages_and_layouts(page, layout):
    check(Batch([1, 33, 140], [500, 333, 140], page, 3, 128, BF16, layout=layout), 6, wide=True)


@pytest.mark.parametrize("window", [1, 2, 16, 100, 128, 129, 5000])
@pytest.mark.parametrize("causal", [True, False])
def test_windows(window, causal):
    check(Batch([1, 5, 200], [700, 130, 450], 16, 2, 64, F16, seed=window), 6, causal=causal, window=window)


def test_not_causal():
    check(Batch([1, 20, 150], [99, 20, 400], 32, 2, 128, F16), 4, causal=False)


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf"), 65504.0])
@pytest.mark.parametrize("new", [1, 50, 200])
def test_slots_past_the_end_may_hold_anything(junk, new):
    check(Batch([new, 1, new], [new + 3, 77, new + 130], 64, 2, 128, F16, junk=junk), 6)


@pytest.mark.parametrize("window", [1, 5, 16, 100, 333])
@pytest.mark.parametrize("new", [1, 3, 60])
def test_what_a_window_leaves_out_may_hold_anything(window, new):
    # Every slot before the window of a sequence's first new token holds NaN;
    # one of the three has one token whatever the others have.
    new = [new, 1, new]
    length = [a + b for a, b in zip(new, (399, 128, 516))]
    b = Batch(new, length, 16, 2, 64, F16, seed=window)
    for i, (n, ln) in enumerate(zip(new, length)):
        for j in range(max(0, ln - n + 1 - window)):
            b.kv[:, b.table[i, j // 16], :, j % 16] = float("nan")
    ref = Batch(new, length, 16, 2, 64, F16, seed=window)
    b.to_gpu(lib())
    q, gq = queries(b, 6)
    out = run(b, gq, 6, window=window)
    want, tol = attention(ref, q, 1 / 8, True, window)
    assert ((out.cpu().double() - want).abs() <= rounded(tol, want, F16)).all()


@pytest.mark.parametrize("new", [40, 300])
def test_keys_that_are_not_finite_hurt_only_rows_that_see_them(new):
    b = Batch([new], [new + 150], 16, 2, 64, F16)
    clean = b.kv.clone()
    bad = new + 150 - 7  # seen by the last seven tokens
    b.kv[0, b.table[0, bad // 16], :, bad % 16] = float("nan")
    b.to_gpu(lib())
    q, gq = queries(b, 4)
    out = run(b, gq, 4).cpu().double()
    b.kv = clean
    want, tol = attention(b, q, 1 / 8, True, 0)
    tol = rounded(tol, want, F16)
    assert ((out - want).abs() <= tol)[:-7].all() and out[-7:].isnan().all()


@pytest.mark.parametrize("f32", [False, True])
def test_rows_that_see_nothing_are_zero(f32):
    # More new tokens than the cache holds: the first rows stand before the
    # first slot; and sequences that are empty or have no new tokens.
    b = Batch([4, 0, 3, 150, 0, 1], [2, 50, 0, 100, 0, 40], 16, 2, 64, F16, extra_tokens=5, junk=float("nan"))
    out = check(b, 4, f32=f32)
    assert (out[:2] == 0).all() and (out[4:7] == 0).all() and (out[7:57] == 0).all()


@pytest.mark.parametrize("new", [1, 40, 260])
def test_no_key_for_a_windowed_row(new):
    # Non-causal with a window reaching past the end: rows still see the later keys.
    check(Batch([new], [new + 20], 16, 1, 64, BF16), 2, causal=False, window=3)


@pytest.mark.parametrize("new", [1, 30, 200])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_large_scores(new, dtype):
    # Scores of some hundreds: the running maximum moves by far more than the
    # exponent's range while the keys go by.
    b = Batch([new], [new + 700], 16, 1, 64, dtype)
    b.kv[0] = (b.kv[0].float() * torch.linspace(0.1, 6, b.n_pages)[:, None, None, None]).to(dtype)
    check(b, 4, scale=1.0)


@pytest.mark.parametrize("d,n_kv,group,window,dtype", [(64, 8, 3, 1024, F16), (64, 8, 4, 0, BF16), (128, 8, 5, 0, BF16),
                                                       (128, 4, 3, 700, F16), (128, 8, 1, 0, F16)])
@pytest.mark.parametrize("new", [[45, 11, 6, 1062, 1463, 1, 539, 82], [30, 60, 17, 5, 41, 90, 33, 77, 2, 64]])
def test_many_blocks_and_tiles_for_every_cta(d, n_kv, group, window, dtype, new):
    # Every CTA has many blocks of several tiles, most sequences end inside a
    # group of 16 keys, and what lies past their ends is NaN.
    ctx = [935, 535, 960, 2224, 2409, 2508, 1289, 187, 3001, 4444]
    check(Batch(new, [a + b for a, b in zip(new, ctx)], 32, n_kv, d, dtype, seed=d + group, junk=float("nan")), n_kv * group,
          window=window)


@pytest.mark.parametrize("new", [1, 12, 400])
def test_large_scores_in_long_runs(new):
    # The running maximum moves in the middle of a CTA's run of blocks.
    b = Batch([new] * 3, [new + 4000, new + 3111, new + 5003], 64, 8, 64, F16, seed=new)
    for i, ln in enumerate(b.len):
        for j, p in enumerate(b.table[i, :-(-ln // 64)].long().tolist()):
            b.kv[0, p] = (b.kv[0, p].float() * (0.2 + 0.1 * j)).to(F16)
    check(b, 16, scale=0.5)


def test_fp32_output_feeds_the_quantiser():
    check(Batch([1, 100], [200, 300], 16, 2, 128, BF16), 8, f32=True)


def test_many_sequences():
    n = 700
    new = [(i * 7) % 3 for i in range(n)]
    check(Batch(new, [max(v, (i * 37) % 90) for i, v in enumerate(new)], 16, 1, 64, F16), 2)


@pytest.mark.parametrize("off,pad", [(0, 8), (8, 16), (16, 32), (8, 8)])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("new", [2, 30, 200])
def test_output_rows_of_a_wider_matrix(new, f32, off, pad):
    # Rows that begin on 16-byte boundaries, or on 32-byte ones too.
    b = Batch([new, new], [new + 100, new + 333], 16, 2, 64, F16)
    b.to_gpu(lib())
    q, gq = queries(b, 6)
    room = torch.full((b.t, off + 6 * 64 + pad), 7.0, dtype=torch.float32 if f32 else F16, device="cuda")
    out = room[:, off:off + 6 * 64].unflatten(1, (6, 64))
    ws = torch.empty(lib().tq1_paged_attn_workspace_size(b.cache, b.t, 6, 2), dtype=torch.uint8, device="cuda")
    lib().tq1_paged_attn(b.cache, b.batch, gq, out, 0.125, ws=ws)
    assert lib().tq1_sync_status() == 0
    ref, tol = attention(b, q, 0.125, True, 0)
    assert ((out.cpu().double() - ref).abs() <= rounded(tol, ref, out.dtype)).all()
    assert (room[:, :off] == 7).all() and (room[:, off + 6 * 64:] == 7).all()


@pytest.mark.parametrize("n", [1, 2, 37, 38, 39, 75, 76, 77, 151, 152, 153])
@pytest.mark.parametrize("new,d", [(1, 64), (1, 128), (6, 64), (40, 128)])
def test_about_as_many_blocks_as_ctas(n, new, d):
    # Shares of one unit and a little more: some begin or end between two tiles
    # and do nothing of either.
    check(Batch([new] * n, [new + (i * 53) % 300 for i in range(n)], 16, 1, d, F16, seed=n, junk=float("nan")), 4)


def test_offsets_past_32_bits():
    # A pool of more than 2^32 bytes of keys; the sequence's pages are its last.
    L = lib()
    b = Batch([2, 150], [300, 400], 16, 2, 128, F16, spare=0)
    b.to_gpu(L)
    n = (1 << 32) // (2 * 16 * 128) + b.n_pages  # over 2^32 elements
    big = [torch.empty(n, 2, 16, 128, dtype=F16, device="cuda") for _ in range(2)]
    for x, y in zip(big, b.gkv):
        x[-b.n_pages:] = y
    b.gtable = torch.where(b.gtable >= 0, b.gtable + (n - b.n_pages), b.gtable)
    b.cache, b.batch = L.tq1_kv_cache(*big), L.tq1_kv_batch(b.gtable, b.gq, b.glen)
    q, gq = queries(b, 4)
    out = run(b, gq, 4)
    ref, tol = attention(b, q, 1 / math.sqrt(128), True, 0)
    assert ((out.cpu().double() - ref).abs() <= rounded(tol, ref, F16)).all()


@pytest.mark.parametrize("new", [1, 200])
def test_same_bits_every_time(new):
    b = Batch([new] * 3, [2000, new, 900], 16, 2, 128, F16).to_gpu(lib())
    _, gq = queries(b, 8)
    first = run(b, gq, 8)
    for _ in range(3):
        assert torch.equal(run(b, gq, 8), first)


def test_page_ids_out_of_range_are_reported():
    L = lib()
    for new in (1, 200):
        b = Batch([new], [new + 100], 16, 1, 64, F16).to_gpu(L)
        q, gq = queries(b, 2)
        b.gtable[0, 1] = b.n_pages
        b.gtable[0, 3] = -5
        out = torch.empty(b.t, 2, 64, dtype=F16, device="cuda")
        ws = torch.empty(L.tq1_paged_attn_workspace_size(b.cache, b.t, 2, 1), dtype=torch.uint8, device="cuda")
        L.tq1_paged_attn(b.cache, b.batch, gq, out, 0.125, ws=ws)
        assert L.tq1_sync_status() == -8
        assert L.tq1_sync_status() == 0
        b.gtable.copy_(b.table)
        ref, tol = attention(b, q, 0.125, True, 0)
        assert ((run(b, gq, 2, scale=0.125).cpu().double() - ref).abs() <= rounded(tol, ref, F16)).all()


def test_lengths_past_the_table_are_cut():
    # kv_len beyond the table's width must not read outside the table.
    L = lib()
    b = Batch([1], [40], 16, 1, 64, F16).to_gpu(L)
    b.glen.fill_(1 << 30)
    _, gq = queries(b, 2)
    out = torch.empty(b.t, 2, 64, dtype=F16, device="cuda")
    ws = torch.empty(L.tq1_paged_attn_workspace_size(b.cache, b.t, 2, 1), dtype=torch.uint8, device="cuda")
    L.tq1_paged_attn(b.cache, b.batch, gq, out, 0.125, ws=ws)
    assert L.tq1_sync_status() == -8  # the entries past its pages are -1


def test_on_another_stream_and_in_a_graph():
    L = lib()
    b = Batch([1, 200], [500, 300], 16, 2, 128, F16).to_gpu(L)
    q, gq = queries(b, 4)
    want = run(b, gq, 4)
    out = torch.zeros_like(want)
    ws = torch.empty(L.tq1_paged_attn_workspace_size(b.cache, b.t, 4, 2), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    L.tq1_paged_attn(b.cache, b.batch, gq, out, 1 / math.sqrt(128), ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.tq1_paged_attn(b.cache, b.batch, gq, out, 1 / math.sqrt(128), ws=ws)
    out.zero_()
    b.glen.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert (out == 0).all()  # lengths are read when the kernels run
    b.glen.copy_(b.kv_len)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
