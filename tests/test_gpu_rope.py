"""tq1_rope_append and tq1_rope_freqs against 64-bit rotations."""
import math

import pytest
import torch

from .gpu_util import lib
from .kv_ref import TINY, UNIT, Batch, rotate

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def freqs(rot, base=10000.0):
    return (base ** (-2 * torch.arange(rot // 2, dtype=torch.float64) / max(rot, 1))).to(F32)


def check(b, n_q, rot, interleaved, in_dtype=F32, mscale=1.0, positions=None, fused=True):
    L = lib()
    b.to_gpu(L)
    n_kv, d, page = b.n_kv, b.d, b.page
    heads = n_q + 2 * n_kv
    x = torch.randn(b.t, heads, d, generator=b.g).to(in_dtype)
    parts = [x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]]
    gx = x.cuda()
    gparts = [gx[:, :n_q], gx[:, n_q:n_q + n_kv], gx[:, n_q + n_kv:]]
    if not fused:
        gparts = [p.contiguous() for p in gparts]
    f = freqs(rot)
    q_out = torch.full((b.t, n_q, d), 7.0, dtype=b.dtype, device="cuda")
    gpos = None if positions is None else positions.to(torch.int32).cuda()
    L.tq1_rope_append(b.cache, b.batch, *gparts, q_out, f.cuda(), rot, interleaved=interleaved, mscale=mscale, positions=gpos)
    status = L.tq1_sync_status()
    want_q = torch.full((b.t, n_q, d), 7.0, dtype=torch.float64)
    size_q = torch.zeros_like(want_q)
    want, size = b.kv.double(), torch.zeros(b.kv.shape, dtype=torch.float64)
    at, missed = 0, False
    for i, (n, ln) in enumerate(zip(b.new, b.len)):
        for j in range(n):
            slot = ln - n + j
            turn = slot if positions is None else int(positions[at + j])
            angle = turn * f.double()
            want_q[at + j], size_q[at + j] = rotate(parts[0][at + j].double(), angle, mscale, rot, interleaved)
            if slot < 0 or slot >= ln:
                missed = True
                continue
            p = int(b.table[i, slot // page])
            want[0, p, :, slot % page], size[0, p, :, slot % page] = rotate(parts[1][at + j].double(), angle, mscale, rot, interleaved)
            want[1, p, :, slot % page] = parts[2][at + j].double()
            size[1, p, :, slot % page] = 0
        at += n
    assert status == (-8 if missed else 0)
    # fp32: the angle to 2^-22 (a half turn in fp32), sine and cosine to 2^-23, two products and a sum; then one
    # rounding to 16 bits.
    for got, ref, sz in ((q_out, want_q, size_q), (b.gkv, want, size)):
        tol = sz * 6 * 2.0 ** -23 + UNIT[b.dtype] * ref.abs() * (1 + 2.0 ** -6) + TINY[b.dtype]
        same = ref == got.cpu().double()
        assert (((got.cpu().double() - ref).abs() <= tol) | same).all()
    return q_out


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("in_dtype", [F32, F16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types_and_layouts(dtype, in_dtype, interleaved):
    check(Batch([1, 7, 40], [300, 7, 99], 16, 2, 64, dtype), 6, 64, interleaved, in_dtype)


@pytest.mark.parametrize("d,rot", [(8, 8), (64, 8), (64, 16), (80, 40), (96, 96), (128, 0), (128, 64), (128, 120), (256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_part_of_the_head(d, rot, interleaved):
    check(Batch([3, 1], [20, 33], 16, 3, d, BF16), 5, rot, interleaved)


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("layout", ["hsd", "shd", "joint"])
def test_pages_and_cache_layouts(page, layout):
    check(Batch([1, 1, 100], [1, page + 1, 300], page, 2, 128, F16, layout=layout), 4, 128, False, fused=layout != "shd")


def test_far_positions_keep_their_angles():
    # A million radians: an fp32 angle would be off by 0.03.
    pos = torch.tensor([0, 1, 131071, 1048575, 16777215, -3, 2 ** 31 - 1])
    check(Batch([7], [50], 16, 1, 128, F16), 2, 128, False, positions=pos, mscale=1.2)


def test_tokens_of_no_sequence_and_without_a_slot():
    b = Batch([3, 0, 2], [2, 9, 2], 16, 1, 64, F16, extra_tokens=4)
    q_out = check(b, 2, 64, True)
    assert (q_out[5:] == 7).all()


@pytest.mark.parametrize("t", [1, 2, 1300])
def test_many_tokens(t):
    check(Batch([t, 1], [t + 5, 70], 32, 1, 64, BF16), 3, 32, False)


def test_bad_page_is_skipped_and_reported():
    L = lib()
    b = Batch([2], [18], 16, 1, 64, F16).to_gpu(L)
    before = b.gkv.clone()
    b.gtable[0, 1] = b.n_pages + 3
    x = torch.randn(2, 3, 64, device="cuda")
    q_out = torch.zeros(2, 1, 64, dtype=F16, device="cuda")
    L.tq1_rope_append(b.cache, b.batch, x[:, :1], x[:, 1:2], x[:, 2:], q_out, freqs(64).cuda(), 64)
    assert L.tq1_sync_status() == -8
    assert torch.equal(before, b.gkv) and (q_out != 0).any()


@pytest.mark.parametrize("rot,base,factor,orig,low,high", [
    (128, 10000.0, 1.0, 0.0, 1.0, 32.0), (64, 500000.0, 8.0, 8192.0, 1.0, 4.0), (128, 10000.0, 40.0, 4096.0, 1.0, 32.0),
    (32, 10000.0, 4.0, 2048.0, math.inf, math.inf), (2, 10000.0, 2.0, 100.0, 1.0, 1.0), (256, 1e6, 1.0, 0.0, 0.0, 0.0),
])
def test_frequencies(rot, base, factor, orig, low, high):
    L = lib()
    got = torch.empty(rot // 2, device="cuda")
    L.tq1_rope_freqs(got, rot, base, factor, orig, low, high)
    for i, v in enumerate(got.cpu().double().tolist()):
        theta = base ** (-2 * i / rot)
        turns = orig * theta / (2 * math.pi)
        if factor == 1:
            keep = 1.0
        elif high > low:
            keep = min(max((turns - low) / (high - low), 0.0), 1.0)
        else:
            keep = 1.0 if turns >= high else 0.0
        want = theta * ((1 - keep) / factor + keep)
        assert abs(v - want) <= want * 2.0 ** -23
