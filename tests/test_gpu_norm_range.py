"""tq1_rms_norm of rows whose squares, or the sum of them, lie outside fp32's range."""
import pytest
import torch

from tests.test_gpu_norm import TYPES, check, gen, ops

pytestmark = pytest.mark.gpu
SIZES = [5e17, 1e18, 1.8e19, 1.6e38, 1e-15, 1e-19, 1e-23, 1e-38, 1e-42]


@pytest.fixture(scope="module")
def tq():
    from bit_quantized_gemv_tq1_gb300 import build
    build.build()
    import bit_quantized_gemv_tq1_gb300 as tq
    return tq


def even(g, *shape):
    return 2 * torch.rand(*shape, device="cuda", generator=g) - 1


def rows_of_all_sizes(g, t, k, delta):
    size = torch.tensor(SIZES, device="cuda").repeat(-(-t // len(SIZES)))[:t, None]
    x = even(g, t, k) * size
    d = None
    if delta:  # as large as the row where the type has such values
        d = (even(g, t, k) * size).clamp(-6e4, 6e4) if delta == "f16" else even(g, t, k) * size
        d = d.to(TYPES[delta])
    return x, d


# One to four groups a thread, rows that are read twice, rows copied ahead (many, with a 16-bit delta).
@pytest.mark.parametrize("t,k,delta", [(9, 32, ""), (9, 2048, ""), (18, 8192, "f32"), (9, 6144, "f16"), (9, 12288, "bf16"), (9, 40960, "f32"),
                                       (9, 40960, ""), (5, 1 << 20, ""), (1000, 1024, "f32"), (1300, 2048, "bf16"), (1250, 5120, "f16"),
                                       (1230, 16640, "bf16")])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-35, 1e-42, 1e38, 3e38])
def test_large_and_small_rows(tq, t, k, delta, eps):
    g = gen(k)
    x, d = rows_of_all_sizes(g, t, k, delta)
    gamma = 1 + 0.3 * torch.randn(k, device="cuda", generator=g)
    # The call takes eps in fp32: 1e-42 is 714 steps of 2^-149 there, 5e-4 more than in 64 bits, and rows of 1e-38 consist of it.
    check(tq, x, d, gamma, float(torch.tensor(eps, dtype=torch.float32)), in_place=k % 64 == 0)


@pytest.mark.parametrize("k", [8192, 1 << 20])
def test_the_borders(tq, k):
    """Rows of one value, either side of what the plain sum holds: 2^128 / k above, a mean of 2^-100 below."""
    for power in (64 - k.bit_length() / 2, -50.0):
        v = torch.tensor([2.0 ** (power + step) for step in (-1.0, -1e-3, 0.0, 1e-3, 0.5, 1.0)], device="cuda")
        y, _ = check(tq, v[:, None].expand(-1, k).contiguous(), None, None, 0.0, in_place=False)
        assert ((y - 1).abs() <= ops(k)).all()


def test_values_far_apart(tq):
    g = gen(2)
    x = even(g, 6, 5120)
    x[0, 7], x[1, 5119], x[2, 0] = 3e38, -1e30, 1e20
    x[3] *= 1e-44
    x[3, 9] = 1e-30
    x[4] *= 1e-30
    x[4, ::3] = 0
    x[5] = 0
    x[5, 100] = 2.0 ** -149
    for eps in (0.0, 1e-6):
        check(tq, x, None, None, eps, in_place=False)


def test_rows_between_leave_the_others_alone(tq):
    g = gen(3)
    x, d = even(g, 1300, 2048), even(g, 1300, 2048).bfloat16()
    some = torch.arange(0, 1300, 7, device="cuda")
    far = x.clone()
    far[some] *= 1e25
    far[some + 1] *= 0
    (ya, qa), (yb, qb) = (check(tq, v, d, None, 1e-6, in_place=False) for v in (x, far))
    same = torch.ones(1300, dtype=torch.bool, device="cuda")
    same[some] = same[some + 1] = False
    assert torch.equal(ya[same], yb[same]) and torch.equal(qa[same], qb[same])


@pytest.mark.parametrize("k", [256, 6144, 40960])
def test_blocks_of_values_that_are_not_finite(tq, k):
    """Finite rows whose y overflows or meets a gamma that is not finite, and rows that are not finite: q8 equals the quantiser's blocks of y."""
    inf, nan = float("inf"), float("nan")
    g = gen(k)
    x, gamma = 5 * torch.randn(8, k, device="cuda", generator=g), 1 + 0.2 * torch.randn(k, device="cuda", generator=g)
    x[0, 3], x[1, 40], x[2, 70], x[2, 71], x[3, 100] = nan, inf, -inf, nan, -inf
    x[4, 32:64] = nan
    x[5, 7] = 3e38
    for values in (gamma, gamma * 3.4e38, gamma * -1e37, torch.where(torch.arange(k, device="cuda") % 37 == 5, inf, gamma),
                   torch.where(torch.arange(k, device="cuda") % 64 == 9, nan, gamma), torch.full_like(gamma, nan), torch.full_like(gamma, -inf)):
        q8, ref = (torch.zeros(8, k // 32, 36, dtype=torch.uint8, device="cuda") for _ in range(2))
        y = torch.empty(8, k, device="cuda")
        tq.tq1_rms_norm(x, values, 1e-6, q8=q8, y=y)
        tq.q8_1_quantize_acts(y, ref, 8, k)
        assert torch.equal(q8[..., 4:], ref[..., 4:])
        scales, want = (b[..., :4].contiguous().view(torch.float16) for b in (q8, ref))
        assert torch.equal(scales.isnan(), want.isnan()) and torch.equal(scales.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("t,k,delta", [(1220, 6144, "bf16"), (1218, 8192, "f16"), (1216, 11264, "bf16")])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 3e38])
def test_far_rows_among_rows_copied_ahead(tq, t, k, delta, eps):
    g = gen(k)
    x, d = rows_of_all_sizes(g, t, k, delta)
    near = torch.arange(t, device="cuda") % 4 != 1
    x[near], d[near] = even(g, t, k)[near], even(g, t, k).to(d.dtype)[near]
    eps = float(torch.tensor(eps, dtype=torch.float32))
    y, q8 = check(tq, x, d, None, eps, in_place=False)
    z, p8 = check(tq, x, d, None, eps, in_place=True)
    assert torch.equal(y, z) and torch.equal(q8, p8)
    only = torch.empty_like(y)  # x' is not kept: it is formed again
    tq.tq1_rms_norm(x, None, eps, y=only, delta=d)
    assert torch.equal(only, y)
