"""The type of the weight gradient, and what it is worth: an fp32 result is as exact as fp32 sums of exact
products are, a bf16 one is rounded to bf16 and made when the caller asks for it."""
import numpy as np
import pytest
import torch

import moe_reference as ref
import oracle
from helpers import dev, say, to_dev
from test_gpu_wgrad import SHAPES as EVERY_SHAPE, _check as check_fp8_sums, _operands as operands_with_zeros

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import moe_grouped_gemm_e4m3_amd as m
    m.lib()
    return m


def _operands(N, K, M, seed, ue8m0):
    """Codes and scales as a cast would leave them."""
    rng = np.random.default_rng(seed)
    dy, x = rng.standard_normal((M, N)).astype(np.float32), rng.standard_normal((M, K)).astype(np.float32)
    (a, sa), (b, sb) = (oracle.cast_per_token(np.ascontiguousarray(t.T), pow2=ue8m0) for t in (dy, x))
    return a, np.ascontiguousarray(sa.T), b, np.ascontiguousarray(sb.T)


@pytest.mark.parametrize("groups", [(128,), (256, 0, 128)], ids=str)
def test_the_result_is_fp32_unless_the_caller_says_bf16(dg, groups):
    N, K = 256, 384
    offsets = np.concatenate([[0], np.cumsum(groups)]).astype(np.int32)
    dd = [to_dev(t) for t in _operands(N, K, int(offsets[-1]), 1, False)]
    off = to_dev(offsets)
    shape = (len(groups), N, K)
    want = dg.grouped_gemm_wgrad(*dd, off, dtype=torch.float32)
    d = dg.grouped_gemm_wgrad(*dd, off)
    assert d.dtype == torch.float32 and torch.equal(d, want)
    for said in (dict(dtype=torch.bfloat16), dict(c=torch.zeros(shape, dtype=torch.bfloat16, device=dev())),
                 dict(d=torch.empty(shape, dtype=torch.bfloat16, device=dev()))):
        h = dg.grouped_gemm_wgrad(*dd, off, **said)
        assert h.dtype == torch.bfloat16
        # within a bf16 rounding, and a little for other sums
        assert ((h.float() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -12 * want.abs().max()).all()
    for said in (dict(c=torch.zeros(shape, device=dev())), dict(d=torch.empty(shape, device=dev()))):
        assert torch.equal(dg.grouped_gemm_wgrad(*dd, off, **said), want)


@pytest.mark.parametrize("N,K,groups", EVERY_SHAPE, ids=str)
@pytest.mark.parametrize("ue8m0", [False, True])
def test_bf16_results(dg, N, K, groups, ue8m0):
    say("wgrad bf16 N=%d K=%d groups=%s ue8m0=%s" % (N, K, groups, ue8m0))
    offsets = np.concatenate([[0], np.cumsum(groups)]).astype(np.int32)
    ops = operands_with_zeros(N, K, int(offsets[-1]) + 128, N + K, ue8m0)
    dd, off = [to_dev(t) for t in ops], to_dev(offsets)
    h = dg.grouped_gemm_wgrad(*dd, off, dtype=torch.bfloat16, ue8m0=ue8m0)
    check_fp8_sums(h, *ops, offsets)
    assert all((h[g] == 0).all() for g, rows in enumerate(groups) if rows == 0)
    c = to_dev(np.random.default_rng(1).standard_normal(h.shape).astype(np.float32)).to(torch.bfloat16)
    kept = c.clone()
    e = dg.grouped_gemm_wgrad(*dd, off, c=c, ue8m0=ue8m0)
    check_fp8_sums(e, *ops, offsets, kept.float().cpu().numpy())
    assert torch.equal(c, kept)
    dg.grouped_gemm_wgrad(*dd, off, c=c, d=c, ue8m0=ue8m0)  # in place
    assert torch.equal(c, e)


U = 2.0 ** -23  # of one fp32 addition, to nearest or cut


def _exact(a, sa, b, sb, offsets):
    table = oracle.decode_table().astype(np.float64)
    want, size, _ = ref.wgrad(table[a], sa, table[b], sb, offsets)
    return want, size


def _check_fp32(d, want, size, blocks):
    # Products of two e4m3 values are exact (8 bits). 127 additions in a block, two roundings for its scales, one
    # addition per block and one for c: each is off by at most U of the sum of the terms' sizes.
    err = np.abs(d.cpu().numpy().astype(np.float64) - want)
    assert (err <= (130 + blocks) * U * size).all()
    # In the 2-norm, for terms of random sign: n additions whose partial sums grow like sqrt(i / n) of the result are
    # off by 2^-24 sqrt(n / 6) of it: 4.6 units of 2^-24 for the 128 of a block, 3.7 for up to 80 blocks, 1 for the
    # scales and c; under 10 together, 16 allowed.
    assert np.sqrt((err ** 2).sum()) <= 2.0 ** -20 * np.sqrt((want ** 2).sum())


SHAPES = [
    # N, K, rows per group
    (128, 128, (128,)), (256, 384, (256, 0, 128, 384)), (384, 256, (0, 0, 128)), (640, 128, (128, 128)),
    (256, 256, (1024, 128, 0, 256, 512)), (128, 256, (10240,)), (1152, 896, (384, 256)), (256, 128, (4096, 4096)),
    # more tiles than two for each of 256 compute units: several to a workgroup, groups without rows between
    (1152, 1152, (128, 0, 256, 128, 384, 0, 0, 128, 512)),
]


@pytest.mark.parametrize("N,K,groups", SHAPES, ids=str)
@pytest.mark.parametrize("ue8m0", [False, True])
def test_fp32_results_are_worth_fp32(dg, N, K, groups, ue8m0):
    say("wgrad fp32 N=%d K=%d groups=%s ue8m0=%s" % (N, K, groups, ue8m0))
    offsets = np.concatenate([[0], np.cumsum(groups)]).astype(np.int32)
    ops = _operands(N, K, int(offsets[-1]) + 128, N + K, ue8m0)  # the last rows belong to no group
    dd, off = [to_dev(t) for t in ops], to_dev(offsets)
    want, size = _exact(*ops, offsets)
    blocks = max(groups) // 128
    d = dg.grouped_gemm_wgrad(*dd, off, ue8m0=ue8m0)
    _check_fp32(d, want, size, blocks)
    assert all((d[g] == 0).all() for g, rows in enumerate(groups) if rows == 0)
    c = np.random.default_rng(1).standard_normal(d.shape).astype(np.float32)
    cd = to_dev(c)
    e = dg.grouped_gemm_wgrad(*dd, off, c=cd, ue8m0=ue8m0)
    _check_fp32(e, want + c, size + np.abs(c), blocks)
    assert np.array_equal(cd.cpu().numpy(), c)
    dg.grouped_gemm_wgrad(*dd, off, c=cd, d=cd, ue8m0=ue8m0)  # in place
    assert torch.equal(cd, e)
    # without a workspace the rows are summed in one piece
    whole = dg.grouped_gemm_wgrad(*dd, off, ue8m0=ue8m0, workspace=torch.empty(0, dtype=torch.uint8, device=dev()))
    _check_fp32(whole, want, size, blocks)


def test_products_of_unlike_sizes_survive(dg):
    # 448^2 beside 2^-18 in neighbouring rows, and the large ones cancel: the sum is the small one's
    codes = oracle.encode(np.array([448.0, -448.0, 2.0 ** -9, 0.0], np.float32))
    for at in range(8):
        a, b = np.full((128, 128), codes[3], np.uint8), np.full((128, 128), codes[3], np.uint8)
        one, two, three = at, (at + 1) % 8, (at + 3) % 8
        a[:, one], a[:, two], a[:, three] = codes[0], codes[1], codes[2]
        b[:, one], b[:, two], b[:, three] = codes[0], codes[0], codes[2]
        s = torch.ones((1, 128), device=dev())
        d = dg.grouped_gemm_wgrad(to_dev(a), s, to_dev(b), s)
        # the two large products are 18 bits above; a sum of 24 bits holds 448^2 to 2^-6 (2^17.6 cut at 24 bits)
        assert (d.abs() <= 2.0 ** -6).all()
    # every code times every code, alone in its column: exact
    table = oracle.decode_table().astype(np.float64)
    a, b = np.full((256, 128), codes[3], np.uint8), np.full((256, 128), codes[3], np.uint8)
    a[:, 77] = b[:, 77] = np.arange(256)
    s = torch.ones((1, 256), device=dev())
    d = dg.grouped_gemm_wgrad(to_dev(a), s, to_dev(b), s)[0].cpu().numpy()
    with np.errstate(invalid="ignore"):
        assert np.array_equal(d, (table[:, None] * table[None, :]).astype(np.float32), equal_nan=True)


def test_scales_whose_product_overflows(dg):
    # the product of the two scales is past fp32, the sums are zero or small beside them
    a = np.zeros((128, 128), np.uint8)
    a[3, 5] = oracle.encode(np.array([2.0 ** -9], np.float32))[0]
    b = a.copy()
    sa = torch.full((1, 128), 2.0 ** 72, device=dev())
    sb = torch.full((1, 128), 2.0 ** 72, device=dev())
    d = dg.grouped_gemm_wgrad(to_dev(a), sa, to_dev(b), sb)[0].cpu().numpy()
    want = np.zeros((128, 128))
    want[3, 3] = 2.0 ** (144 - 18)
    assert np.array_equal(d, want)
