"""The type of the weight gradient, and what it is worth: an fp32 result is as exact as fp32 sums of exact
products are, a bf16 one is rounded to bf16 and made when the caller asks for it."""
import numpy as np
import pytest
import torch

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
