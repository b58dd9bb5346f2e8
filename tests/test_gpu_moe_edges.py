"""Values at the edges of the mixture-of-experts operators: signed zeros, confident and vanishing scores,
infinities and NaN, more workgroups than one launch holds."""
import numpy as np
import pytest
import torch

import oracle
from helpers import assert_same_bits, assert_same_bytes, dev, kmajor, say, to_dev

pytestmark = pytest.mark.gpu

U32, UBF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def dg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import moe_grouped_gemm_e4m3_amd as m
    m.lib()
    return m


def _device(x, bf16):
    return to_dev(x).to(torch.bfloat16) if bf16 else to_dev(x)


# ---- signed zeros --------------------------------------------------------------------------
def _with_negative_zeros(M, H, bf16, neighbour, seed):
    """Normal values with -0 among them in every chunk; `neighbour` makes some chunks all zero, of both signs."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, H)).astype(np.float32)
    x[rng.random((M, H)) < 0.2] = -0.0
    x[rng.random((M, H)) < 0.1] = 0.0
    if neighbour:
        x[::2, 128:256] = 0.0
        x[::2, 130] = -0.0
    return torch.from_numpy(x).to(torch.bfloat16).float().numpy() if bf16 else x


@pytest.mark.parametrize("neighbour", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("ue8m0", [False, True])
def test_negative_zeros_keep_their_sign(dg, ue8m0, bf16, neighbour):
    say("negative zeros ue8m0=%s bf16=%s neighbour=%s" % (ue8m0, bf16, neighbour))
    x = _with_negative_zeros(130, 1024, bf16, neighbour, 3)
    qx, sx = oracle.cast_per_token(x, pow2=ue8m0)
    assert (qx == 0x80).any()
    pos, row_pair, _ = dg.moe_layout_masked(torch.zeros((130, 1), dtype=torch.int32, device=dev()), 1, 130)
    q, sf = dg.moe_dispatch_fp8(_device(x, bf16), pos, row_pair, ue8m0=ue8m0)
    assert_same_bytes(q[0], qx, "dispatch")
    assert_same_bits(sf[0], kmajor(sx), "dispatch")
    # along the rows: the same values turned round
    y = np.ascontiguousarray(x[:, :1024].T)      # [1024 rows, 130] -> 128 channels
    y = np.ascontiguousarray(y[:, :128])
    qy, sy = oracle.cast_per_token(np.ascontiguousarray(y.T), pow2=ue8m0)
    q, sf = dg.cast_fp8_per_channel(_device(y, bf16), ue8m0=ue8m0)
    assert_same_bytes(q, qy, "per channel")
    assert_same_bits(sf, np.ascontiguousarray(sy.T), "per channel")
