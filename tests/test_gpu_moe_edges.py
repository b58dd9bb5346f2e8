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


# ---- sigmoid gradients at the ends of the range --------------------------------------------
def _sigmoid_backward(x, ids, g, renormalise, scale):
    """-> (dlogits, the sizes of the terms of each element), 64 bits; 1 - s as the sigmoid of -x."""
    x = x.astype(np.float64)
    with np.errstate(over="ignore"):
        s, rest = 1.0 / (1.0 + np.exp(-x)), 1.0 / (1.0 + np.exp(x))
    g = g.astype(np.float64) * scale
    top = np.take_along_axis(s, ids, 1)
    size = np.abs(g) * top
    own = g * top
    if renormalise:
        r = top / top.sum(axis=1, keepdims=True)
        size = (np.abs(g) + (np.abs(g) * r).sum(axis=1, keepdims=True)) * r
        own = (g - (g * r).sum(axis=1, keepdims=True)) * r
    rest = np.take_along_axis(rest, ids, 1)
    want, bound = np.zeros_like(x), np.zeros_like(x)
    np.put_along_axis(want, ids, own * rest, 1)
    np.put_along_axis(bound, ids, size * rest, 1)
    return want, bound


def _sigmoid_case(dg, x, ids, g, renormalise, scale, bf16):
    dx = dg.moe_route_backward(_device(x, bf16), to_dev(ids), to_dev(g), dg.SCORES_SIGMOID, renormalise=renormalise,
                               scale=scale).float().cpu().numpy().astype(np.float64)
    want, bound = _sigmoid_backward(x, ids, g, renormalise, scale)
    # the exponential (2 units), the sum and the quotient of each of two sigmoids, the sums over the choices and the
    # products between them: some topk + 16 roundings, each of the terms' sizes; subnormal numbers have a step of 2^-149
    topk = ids.shape[1]
    tol = 2 * (topk + 16) * U32 * bound + 2.0 ** -148 * (1 + np.abs(g).max() * scale) + (UBF * np.abs(want) if bf16 else 0)
    assert np.isfinite(dx).all()
    assert (np.abs(dx - want) <= tol).all(), float((np.abs(dx - want) / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("renormalise", [False, True])
def test_sigmoid_gradient_of_confident_scores(dg, renormalise, bf16):
    say("sigmoid gradient renormalise=%s bf16=%s" % (renormalise, bf16))
    rng = np.random.default_rng(4)
    x = rng.choice(np.array([10, 12, 16, 17, 20, 30, 60, 80, 1, -1, -10, -30, -60], np.float32), (40, 64))
    ids = np.argsort(rng.random((40, 64)), axis=1)[:, :6].astype(np.int32)
    g = rng.standard_normal((40, 6)).astype(np.float32)
    _sigmoid_case(dg, x, ids, g, renormalise, 2.5, bf16)


@pytest.mark.parametrize("bf16", [False, True])
def test_sigmoid_gradient_of_vanishing_scores(dg, bf16):
    # renormalised weights do not vanish with the scores: s of 1e-37 and less, their sum's reciprocal past fp32
    say("sigmoid gradient of vanishing scores bf16=%s" % bf16)
    rng = np.random.default_rng(5)
    x = rng.choice(np.array([-84, -86, -87, -88], np.float32), (40, 64))
    x[:5] = -88
    ids = np.argsort(rng.random((40, 64)), axis=1)[:, :6].astype(np.int32)
    g = (rng.standard_normal((40, 6)) * 100).astype(np.float32)
    x64 = x.astype(np.float64)
    s = 1.0 / (1.0 + np.exp(-x64))
    r = np.take_along_axis(s, ids, 1)
    steps = 2.0 ** -149 / r.min()               # what a subnormal score is good for
    assert steps < 2.0 ** -21
    dx = dg.moe_route_backward(_device(x, bf16), to_dev(ids), to_dev(g), dg.SCORES_SIGMOID, scale=2.5)
    dx = dx.float().cpu().numpy().astype(np.float64)
    want, bound = _sigmoid_backward(x, ids, g, True, 2.5)
    # a score, its share of the sum and the sum over the shares each carry that step
    tol = (4 * steps + 2 * (6 + 16) * U32) * bound + (UBF * np.abs(want) if bf16 else 0)
    assert np.isfinite(dx).all()
    assert (np.abs(dx - want) <= tol).all()


# ---- infinities and NaN among the logits ---------------------------------------------------
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("how", [dict(), dict(bias=True), dict(groups=10, topk_groups=3, group_top=2),
                                 dict(bias=True, groups=2, topk_groups=1)], ids=str)
def test_softmax_rows_with_an_infinity_weigh_nan(dg, how, renormalise):
    how, E = dict(how), 130
    x = np.random.default_rng(7).standard_normal((7, E)).astype(np.float32)
    x[1, 100] = x[2, 0] = x[5, 129] = np.inf
    x[3, 64] = np.nan
    if how.pop("bias", False):
        how["bias"] = to_dev(np.linspace(0.01, 0.0, E).astype(np.float32))
    for bf16 in (False, True):
        ids, w = dg.moe_route(_device(x, bf16), 5, dg.SCORES_SOFTMAX, renormalise=renormalise, **how)
        ids, w = ids.cpu().numpy(), w.cpu().numpy()
        assert (ids >= 0).all() and (ids < E).all() and all(len(set(r)) == 5 for r in ids.tolist())
        assert np.isnan(w[[1, 2, 3, 5]]).all()
        assert np.isfinite(w[[0, 4, 6]]).all()


@pytest.mark.parametrize("T,E", [(6, 130), (5, 256), (7, 600)])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_softmax_gradient_of_rows_whose_weights_are_nan(dg, bf16, renormalise, T, E):
    # the weights of such a row are NaN, whichever expert brought it, and so is their gradient
    say("softmax gradient of NaN rows E=%d renormalise=%s bf16=%s" % (E, renormalise, bf16))
    x = np.random.default_rng(8).standard_normal((T, E)).astype(np.float32)
    x[1, E - 1], x[2, 3], x[3, E // 2] = np.nan, np.inf, -np.inf
    ids = np.tile(np.array([5, 9, 11], np.int32), (T, 1))  # none of those
    g = np.random.default_rng(9).standard_normal((T, 3)).astype(np.float32)
    dx = dg.moe_route_backward(_device(x, bf16), to_dev(ids), to_dev(g), dg.SCORES_SOFTMAX, renormalise=renormalise)
    dx = dx.float().cpu().numpy()
    assert np.isnan(dx[[1, 2]]).all()
    keep = [t for t in range(T) if t not in (1, 2)]
    assert np.isfinite(dx[keep]).all() and (dx[keep][:, [5, 9, 11]] != 0).any()


# ---- more workgroups than one launch holds -------------------------------------------------
WORKGROUPS = (1 << 24) + 1  # of 256 threads, 2^32 threads and more


def test_routing_more_tokens_than_one_launch_holds(dg):
    T = WORKGROUPS * 8 - 3                      # 8 tokens to a workgroup
    say("routing of %d tokens" % T)
    x = torch.randn((T, 2), device=dev(), dtype=torch.bfloat16)
    ids, w = dg.moe_route(x, 1, dg.SCORES_SIGMOID, renormalise=False)
    assert torch.equal(ids[:, 0], (x[:, 1] > x[:, 0]).int())
    g = torch.randn((T, 1), device=dev())
    dx = dg.moe_route_backward(x, ids, g, dg.SCORES_SIGMOID, renormalise=False)
    assert bool((dx.gather(1, 1 - ids.long()) == 0).all())
    top = x.gather(1, ids.long()).float()
    assert bool(((w - torch.sigmoid(top)).abs() <= 1e-6).all())
    assert bool(((dx.gather(1, ids.long()).float() - g * torch.sigmoid(top) * torch.sigmoid(-top)).abs()
                 <= 2.0 ** -8 * g.abs()).all())


def test_moving_more_tokens_than_one_launch_holds(dg):
    H, rows = 128, 128
    T = WORKGROUPS * 4 - 1                      # a token to a wave
    say("moving %d tokens" % T)
    at = torch.tensor([0, T // 2, ((1 << 24) - 8) * 4 - 1, ((1 << 24) - 8) * 4, T - 2, T - 1], device=dev())
    n = len(at)
    pos = torch.full((T, 1), -1, dtype=torch.int32, device=dev())
    pos[at, 0] = torch.arange(n, dtype=torch.int32, device=dev())
    w = torch.full((T, 1), 2.0, device=dev())
    y = torch.randn((rows, H), device=dev()).to(torch.bfloat16)
    out = torch.full((T, H), 3.0, dtype=torch.bfloat16, device=dev())
    dg.moe_combine(y, pos, w, out=out)
    assert torch.equal(out[at], (2.0 * y[:n].float()).to(torch.bfloat16))
    assert int(torch.stack([out[i:i + (1 << 22)].count_nonzero() for i in range(0, T, 1 << 22)]).sum()) == int(
        y[:n].count_nonzero())
    row_pair = torch.full((rows,), -1, dtype=torch.int32, device=dev())
    row_pair[:n] = at.int()
    out.copy_(torch.randn((1, H), device=dev()).expand(T, H))
    out[at] = torch.randn((n, H), device=dev()).to(torch.bfloat16)
    dy = torch.full((rows, H), 3.0, dtype=torch.bfloat16, device=dev())
    _, dw = dg.moe_combine_backward(out, y, pos, row_pair, w, dy=dy)
    assert torch.equal(dy[:n], (2.0 * out[at].float()).to(torch.bfloat16)) and bool((dy[n:] == 0).all())
    want = (out[at].double() * y[:n].double()).sum(1)
    assert bool(((dw[at, 0].double() - want).abs() <= 1e-5 * out[at].double().norm(dim=1) * y[:n].double().norm(dim=1)).all())
    dw[at] = 0
    assert int(dw.count_nonzero()) == 0
    q, sf = dg.moe_dispatch_fp8(out, pos, row_pair)
    want_q, want_s = dg.cast_fp8_per_token(out[at])
    assert torch.equal(q[:n], want_q) and torch.equal(sf[:, :n], want_s)
    assert bool((q[n:] == 0).all()) and bool((sf[:, n:] == 0).all())


def test_chunks_of_nan_alone_stay_nan(dg):
    # a power-of-two scale of such a chunk is NaN, as its fp32 scale is; it does not turn into zeros
    say("chunks of NaN alone")
    x = np.random.default_rng(10).standard_normal((128, 256)).astype(np.float32)
    x[3, 128:] = np.nan
    rows = np.random.default_rng(11).standard_normal((128, 256)).astype(np.float32)
    rows[:, 7] = -np.nan
    pos, row_pair, _ = dg.moe_layout_masked(torch.zeros((128, 1), dtype=torch.int32, device=dev()), 1, 128)
    for bf16 in (False, True):
        for ue8m0 in (False, True):
            q, sf = (t[0].cpu().numpy() for t in dg.moe_dispatch_fp8(_device(x, bf16), pos, row_pair, ue8m0=ue8m0))
            assert ((q[3, 128:] & 0x7F) == 0x7F).all() and np.isnan(sf[1, 3])
            assert np.isfinite(sf).sum() == sf.size - 1 and ((q & 0x7F) == 0x7F).sum() == 128
            q, sf = (t.cpu().numpy() for t in dg.cast_fp8_per_channel(_device(rows, bf16), ue8m0=ue8m0))
            assert ((q[7] & 0x7F) == 0x7F).all() and np.isnan(sf[0, 7])
            assert np.isfinite(sf).sum() == sf.size - 1 and ((q & 0x7F) == 0x7F).sum() == 128
