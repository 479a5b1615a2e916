"""Sums over rows on the GPU with inputs whose sums are whole numbers: every row adds
at least 1 to every channel of every sum, so a row that is lost or counted twice shows
at any size, which a bound on roundings that grows with the row count does not."""
import math

import pytest
import torch

from tests import train_reference as ref
from tests.test_train_gpu import BF, DEV, F32, RNG, ROWS, _rng, ids
from video_diffusion_transformer_rms_b200 import _abi, api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    _abi.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


# the shapes of the other tests, and row counts that end in the middle of a share
SUMS = ROWS + [
    # B, L, n_video, D, dtype
    (1, 9001, 8000, 256, F32),
    (2, 2401, 2399, 512, BF),
    (3, 5003, 1, 648, BF),
    (130, 37, 11, 1152, BF),      # many samples: 260 keys
    (1, 20011, 20011, 64, BF),
    (1, 3001, 2903, 6144, BF),
]


def whole(shape, lo, hi, dt, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV).to(dt)


def counted(got, want, least, slack, what):
    """got is the whole number want to within `slack`, less than half of `least`, the
    least that one row adds (numbers, or one for each channel): a sum without any one row
    is refused."""
    least, slack = (torch.as_tensor(v, dtype=torch.float64, device=DEV) for v in (least, slack))
    assert (least >= 1).all() and (slack < least / 2).all()
    assert got.dtype == torch.float32 and got.shape == want.shape
    far = (got.double() - want).abs()
    assert (far <= slack).all(), f"{what}: off by {float(far.max())}"
    assert ((got.double() - (want - least)).abs() > slack).all()


@pytest.mark.parametrize("case", SUMS, ids=ids)
def test_layer_norm_backward_counts_every_row(case):
    B, L, nv, D, dt = case
    x, dy = whole((B, L, D), 1, 2, dt, 1), whole((B, L, D), 1, 3, dt, 2)
    gamma, beta = whole((D,), 1, 2, dt, 3), whole((D,), 1, 2, dt, 4)
    scale = whole((B, 2, D), 0, 1, dt, 5)
    mean, rstd = torch.zeros((B, L), device=DEV), torch.ones((B, L), device=DEV)
    got = api.layer_norm_backward(dy, x, mean, rstd, gamma, beta, scale, n_video=nv)
    s1, s0 = ref.key_sums((dy * x).double(), nv), ref.key_sums(dy.double(), nv)
    fac = 1 + scale.double()
    assert 12 * B * L < 2 ** 24            # every partial sum is exact in fp32
    counted(got.dshift, s0, 1, 0, "dshift")
    counted(got.dscale, gamma.double() * s1 + beta.double() * s0, 2, 0, "dscale")
    counted(got.dgamma, (fac * s1).sum((0, 1)), 1, 0, "dgamma")
    counted(got.dbeta, (fac * s0).sum((0, 1)), 1, 0, "dbeta")
    # without scale: one sum over all rows
    one = api.layer_norm_backward(dy, x, mean, rstd, gamma, beta, n_video=nv)
    counted(one.dgamma, s1.sum((0, 1)), 1, 0, "dgamma")
    counted(one.dbeta, s0.sum((0, 1)), 1, 0, "dbeta")


@pytest.mark.parametrize("case", SUMS, ids=ids)
@pytest.mark.parametrize("dres", [False, True])
def test_rms_adaln_backward_counts_every_row(case, dres):
    B, L, nv, D, dt = case
    x, dy = torch.ones((B, L, D), dtype=dt, device=DEV), whole((B, L, D), 1, 2, dt, 2)
    gamma, scale = torch.ones((D,), dtype=dt, device=DEV), whole((B, 2, D), 0, 1, dt, 5)
    _, dscale, dshift, dgamma = api.rms_adaln_backward(dy, x, scale, nv, gamma=gamma, eps=0.0,
                                                       dres=dy if dres else None)
    s0 = ref.key_sums(dy.double(), nv)
    # x^ is 1 to within two steps of the reciprocal root and two roundings of the mean
    # (2^-21 together).  A thread adds at most the rows of one share of 148 or more (four
    # in short calls) and then eight groups' sums, a rounding of the sum so far each
    rel = 2 ** -21 + (math.ceil(B * L / 148) + 12) * ref.U32
    counted(dshift, s0, 1, 0, "dshift")
    counted(dscale, s0, 1, s0 * rel, "dscale")
    fac = 1 + scale.double()
    want = (fac * s0).sum((0, 1))
    least = torch.where(s0 > 0, fac, math.inf).amin((0, 1))
    counted(dgamma, want, least, want * rel, "dgamma")


@pytest.mark.parametrize("case", SUMS, ids=ids)
@pytest.mark.parametrize("p", [0.0, 0.5])
def test_dropout_residual_backward_counts_every_row(case, p):
    B, L, nv, D, dt = case
    br, do = whole((B, L, D), 1, 2, dt, 1), whole((B, L, D), 1, 3, dt, 2)
    gate = whole((B, 2, D), 0, 1, dt, 5)
    _, dgate = api.dropout_residual_backward(do, br, gate, nv, p, _rng(), site=3)
    keep = ref.keep_mask(do.numel(), RNG[0], RNG[1] + 3, p, DEV).view(do.shape)
    want = ref.key_sums((do * br * keep).double() / (1 - p), nv)
    counted(dgate, want, 1, 0, "dgate")


@pytest.mark.parametrize("B,L,Hq,Hk,hd,dt", [
    (1, 1, 1, 1, 16, BF), (2, 1, 40, 8, 128, BF), (1, 301, 16, 2, 64, BF), (2, 50, 2, 3, 96, BF),
    (1, 129, 1, 1, 256, BF), (1, 19, 33, 1, 128, F32), (2, 65, 3, 2, 40, F32),
    (2, 2401, 3, 2, 64, BF), (1, 9001, 1, 3, 32, F32), (1, 20011, 2, 1, 128, BF),
    (1, 2369, 5, 4, 72, BF), (3, 1579, 1, 2, 128, F32),
])
@pytest.mark.parametrize("half", [False, True])
def test_rope_axes_backward_counts_every_head_of_every_row(B, L, Hq, Hk, hd, dt, half):
    if half and hd // 2 % (8 if dt == BF else 4):
        half = False
    q, k = (torch.ones((B, L, H, hd), dtype=dt, device=DEV) for H in (Hq, Hk))
    dq, dk = whole(q.shape, 1, 2, dt, 1), whole(k.shape, 1, 2, dt, 2)
    gq, gk = whole((hd,), 1, 2, dt, 3), whole((hd,), 1, 2, dt, 4)
    plan = api.RopeAxes(hd, (hd // 2,), half_split=half)
    pos = torch.zeros((1, L), dtype=torch.int32, device=DEV)      # the turn by 0 is exact
    r = api.rope_axes_backward(dq, dk, pos, plan, q, k, gq, gk, qk_norm=True, eps=0.0)
    for got, d, H in ((r.dgamma_q, dq, Hq), (r.dgamma_k, dk, Hk)):
        # as above; a lane adds at most all heads of its warp's rows, of which each warp of
        # 148 or more CTAs of 8 has ceil(rows / 1,184) at most; then a thread the groups of
        # lanes, 256 over the power of two that holds a head's vectors
        lanes = 2 ** max(1, math.ceil(math.log2(hd / (8 if dt == BF else 4))))
        rel = 2 ** -21 + (math.ceil(B * L / 1184) * H + 256 // lanes) * ref.U32
        want = d.double().sum((0, 1, 2))
        counted(got, want, 1, want * rel, "dgamma")
