"""Training operators on the GPU against their definitions in 64 bits
(tests/train_reference.py): sizes from one row up, ragged widths and row counts,
one modality empty, strides, grouped heads, aliasing, guard bytes, captured
graphs, side streams, and a block's forward and backward pass as a whole."""
import pytest
import torch

from tests import train_reference as ref
from video_diffusion_transformer_rms_b200 import _abi, api
from video_diffusion_transformer_rms_b200.workloads import WORKLOADS, activation, vectors

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    _abi.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def act(B, L, D, dt, seed, outliers=True, offset=0.0):
    t = activation(max(B * L, 1), D, torch.float32, DEV, seed, outliers=outliers)[:B * L]
    return (t + offset).to(dt).view(B, L, D)


def vec(shape, mean, std, dt, seed):
    return vectors(shape, mean, std, dt, DEV, seed)


ROWS = [
    # B, L, n_video, D, dtype
    (1, 1, 1, 8, BF),             # one vector, one row
    (1, 1, 0, 4, F32),
    (1, 56, 48, 256, F32),        # the tiny workload
    (2, 3, 1, 264, BF),
    (3, 37, 20, 5128, BF),        # ragged width: 641 vectors
    (2, 300, 0, 4096, BF),        # one modality without rows
    (2, 301, 301, 2056, BF),
    (5, 1, 1, 640, BF),           # one row per sample
    (1, 33, 16, 16384, BF),       # widest rows
    (1, 17, 5, 8192, F32),
    (1, 4099, 4000, 128, BF),     # many more rows than CTAs
    (7, 613, 600, 1000, F32),
    (1, 1201, 1100, 5120, BF),
    (40, 9, 5, 264, BF),          # more (sample, modality) keys than a CTA of the join takes
]
ids = lambda c: "x".join(str(v).replace("torch.", "") for v in c)  # noqa: E731


@pytest.mark.parametrize("case", ROWS, ids=ids)
@pytest.mark.parametrize("affine,mod", [(True, True), (True, False), (False, True),
                                        (False, False)])
def test_layer_norm(case, affine, mod):
    B, L, nv, D, dt = case
    x = act(B, L, D, dt, D + L, offset=3.0)
    g = vec((D,), 1.0, 0.1, dt, 1) if affine else None
    b = vec((D,), 0.0, 0.3, dt, 2) if affine else None
    sc = vec((B, 2, D), 0.0, 0.5, dt, 3) if mod else None
    sh = vec((B, 2, D), 0.0, 0.5, dt, 4) if mod else None
    y, mean, rstd = api.layer_norm(x, g, b, sc, sh, n_video=nv, eps=EPS)
    wy, wm, wr = ref.layer_norm(x, g, b, sc, sh, nv, EPS)
    depth = ref.depth_row(D)
    ref.check(mean, wm, depth, "mean")
    ref.check(rstd, wr, depth, "rstd")
    ref.check(y, wy, depth, "y")


@pytest.mark.parametrize("D", [1160, 2056, 2568, 3592, 4616, 6664, 8208, 10248, 12296, 14344])
def test_layer_norm_of_ragged_widths(D):
    # every split of a row over threads, its last vectors missing
    B, L, nv = 2, 75, 70
    x, dy = act(B, L, D, BF, D), act(B, L, D, BF, D + 1, outliers=False)
    sc, sh = vec((B, 2, D), 0, 0.5, BF, 3), vec((B, 2, D), 0, 0.5, BF, 4)
    y, mean, rstd = api.layer_norm(x, scale=sc, shift=sh, n_video=nv, eps=EPS)
    want, wm, wr = ref.layer_norm(x, None, None, sc, sh, nv, EPS)
    for got, w, what in ((y, want, "y"), (mean, wm, "mean"), (rstd, wr, "rstd")):
        ref.check(got, w, ref.depth_row(D), what)
    got = api.layer_norm_backward(dy, x, mean, rstd, scale=sc, n_video=nv)
    want = ref.norm_backward(dy, x, mean, rstd, None, None, sc, None, nv, EPS, False)
    ref.check(got.dx, want["dx"], ref.depth_row(D), "dx")
    ref.check(got.dscale, want["dscale"], ref.depth_rows(B * L), "dscale")
    ref.check(got.dshift, want["dshift"], ref.depth_rows(B * L), "dshift")


@pytest.mark.parametrize("D,dt", [(1024, BF), (1016, BF), (8192, BF), (8184, BF), (512, F32),
                                  (4096, F32), (6144, BF)])
def test_layer_norm_of_full_and_almost_full_widths(D, dt):
    # 32 x 4 and 256 x 4 vectors, filled and one vector short; 1536 vectors do for three
    # vectors per thread in the gradients
    B, L, nv = 2, 75, 70
    x, dy = act(B, L, D, dt, D), act(B, L, D, dt, D + 1, outliers=False)
    g, b = vec((D,), 1, 0.1, dt, 1), vec((D,), 0, 0.3, dt, 2)
    sc, sh = vec((B, 2, D), 0, 0.5, dt, 3), vec((B, 2, D), 0, 0.5, dt, 4)
    y, mean, rstd = api.layer_norm(x, g, b, sc, sh, n_video=nv, eps=EPS)
    want, wm, wr = ref.layer_norm(x, g, b, sc, sh, nv, EPS)
    for got, w, what in ((y, want, "y"), (mean, wm, "mean"), (rstd, wr, "rstd")):
        ref.check(got, w, ref.depth_row(D), what)
    for dres in (None, act(B, L, D, dt, D + 2)):
        t = dict(x=x, dy=dy, gamma=g, beta=b, scale=sc, dres=dres)
        got = api.layer_norm_backward(dy, x, mean, rstd, g, b, sc, n_video=nv, dres=dres)
        want = ref.norm_backward(dy, x, mean, rstd, g, b, sc, dres, nv, EPS, False)
        _check_norm_grads(got._asdict(), want, (B, L, nv, D, dt), t)


# every count of vectors per thread of the gradients, full (an instantiation without
# guards in the RMS form) and ragged
@pytest.mark.parametrize("D,dt", [(256, BF), (248, BF), (1024, BF), (2056, BF), (5120, BF),
                                  (5128, BF), (6144, BF), (10248, BF), (12288, BF), (12296, BF),
                                  (14344, BF), (16384, BF), (16376, BF), (6148, F32), (8192, F32)])
@pytest.mark.parametrize("dres", [False, True])
def test_rms_adaln_backward_of_every_width(D, dt, dres):
    case = (2, 75, 70, D, dt)
    t, want = _norm_case(case, True, True, True, dres)
    dx, dscale, dshift, dgamma = api.rms_adaln_backward(t["dy"], t["x"], t["scale"], 70,
                                                        gamma=t["gamma"], eps=EPS,
                                                        dres=t["dres"])
    _check_norm_grads(dict(dx=dx, dscale=dscale, dshift=dshift, dgamma=dgamma), want, case, t)


@pytest.mark.parametrize("D,dt", [(8, BF), (264, BF), (5120, BF), (5128, BF), (1000, F32),
                                  (16384, BF)])
def test_norms_keep_bad_rows_to_themselves(D, dt):
    # an Inf or NaN in one element makes its row bad, and the channel's or the whole
    # sums, but no other row, whatever shares its warp, ring or CTA
    B, L, nv = 2, 61, 40
    x, dy = act(B, L, D, dt, D), act(B, L, D, dt, D + 1, outliers=False)
    sc, sh = vec((B, 2, D), 0, 0.5, dt, 3), vec((B, 2, D), 0, 0.5, dt, 4)
    rows = [(0, 0), (0, 33), (0, L - 1), (1, 7)]
    bx, bdy = x.clone(), dy.clone()
    good = torch.ones((B, L), dtype=torch.bool, device=DEV)
    for i, (b, r) in enumerate(rows):
        bx[b, r, (5 * i) % D] = (INF, NAN, -INF, INF)[i]
        bdy[b, (r + 3) % L, i % D] = (NAN, INF, INF, -INF)[i]
        good[b, r] = good[b, (r + 3) % L] = False
    fx = torch.isfinite(bx).all(-1)
    clean = api.layer_norm(x, scale=sc, shift=sh, n_video=nv)
    got = api.layer_norm(bx, scale=sc, shift=sh, n_video=nv)
    for a, b in zip(got, clean):
        assert torch.equal(a[fx], b[fx])
    assert torch.isnan(got[0][~fx]).any(-1).all()
    args = dict(scale=sc, n_video=nv)
    a = api.layer_norm_backward(dy, x, clean[1], clean[2], **args).dx
    b = api.layer_norm_backward(bdy, bx, *got[1:], **args).dx
    assert torch.equal(a[good], b[good]) and not torch.isfinite(b[~good]).all(-1).any()
    a = api.rms_adaln_backward(dy, x, sc, nv)[0]
    b, _, dshift, _ = api.rms_adaln_backward(bdy, bx, sc, nv)
    assert torch.equal(a[good], b[good]) and not torch.isfinite(b[~good]).all(-1).any()
    # the sums of dy alone: bad in the channels that hold something bad, elsewhere not
    want = ref.key_sums(bdy.double(), nv)
    assert torch.equal(torch.isfinite(dshift), torch.isfinite(want))


def test_layer_norm_of_a_row_far_from_zero():
    # spread 1 about a mean of 4096: mean(x^2) - mean^2 would lose it in fp32
    x = act(2, 5, 1024, F32, 9, outliers=False, offset=4096.0)
    y, mean, rstd = api.layer_norm(x)
    wy, wm, wr = ref.layer_norm(x, None, None, None, None, 5, EPS)
    # a warp's mean passes 14 additions (8 in a lane, 5 joins, the lane's halves), the
    # join of the warps a few more: 20 roundings of 2^-24 of 4096 at most, which y sees
    # as they are and rstd squared
    assert (y.double() - wy[0]).abs().max() <= 20 * 2 ** -12
    assert ((rstd.double() - wr[0]) / wr[0]).abs().max() <= (20 * 2 ** -12) ** 2 + 2 ** -17
    # constant rows: no spread at all, y is the shift
    c = torch.full((1, 3, 256), 7.0, device=DEV)
    y, _, rstd = api.layer_norm(c, beta=vec((256,), 0.0, 1.0, F32, 1), eps=1e-6)
    assert torch.equal(y, vec((256,), 0.0, 1.0, F32, 1).expand(1, 3, 256))
    assert torch.allclose(rstd, torch.full_like(rstd, 1e3), rtol=1e-6)


def _norm_case(case, rms, affine=True, mod=True, dres=True):
    B, L, nv, D, dt = case
    x = act(B, L, D, dt, D + L, offset=0.0 if rms else 1.0)
    dy = act(B, L, D, dt, D + L + 1, outliers=False)
    t = dict(x=x, dy=dy, gamma=vec((D,), 1.0, 0.1, dt, 1) if affine else None,
             beta=vec((D,), 0.0, 0.3, dt, 2) if affine and not rms else None,
             scale=vec((B, 2, D), 0.0, 0.5, dt, 3) if mod else None,
             dres=act(B, L, D, dt, D + L + 2) if dres else None)
    if not rms:
        xd = x.double()
        t["mean"] = xd.mean(-1).float()
        t["rstd"] = (1.0 / torch.sqrt(xd.var(-1, correction=0) + EPS)).float()
    want = ref.norm_backward(dy, x, t.get("mean"), t.get("rstd"), t["gamma"], t["beta"],
                             t["scale"], t["dres"], nv, EPS, rms)
    return t, want


def _check_norm_grads(got, want, case, t):
    B, L, nv, D, dt = case
    ref.check(got["dx"], want["dx"], ref.depth_row(D), "dx")
    depth = ref.depth_rows(B * L)
    for n, given in (("dgamma", t["gamma"]), ("dbeta", t["beta"]), ("dscale", t["scale"]),
                     ("dshift", t["scale"])):
        if given is None:
            assert got.get(n) is None
        else:
            assert got[n].dtype == torch.float32
            ref.check(got[n], want[n], depth, n)


@pytest.mark.parametrize("case", ROWS, ids=ids)
@pytest.mark.parametrize("affine,mod,dres", [(True, True, False), (True, False, True),
                                             (False, True, True), (False, False, False)])
def test_layer_norm_backward(case, affine, mod, dres):
    t, want = _norm_case(case, False, affine, mod, dres)
    got = api.layer_norm_backward(t["dy"], t["x"], t["mean"], t["rstd"], t["gamma"], t["beta"],
                                  t["scale"], n_video=case[2], dres=t["dres"])
    _check_norm_grads(got._asdict(), want, case, t)


@pytest.mark.parametrize("case", ROWS, ids=ids)
@pytest.mark.parametrize("affine,dres", [(True, False), (False, True)])
def test_rms_adaln_backward(case, affine, dres):
    t, want = _norm_case(case, True, affine, True, dres)
    dx, dscale, dshift, dgamma = api.rms_adaln_backward(t["dy"], t["x"], t["scale"], case[2],
                                                        gamma=t["gamma"], eps=EPS,
                                                        dres=t["dres"])
    _check_norm_grads(dict(dx=dx, dscale=dscale, dshift=dshift, dgamma=dgamma), want, case, t)


def test_norm_backward_in_place_guards_and_repeats():
    case = (2, 77, 50, 1032, BF)
    t, want = _norm_case(case, False)
    args = (t["mean"], t["rstd"], t["gamma"], t["beta"], t["scale"])
    first = api.layer_norm_backward(t["dy"], t["x"], *args, n_video=50, dres=t["dres"])
    for name in ("dy", "x", "dres"):
        u = {n: t[n].clone() for n in ("dy", "x", "dres")}
        again = api.layer_norm_backward(u["dy"], u["x"], *args, n_video=50, dres=u["dres"],
                                        dx=u[name])
        for a, b in zip(first, again):
            assert torch.equal(a, b)     # the same bits, in place or not
    # a workspace full of NaN and a guarded output
    need = _abi.sol_norm_backward_workspace_bytes(2, 77, 1032)
    ws = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=DEV)
    buf = torch.full((t["x"].numel() + 4096,), 5.0, dtype=BF, device=DEV)
    dx = buf[2048:-2048].view_as(t["x"])
    again = api.layer_norm_backward(t["dy"], t["x"], *args, n_video=50, dres=t["dres"], dx=dx,
                                    workspace=ws[:need])
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    assert torch.all(buf[:2048] == 5.0) and torch.all(buf[-2048:] == 5.0)
    assert torch.all(ws[need:] == 0xFF)


@pytest.mark.parametrize("B,L", [(0, 5), (2, 0)])
def test_zero_rows(B, L):
    x = torch.empty((B, L, 64), device=DEV)
    g, sc = torch.ones(64, device=DEV), torch.zeros((B, 2, 64), device=DEV)
    y, mean, rstd = api.layer_norm(x, g, g, sc, sc, n_video=0)
    assert y.shape == x.shape and mean.shape == (B, L)
    got = api.layer_norm_backward(x, x, mean, rstd, g, g, sc, n_video=0)
    assert torch.all(got.dgamma == 0) and torch.all(got.dbeta == 0)
    assert got.dscale.shape == (B, 2, 64) and torch.all(got.dscale == 0)
    rng = torch.tensor([1, 2], device=DEV)
    d, dg = api.dropout_residual_backward(x, x, sc, 0, 0.5, rng)
    assert d.shape == x.shape and torch.all(dg == 0)
    assert api.dropout(x, 0.5, rng).shape == x.shape
    q = torch.empty((B, L, 2, 64), device=DEV)
    plan = api.RopeAxes(64, (16, 16))
    pos = torch.zeros((2, B, L), dtype=torch.int32, device=DEV)
    gq = torch.ones(64, device=DEV)
    a, b = api.rope_axes(q, q, pos, plan, gq, gq, qk_norm=True)
    assert a.shape == q.shape and b.shape == q.shape
    r = api.rope_axes_backward(a, b, pos, plan, q, q, gq, gq, qk_norm=True)
    assert torch.all(r.dgamma_q == 0) and torch.all(r.dgamma_k == 0)


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------

RNG = (0x1234567890ABCDEF, 2 ** 40 + 17)


def _rng(seed=RNG[0], offset=RNG[1]):
    to = lambda v: v - 2 ** 64 if v >= 2 ** 63 else v  # noqa: E731
    return torch.tensor([to(seed), to(offset)], dtype=torch.int64, device=DEV)


@pytest.mark.parametrize("case", ROWS, ids=ids)
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5])
def test_dropout_residual(case, p):
    B, L, nv, D, dt = case
    h, br = act(B, L, D, dt, D), act(B, L, D, dt, D + 1)
    gate = vec((B, 2, D), 0.0, 0.3, dt, 5)
    y = ref.dropped(br, RNG, 7, p)
    gf = ref.spread(gate, nv, L)
    rng = _rng()
    for hh, gg in ((h, gate), (None, gate), (h, None), (None, None)):
        out = api.dropout_residual(hh, br, gg, nv, p, rng, site=7)
        v = (y * gf if gg is not None else y) + (hh.double() if hh is not None else 0.0)
        mag = (y * gf).abs() if gg is not None else y.abs()
        ref.check(out, (v, mag + (hh.double().abs() if hh is not None else 0.0)), 4, "out")
    assert torch.equal(api.dropout(br, p, rng, site=7),
                       api.dropout_residual(None, br, None, nv, p, rng, site=7))
    # in place on either input
    want = api.dropout_residual(h, br, gate, nv, p, rng, site=7)
    for t in ("h", "br"):
        hc, bc = h.clone(), br.clone()
        got = api.dropout_residual(hc, bc, gate, nv, p, rng, site=7, out=hc if t == "h" else bc)
        assert torch.equal(got, want)


@pytest.mark.parametrize("case", ROWS, ids=ids)
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_dropout_residual_backward(case, p):
    B, L, nv, D, dt = case
    do, br = act(B, L, D, dt, D, outliers=False), act(B, L, D, dt, D + 1)
    gate = vec((B, 2, D), 0.0, 0.3, dt, 5)
    rng = _rng()
    d = ref.dropped(do, RNG, 3, p)
    gf = ref.spread(gate, nv, L)
    dbranch, dgate = api.dropout_residual_backward(do, br, gate, nv, p, rng, site=3)
    ref.check(dbranch, (d * gf, (d * gf).abs()), 4, "dbranch")
    prod = d * br.double()
    ref.check(dgate, (ref.key_sums(prod, nv), ref.key_sums(prod.abs(), nv)),
              ref.depth_rows(B * L), "dgate")
    # without the gate's gradient, and in place
    again, none = api.dropout_residual_backward(do, None, None, nv, p, rng, site=3)
    assert none is None and torch.equal(again, api.dropout(do, p, rng, site=3))
    for i in range(2):
        c = [do.clone(), br.clone()]
        a, b = api.dropout_residual_backward(c[0], c[1], gate, nv, p, rng, site=3, dbranch=c[i])
        assert torch.equal(a, dbranch) and torch.equal(b, dgate)


@pytest.mark.parametrize("case", ROWS, ids=ids)
@pytest.mark.parametrize("p", [0.1, 0.25])
def test_dropout_gradient_rounds_in_the_order_of_its_formula(case, p):
    # gate * (dout / (1 - p)): the quotient is rounded to fp32, then the product, then the
    # output.  Many of the exact results are ties of bf16 (p = 1/4: all whose factors have
    # a 3), which another order rounds the other way.
    B, L, nv, D, dt = case
    do, br = act(B, L, D, dt, D, outliers=False), act(B, L, D, dt, D + 1)
    gate = vec((B, 2, D), 0.0, 0.3, dt, 5)
    rng = _rng()
    keep = ref.keep_mask(do.numel(), RNG[0], RNG[1] + 3, ref.p32(p), DEV).view_as(do)
    ks = torch.tensor(1.0 / (1.0 - ref.p32(p)), dtype=torch.float32, device=DEV)
    want = ref.spread(gate, nv, L).float() * (do.float() * ks)
    want = torch.where(keep, want, torch.zeros((), device=DEV)).to(dt)
    dbranch, _ = api.dropout_residual_backward(do, br, gate, nv, p, rng, site=3)
    assert torch.equal(dbranch, want)
    # and where dgate is not wanted
    other = torch.empty_like(do)
    _abi.check(_abi.sol_dropout_residual_backward(
        do.data_ptr(), None, gate.data_ptr(), other.data_ptr(), None, rng.data_ptr(), 3, p, B, L,
        nv, D, None, 0, _abi.SOL_BF16 if dt == BF else _abi.SOL_F32,
        torch.cuda.current_stream().cuda_stream))
    assert torch.equal(other, want)


def test_dropout_mask_is_a_function_of_seed_offset_and_element():
    x = torch.ones((1, 513, 520), device=DEV)
    a = api.dropout(x, 0.5, _rng(), site=1)
    # offset + site, modulo 2^64, in both words
    assert torch.equal(a, api.dropout(x, 0.5, _rng(offset=RNG[1] + 1)))
    assert torch.equal(api.dropout(x, 0.5, _rng(offset=2 ** 64 - 1), site=3),
                       api.dropout(x, 0.5, _rng(offset=2)))
    assert not torch.equal(a, api.dropout(x, 0.5, _rng(), site=2))
    assert not torch.equal(a, api.dropout(x, 0.5, _rng(seed=RNG[0] ^ (1 << 63)), site=1))
    # the same elements under another shape, type and split
    assert torch.equal(a.flatten(), api.dropout(x.view(-1, 8), 0.5, _rng(), site=1).flatten())
    b = api.dropout(x.to(BF), 0.5, _rng(), site=1)
    assert torch.equal(b.float(), a)
    # the rate: 266,760 independent halves, 6 standard deviations
    kept = int((a != 0).sum())
    assert abs(kept - a.numel() / 2) < 6 * (a.numel() / 4) ** 0.5


def test_dropout_counters_past_32_bits():
    # elements past 2^34 have counters past 2^32: 2^21 rows of 8,200 are 17.2e9 elements
    rows, D = 2 ** 21, 8200
    x = torch.ones((rows, D), dtype=BF, device=DEV)
    out = api.dropout(x, 0.5, _rng(), site=0, out=x)
    for r in (0, 1, rows // 2 + 1, rows - 2, rows - 1):
        keep = ref.keep_mask(D, RNG[0], RNG[1], 0.5, DEV, first=r * D)
        assert torch.equal(out[r] != 0, keep), r


def test_dropout_of_nothing_everything_and_bad_values():
    h, br = act(1, 9, 64, F32, 1), act(1, 9, 64, F32, 2)
    gate = vec((1, 2, 64), 0.0, 0.3, F32, 5)
    rng = _rng()
    bad = br.clone()
    bad[0, 3] = float("inf")
    bad[0, 4] = float("nan")
    assert torch.equal(api.dropout_residual(h, bad, gate, 5, 1.0, rng), h)
    d, dg = api.dropout_residual_backward(bad, bad, gate, 5, 1.0, rng)
    assert torch.all(d == 0) and torch.all(dg == 0)
    # p = 0 needs no generator and is the gated residual
    assert torch.equal(api.dropout_residual(h, br, gate, 5, 0.0, None),
                       api.gate_residual(h, br, gate, 5))
    # a dropped element adds 0 whatever it holds; a kept one carries it
    out = api.dropout_residual(h, bad, gate, 5, 0.5, rng)
    keep = ref.keep_mask(h.numel(), *RNG, 0.5, DEV).view_as(h)
    assert torch.equal(out[~keep], h[~keep])
    assert torch.isnan(out[0, 4][keep[0, 4]]).all() and torch.isinf(out[0, 3][keep[0, 3]]).all()
    _, dg = api.dropout_residual_backward(h, bad, gate, 5, 0.5, rng)
    cols = ~(keep[0, 3] | keep[0, 4])
    assert torch.isfinite(dg[0, 0][cols]).all()


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

ROPE = [
    # B, L, Hq, Hk, hd, sections, dtype, half, interleaved, per_axis, pos dtype
    (1, 1, 1, 1, 16, (3, 5), BF, False, False, False, torch.int32),
    (2, 1, 40, 8, 128, (16, 24, 24), BF, True, False, False, torch.int64),
    (1, 7, 3, 1, 128, (24, 20, 20), BF, False, True, False, torch.int32),
    (3, 37, 5, 5, 72, (18, 18), F32, False, False, True, torch.float32),
    (1, 301, 16, 2, 64, (8, 12, 12), BF, True, True, False, torch.int32),
    (2, 50, 2, 2, 96, (7, 20, 5), BF, True, False, True, torch.float32),    # 64 of 96 turned
    (1, 33, 4, 3, 80, (1, 0, 11), BF, False, True, True, torch.int64),      # an empty axis
    (1, 129, 1, 1, 256, (128,), BF, True, False, False, torch.int64),
    (1, 19, 33, 1, 128, (10, 20, 30, 4), F32, True, True, True, torch.int32),
    (1, 700, 2, 1, 8, (1, 1), F32, False, False, False, torch.int32),
    (2, 65, 3, 2, 40, (16, 4), F32, True, False, False, torch.float32),
    (1, 400, 40, 40, 128, (16, 24, 24), BF, False, False, False, torch.int32),
    (2, 2401, 3, 2, 64, (8, 12, 12), BF, True, False, False, torch.int32),   # a round and a tail
    (1, 9001, 1, 3, 32, (10, 6), F32, False, True, False, torch.int64),
]


def _rope_case(c, seed=0):
    B, L, Hq, Hk, hd, sec, dt, half, inter, per_axis, pdt = c
    g = torch.Generator(device=DEV).manual_seed(seed + L)
    pos = torch.randint(-50, 5000, (len(sec), B, L), generator=g, device=DEV)
    pos = (pos.double() / 3).float() if pdt == torch.float32 else pos.to(pdt)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV).to(dt)  # noqa: E731
    q, k, dq, dk = rnd(B, L, Hq, hd), rnd(B, L, Hk, hd), rnd(B, L, Hq, hd), rnd(B, L, Hk, hd)
    plan = api.RopeAxes(hd, sec, theta=10000.0, per_axis_freq=per_axis, interleaved=inter,
                        half_split=half)
    pairs = ref.pair_map(sec, 10000.0, per_axis, inter)
    gq, gk = (1 + 0.1 * rnd(hd)).to(dt), (1 + 0.1 * rnd(hd)).to(dt)
    return pos, q, k, dq, dk, plan, pairs, half, gq, gk


@pytest.mark.parametrize("c", ROPE, ids=ids)
@pytest.mark.parametrize("norm", [False, True])
def test_rope_axes(c, norm):
    pos, q, k, _, _, plan, pairs, half, gq, gk = _rope_case(c)
    if not norm:
        gq = gk = None
    qo, ko = api.rope_axes(q, k, pos, plan, gq, gk, qk_norm=norm, eps=EPS)
    for got, x, gm in ((qo, q, gq), (ko, k, gk)):
        # norm: a 256-channel sum of 8 per lane and 5 joins, then scale, turn
        ref.check(got, ref.rope(x, pos, pairs, half, norm, gm, EPS), 32, "out")
    only, none = api.rope_axes(q, None, pos, plan, gq, qk_norm=norm, eps=EPS)
    assert none is None and torch.equal(only, qo)
    qi, ki = q.clone(), k.clone()
    api.rope_axes(qi, ki, pos, plan, gq, gk, qk_norm=norm, eps=EPS, q_out=qi, k_out=ki)
    assert torch.equal(qi, qo) and torch.equal(ki, ko)


@pytest.mark.parametrize("c", ROPE, ids=ids)
@pytest.mark.parametrize("norm,weights", [(False, False), (True, True), (True, False)])
def test_rope_axes_backward(c, norm, weights):
    pos, q, k, dq, dk, plan, pairs, half, gq, gk = _rope_case(c)
    B, L, Hq, Hk = c[:4]
    if not weights:
        gq = gk = None
    r = api.rope_axes_backward(dq, dk, pos, plan, q, k, gq, gk, qk_norm=norm, eps=EPS)
    for got, dgot, d, x, gm, H in ((r.dq, r.dgamma_q, dq, q, gq, Hq),
                                   (r.dk, r.dgamma_k, dk, k, gk, Hk)):
        (w, wm), dw = ref.rope_backward(d, x, pos, pairs, half, norm, gm, EPS)
        ref.check(got, (w, wm), 48, "dx")
        if weights:
            ref.check(dgot, dw, ref.depth_rows(B * L * H), "dgamma")
        else:
            assert dgot is None
    for src in (0, 1) if norm else (0,):      # in place over either input
        t = [x.clone() for x in (dq, dk, q, k)]
        again = api.rope_axes_backward(t[0], t[1], pos, plan, t[2], t[3], gq, gk, qk_norm=norm,
                                       eps=EPS, dq=t[2 * src], dk=t[2 * src + 1])
        for a, b in zip(r, again):
            assert (a is None and b is None) or torch.equal(a, b)


def test_rope_axes_strides_and_shared_positions():
    B, L, H, hd = 2, 45, 3, 64
    plan = api.RopeAxes(hd, (8, 12, 12), half_split=True)
    g = torch.Generator(device=DEV).manual_seed(3)
    qkv = torch.randn((B, L, 3 * H * hd), generator=g, device=DEV).to(BF)
    q = qkv[..., :H * hd].view(B, L, H, hd)
    k = qkv[..., H * hd:2 * H * hd].view(B, L, H, hd)
    pos = torch.randint(0, 999, (3, L), generator=g, device=DEV, dtype=torch.int32)
    want = api.rope_axes(q.contiguous(), k.contiguous(), pos[:, None].expand(3, B, L).contiguous(),
                         plan)
    for p in (pos, pos[:, None].expand(3, B, L)):
        got = api.rope_axes(q, k, p, plan)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # attention's [B, H, L, hd], and columns of one merged output
    bhld = [torch.empty((B, H, L, hd), dtype=BF, device=DEV).transpose(1, 2) for _ in range(2)]
    api.rope_axes(q, k, pos, plan, q_out=bhld[0], k_out=bhld[1])
    assert torch.equal(bhld[0], want[0]) and torch.equal(bhld[1], want[1])
    merged = torch.full((B, L, 3 * H * hd), 7.0, dtype=BF, device=DEV)
    mv = merged.view(B, L, 3, H, hd)
    r = api.rope_axes_backward(want[0], want[1], pos, plan, dq=mv[:, :, 0], dk=mv[:, :, 1])
    ref_r = api.rope_axes_backward(want[0], want[1], pos, plan)
    assert torch.equal(r.dq, ref_r.dq) and torch.equal(r.dk, ref_r.dk)
    assert torch.all(mv[:, :, 2] == 7.0)
    # in place inside the projection; v untouched
    v = qkv[..., 2 * H * hd:].clone()
    api.rope_axes(q, k, pos, plan, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[..., 2 * H * hd:], v)


@pytest.mark.parametrize("shape,perm,sl", [
    # q and k as slices of one tensor, and where b, r, h, c of its axes are
    ((2, 7, 45, 64), (0, 2, 1, 3), "heads"),          # [B, Hq + Hk, L, hd]
    ((2, 3, 5, 45, 64), (0, 2, 1, 3), "axis"),        # [B, 3, H, L, hd]
    ((2, 45, 5, 3, 64), (0, 1, 2, 3), "last"),        # [B, L, H, 3, hd]
])
@pytest.mark.parametrize("norm", [False, True])
def test_rope_axes_in_place_on_slices_of_one_tensor(shape, perm, sl, norm):
    g = torch.Generator(device=DEV).manual_seed(11)
    buf = torch.randn(shape, generator=g, device=DEV).to(BF)
    cut = {"heads": lambda t: (t[:, :5], t[:, 5:]), "axis": lambda t: (t[:, 0], t[:, 1]),
           "last": lambda t: (t[..., 0, :], t[..., 1, :])}[sl]
    heads = lambda t: [v.permute(perm) for v in cut(t)]  # noqa: E731
    pos = torch.randint(0, 999, (3, 45), generator=g, device=DEV, dtype=torch.int32)
    plan = api.RopeAxes(64, (8, 12, 12), half_split=True)
    gam = [vec((64,), 1, 0.1, BF, i) if norm else None for i in (5, 6)]
    q, k = heads(buf)
    want = api.rope_axes(q.contiguous(), k.contiguous(), pos, plan, *gam, qk_norm=norm)
    # two outputs in one tensor, then in place
    out = torch.full(shape, 7.0, dtype=BF, device=DEV)
    oq, ok = heads(out)
    api.rope_axes(q, k, pos, plan, *gam, qk_norm=norm, q_out=oq, k_out=ok)
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1])
    if sl != "heads":
        v = out[:, 2] if sl == "axis" else out[..., 2, :]
        assert torch.all(v == 7.0)
    api.rope_axes(q, k, pos, plan, *gam, qk_norm=norm, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    # the gradient, over the outputs' gradients
    x = heads(torch.randn(shape, generator=g, device=DEV).to(BF)) if norm else (None, None)
    ref_r = api.rope_axes_backward(q.contiguous(), k.contiguous(), pos, plan, *x, *gam,
                                   qk_norm=norm)
    r = api.rope_axes_backward(q, k, pos, plan, *x, *gam, qk_norm=norm, dq=q, dk=k)
    for a, b in zip(r, ref_r):
        assert (a is None and b is None) or torch.equal(a, b)


def test_rope_axes_matches_the_grid_entry_point():
    # the implicit T x H x W grid written out as position ids
    w = WORKLOADS["tiny"]
    r = torch.arange(w.L, device=DEV)
    grid = r < w.n_video
    HW = w.H * w.W
    pos = torch.stack([torch.where(grid, r // HW, r - w.n_video),
                       torch.where(grid, (r // w.W) % w.H, 0), torch.where(grid, r % w.W, 0)])
    qkv = act(w.B, w.L, 3 * w.D, F32, 4)
    gq, gk = vec((w.head_dim,), 1, 0.1, F32, 5), vec((w.head_dim,), 1, 0.1, F32, 6)
    wq, wk = api.qknorm_rope3d(qkv, w.T, w.H, w.W, w.n_audio, w.n_heads, w.head_dim, w.sections,
                               gq, gk, w.eps, w.theta)
    plan = api.RopeAxes(w.head_dim, w.sections, theta=w.theta)
    v = qkv.view(w.B, w.L, 3, w.n_heads, w.head_dim)
    q, k = api.rope_axes(v[:, :, 0], v[:, :, 1], pos, plan, gq, gk, qk_norm=True, eps=w.eps)
    for a, b in ((q, wq), (k, wk)):
        # each within 16 roundings of the exact rotation of pairs below 8 in sum
        assert (a.flatten() - b.flatten()).abs().max() <= 2 * 16 * 2 ** -24 * 8


def test_rope_axes_far_positions():
    # angles of 2^31 - 1 and 2^31 / 3: exact products reduced in fp64
    pos = torch.tensor([[[2 ** 31 - 1, 2 ** 31 // 3, -(2 ** 31), 12345678]]], device=DEV)
    q = torch.randn((1, 4, 2, 64), device=DEV)
    for half in (False, True):
        plan = api.RopeAxes(64, (32,), half_split=half)
        got, _ = api.rope_axes(q, None, pos, plan)
        want = ref.rope(q, pos, ref.pair_map((32,), 10000.0, False, False), half, False, None, 0)
        # angle: half a step of 2^31 rad in the product and in the frequency, on
        # either side, 2^-23 each; pairs are below 8 in sum
        assert (got.double() - want[0]).abs().max() <= 8 * 4 * 2 ** -23 + 2 ** -20
    for dt in (torch.int32, torch.float32):
        small = torch.tensor([[[0, 1, -7, 2 ** 24]]], device=DEV)
        plan = api.RopeAxes(64, (32,))
        assert torch.equal(api.rope_axes(q, None, small.to(dt), plan)[0],
                           api.rope_axes(q, None, small, plan)[0])


# heads turned in part, the channels past rot_dim holding what arithmetic would spread:
# rot_dim inside a lane's vector, at its end, one pair only, and several rounds of rows
PARTIAL = [
    # B, L, Hq, Hk, hd, sections, dtype, half, interleaved, per_axis, pos dtype
    (1, 7, 3, 2, 16, (3,), BF, False, False, False, torch.int32),
    (1, 33, 4, 3, 80, (1, 0, 11), BF, False, True, True, torch.int64),
    (2, 19, 5, 1, 128, (10, 7), BF, False, True, False, torch.float32),
    (2, 50, 2, 2, 96, (7, 20, 5), BF, True, False, True, torch.float32),
    (1, 2401, 3, 2, 256, (32,), BF, True, False, False, torch.int32),
    (1, 129, 2, 1, 128, (5,), F32, False, False, False, torch.int64),
    (3, 700, 2, 1, 8, (1,), F32, False, False, False, torch.int32),
    (2, 65, 3, 2, 40, (8, 4), F32, True, False, False, torch.float32),
]


def _spoil(x, rot, values):
    """x with `values` in turn in one channel past rot_dim of every other head vector (each
    channel's neighbours stay finite), everything else as it was."""
    x = x.clone()
    B, L, H, hd = x.shape
    i = torch.arange(B * L * H, device=DEV)
    col = rot + i // 2 % (hd - rot)
    v = torch.tensor(values, device=DEV, dtype=x.dtype)[i % len(values)]
    flat = x.view(-1, hd)
    flat[i[::2], col[::2]] = v[::2]
    return x


def _bits(t):
    return t.view(torch.int16 if t.dtype == BF else torch.int32)


def _check_with_bad(got, want, depth, what):
    """ref.check where the exact value is finite; the same Inf or NaN where not."""
    value, mag = want
    bad = ~torch.isfinite(value)
    assert torch.equal(torch.isnan(got), torch.isnan(value)), f"{what}: NaN elsewhere"
    inf = torch.isinf(value)
    assert torch.equal(got[inf].double(), value[inf]), f"{what}: Inf elsewhere"
    z = lambda t: torch.where(bad, torch.zeros((), dtype=t.dtype, device=DEV), t)  # noqa: E731
    ref.check(z(got), (z(value), z(mag)), depth, what)


@pytest.mark.parametrize("c", PARTIAL, ids=ids)
def test_rope_axes_leaves_unrotated_channels_as_they_are(c):
    pos, q, k, dq, dk, plan, pairs, half, _, _ = _rope_case(c)
    rot = 2 * len(pairs)
    for a, b, call in ((q, k, lambda a, b: api.rope_axes(a, b, pos, plan)),
                       (dq, dk, lambda a, b: api.rope_axes_backward(a, b, pos, plan)[:2])):
        clean = call(a, b)
        sa, sb = (_spoil(t, rot, (INF, NAN, -INF, -0.0)) for t in (a, b))
        for got, want, src in zip(call(sa, sb), clean, (sa, sb)):
            assert torch.equal(_bits(got[..., rot:]), _bits(src[..., rot:]))
            assert torch.equal(_bits(got[..., :rot]), _bits(want[..., :rot]))


@pytest.mark.parametrize("c", PARTIAL, ids=ids)
def test_rope_axes_with_the_norm_and_bad_unrotated_channels(c):
    pos, q, k, dq, dk, plan, pairs, half, gq, gk = _rope_case(c)
    B, L, Hq, Hk = c[:4]
    rot = 2 * len(pairs)
    args = dict(qk_norm=True, eps=EPS)
    # the forward pass: an Inf makes its head's norm 0 and itself NaN
    for bad in (INF, NAN):
        sq, sk = _spoil(q, rot, (bad,)), _spoil(k, rot, (bad,))
        for got, x, gm in zip(api.rope_axes(sq, sk, pos, plan, gq, gk, **args), (sq, sk), (gq, gk)):
            _check_with_bad(got, ref.rope(x, pos, pairs, half, True, gm, EPS), 32, "out")
    # a bad weight of one unrotated channel stays there
    hq, hk = gq.clone(), gk.clone()
    hq[rot], hk[-1] = INF, NAN
    for got, x, gm in zip(api.rope_axes(q, k, pos, plan, hq, hk, **args), (q, k), (hq, hk)):
        _check_with_bad(got, ref.rope(x, pos, pairs, half, True, gm, EPS), 32, "out")
    # the gradient: bad incoming gradients of one channel reach that channel's dgamma
    # alone, and dx through the head's mean
    for bad in (INF, NAN):
        sq, sk = dq.clone(), dk.clone()
        sq[:, ::2, :, rot], sk[:, ::3, :, -1] = bad, bad
        r = api.rope_axes_backward(sq, sk, pos, plan, q, k, gq, gk, **args)
        for got, dgot, d, x, gm, H in ((r.dq, r.dgamma_q, sq, q, gq, Hq),
                                       (r.dk, r.dgamma_k, sk, k, gk, Hk)):
            dx, dg = ref.rope_backward(d, x, pos, pairs, half, True, gm, EPS)
            _check_with_bad(got, dx, 48, "dx")
            _check_with_bad(dgot, dg, ref.depth_rows(B * L * H), "dgamma")


# ---------------------------------------------------------------------------
# streams, graphs, a block
# ---------------------------------------------------------------------------

def test_calls_on_a_side_stream():
    t, _ = _norm_case((1, 900, 800, 1024, BF), False)
    args = (t["dy"], t["x"], t["mean"], t["rstd"], t["gamma"], t["beta"], t["scale"])
    want = api.layer_norm_backward(*args, n_video=800)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.layer_norm_backward(*args, n_video=800, stream=side)
    # what the call allocated belongs to the side stream: the current stream may
    # allocate and write freely meanwhile
    junk = [torch.full((1, 900, 1024), float("nan"), dtype=BF, device=DEV) for _ in range(4)]
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    del junk


def test_two_threads_on_two_streams():
    import threading
    t, _ = _norm_case((1, 3000, 2500, 1024, BF), False)
    br = act(1, 3000, 1024, BF, 8)
    gate = vec((1, 2, 1024), 0, 0.3, BF, 9)
    rng = _rng()

    def work():
        n = api.layer_norm_backward(t["dy"], t["x"], t["mean"], t["rstd"], t["gamma"], t["beta"],
                                    t["scale"], n_video=2500)
        return (*n, *api.dropout_residual_backward(n.dx, br, gate, 2500, 0.3, rng))

    want = work()
    torch.cuda.synchronize()
    got, errors = {}, []

    def run(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got[i] = [work() for _ in range(20)]
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors
    for runs in got.values():
        for res in runs:
            for a, b in zip(want, res):
                assert torch.equal(a, b)


def test_captured_graphs_draw_new_masks_and_share_nothing():
    B, L, D, nv = 1, 130, 512, 100
    h, br, do = act(B, L, D, BF, 1), act(B, L, D, BF, 2), act(B, L, D, BF, 3)
    gate, sc = vec((B, 2, D), 0, 0.3, BF, 4), vec((B, 2, D), 0, 0.3, BF, 5)
    rng = _rng()
    plan, pos = api.RopeAxes(64, (10, 22)), torch.arange(2 * L, device=DEV).view(2, L)
    gq = vec((64,), 1, 0.1, BF, 6)

    def step(site):
        out = api.dropout_residual(h, br, gate, nv, 0.3, rng, site=site)
        y, mean, rstd = api.layer_norm(out, scale=sc, shift=sc, n_video=nv)
        heads = y.view(B, L, 8, 64)
        q, _ = api.rope_axes(heads, None, pos, plan, gq, qk_norm=True)
        r = api.rope_axes_backward(q, None, pos, plan, heads, None, gq, qk_norm=True)
        g = api.layer_norm_backward(r.dq.view(B, L, D), out, mean, rstd, scale=sc, n_video=nv,
                                    dres=do)
        return (out, y, q, *api.dropout_residual_backward(g.dx, br, gate, nv, 0.3, rng, site=site),
                g.dscale, g.dshift, r.dq, r.dgamma_q)

    step(0)
    torch.cuda.synchronize()
    graphs = []
    for site in (0, 1):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = step(site)
        graphs.append((graph, res))
    for offset in (5, 9):
        rng[1] = offset
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for site, (_, res) in enumerate(graphs):
            for a, b in zip(res, step(site)):
                assert torch.equal(a, b)


def test_a_block_forward_and_backward():
    """h1 = h + gate * dropout(rope(norm(h) W) ... ): the operators chained as
    a block uses them, against autograd of the same formulas in 64 bits."""
    B, L, nv, H, hd = 2, 61, 50, 2, 64
    D, p, eps = H * hd, 0.2, 1e-5
    g = torch.Generator(device=DEV).manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    h, sc, sh, gate = rnd(B, L, D), 0.3 * rnd(B, 2, D), 0.3 * rnd(B, 2, D), 0.3 * rnd(B, 2, D)
    W = rnd(D, 2 * D) / D ** 0.5
    gam, bet, gq, gk = 1 + 0.1 * rnd(D), 0.1 * rnd(D), 1 + 0.1 * rnd(hd), 1 + 0.1 * rnd(hd)
    sc2, sh2 = 0.3 * rnd(B, 2, D), 0.3 * rnd(B, 2, D)
    pos = torch.randint(0, 90, (3, B, L), generator=g, device=DEV)
    plan = api.RopeAxes(hd, (8, 12, 12))
    rng = _rng()
    dy = rnd(B, L, D)

    # forward
    y, mean, rstd = api.layer_norm(h, gam, bet, sc, sh, n_video=nv, eps=eps)
    qk = (y.view(-1, D) @ W).view(B, L, 2, H, hd)
    q, k = api.rope_axes(qk[:, :, 0], qk[:, :, 1], pos, plan, gq, gk, qk_norm=True, eps=eps)
    br = (q * k).reshape(B, L, D)
    h1 = api.dropout_residual(h, br, gate, nv, p, rng, site=4)
    z = api.rms_adaln(h1, sc2, sh2, nv, eps=eps)
    # backward of sum(z * dy)
    dh1, dsc2, dsh2, _ = api.rms_adaln_backward(dy, h1, sc2, nv, eps=eps)
    dbr, dgate = api.dropout_residual_backward(dh1, br, gate, nv, p, rng, site=4)
    d4 = dbr.view(B, L, H, hd)
    dqk = torch.empty_like(qk)
    r = api.rope_axes_backward(d4 * k, d4 * q, pos, plan, qk[:, :, 0], qk[:, :, 1], gq, gk,
                               qk_norm=True, eps=eps, dq=dqk[:, :, 0], dk=dqk[:, :, 1])
    dyn = (dqk.view(-1, 2 * D) @ W.T).view(B, L, D)
    n = api.layer_norm_backward(dyn, h, mean, rstd, gam, bet, sc, n_video=nv, dres=dh1)
    got = dict(h=n.dx, gam=n.dgamma, bet=n.dbeta, sc=n.dscale, sh=n.dshift, gate=dgate,
               gq=r.dgamma_q, gk=r.dgamma_k, sc2=dsc2, sh2=dsh2)

    # the same in fp64 with autograd
    v = {n_: t.double().requires_grad_() for n_, t in dict(
        h=h, gam=gam, bet=bet, sc=sc, sh=sh, gate=gate, gq=gq, gk=gk, sc2=sc2, sh2=sh2).items()}
    key = ref.key_of_rows(B, L, nv, DEV)
    rows = lambda t: t.reshape(2 * B, D)[key]  # noqa: E731
    hc = v["h"] - v["h"].mean(-1, keepdim=True)
    yn = hc / torch.sqrt((hc * hc).mean(-1, keepdim=True) + eps) * v["gam"] + v["bet"]
    yn = yn * (1 + rows(v["sc"])) + rows(v["sh"])
    qk64 = (yn.view(-1, D) @ W.double()).view(B, L, 2, H, hd)
    pairs = ref.pair_map((8, 12, 12), 10000.0, False, False)
    phi = torch.stack([pos[a].double() * f for a, f in pairs], -1)
    ph = torch.polar(torch.ones_like(phi), phi)[:, :, None]
    turned = []
    for i, gm in enumerate(("gq", "gk")):
        x = qk64[:, :, i]
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * v[gm]
        c = torch.view_as_complex(x.reshape(B, L, H, hd // 2, 2).contiguous()) * ph
        turned.append(torch.view_as_real(c).reshape(B, L, H, hd))
    br64 = (turned[0] * turned[1]).reshape(B, L, D)
    keep = ref.keep_mask(br64.numel(), RNG[0], RNG[1] + 4, ref.p32(p), DEV).view_as(br64)
    h64 = v["h"] + rows(v["gate"]) * br64 * keep / (1 - ref.p32(p))
    z64 = h64 / torch.sqrt((h64 * h64).mean(-1, keepdim=True) + eps)
    z64 = z64 * (1 + rows(v["sc2"])) + rows(v["sh2"])
    (z64 * dy.double()).sum().backward()
    # fp32 through two products over 128 and 256 terms and six operators: 2^-24
    # times about 1,000 operations, relative to the largest element
    tol = 1000 * ref.U32
    assert (z.double() - z64).abs().max() <= tol * z64.abs().max()
    for name, t in got.items():
        want = v[name].grad
        assert (t.double() - want).abs().max() <= tol * want.abs().max(), name


# the launch the largest workload takes, on sampled rows
def test_clip_sized_gradients_on_sampled_rows():
    w = WORKLOADS["clip5s"]
    B, L, nv, D = w.B, w.L, w.n_video, w.D
    x, dy = act(B, L, D, BF, 1), act(B, L, D, BF, 2, outliers=False)
    sc, sh = vec((B, 2, D), 0, 0.5, BF, 3), vec((B, 2, D), 0, 0.5, BF, 4)
    y, mean, rstd = api.layer_norm(x, scale=sc, shift=sh, n_video=nv, eps=EPS)
    got = api.layer_norm_backward(dy, x, mean, rstd, scale=sc, n_video=nv)
    pick = torch.tensor(sorted({0, 1, 427, 428, nv - 1, nv, nv + 1, L - 2, L - 1}
                               | set(range(11, L, 2999))), device=DEV)
    nvp = int((pick < nv).sum())
    wy, _, _ = ref.layer_norm(x[:, pick], None, None, sc, sh, nvp, EPS)
    ref.check(y[:, pick], wy, ref.depth_row(D), "y")
    want = ref.norm_backward(dy[:, pick], x[:, pick], mean[:, pick], rstd[:, pick], None, None, sc,
                             None, nvp, EPS, False)
    ref.check(got.dx[:, pick], want["dx"], ref.depth_row(D), "dx")
    # the sums, over all rows, in blocks: a thread adds 428 rows at most, the rest is fp64
    for m, (r0, r1) in enumerate(((0, nv), (nv, L))):
        s = torch.zeros(2, 2, D, dtype=torch.float64, device=DEV)
        for i in range(r0, r1, 4096):
            j = min(i + 4096, r1)
            xh = (x[0, i:j].double() - mean[0, i:j, None].double()) * rstd[0, i:j, None].double()
            xa = (x[0, i:j].double().abs() + mean[0, i:j, None].abs()) * rstd[0, i:j, None]
            d = dy[0, i:j].double()
            s[0] += torch.stack([(d * xh).sum(0), (d.abs() * xa).sum(0)])
            s[1] += torch.stack([d.sum(0), d.abs().sum(0)])
        ref.check(got.dscale[0, m], (s[0, 0], s[0, 1]), ref.depth_rows(428), "dscale")
        ref.check(got.dshift[0, m], (s[1, 0], s[1, 1]), ref.depth_rows(428), "dshift")


def test_more_elements_than_32_bits_count():
    # 2^20 + 3 rows of 57 heads of 72: 4.3e9 elements, 8.6 GB each tensor
    L, H, hd = 2 ** 20 + 3, 57, 72
    nv, D = L - 2, H * hd
    g = torch.Generator(device=DEV).manual_seed(3)
    x, dy = (torch.empty((1, L, D), dtype=BF, device=DEV).normal_(generator=g) for _ in "xy")
    sc, sh = vec((1, 2, D), 0, 0.5, BF, 3), vec((1, 2, D), 0, 0.5, BF, 4)
    pick = torch.tensor([0, 1, L // 2, L - 130, nv - 1, nv, L - 1], device=DEV)
    nvp = 5
    px, pdy = x[:, pick], dy[:, pick]
    y, mean, rstd = api.layer_norm(x, scale=sc, shift=sh, n_video=nv, eps=EPS)
    ref.check(y[:, pick], ref.layer_norm(px, None, None, sc, sh, nvp, EPS)[0], ref.depth_row(D),
              "y")
    got = api.layer_norm_backward(dy, x, mean, rstd, scale=sc, n_video=nv, dx=y)
    args = (sc, None, nvp, EPS)
    want = ref.norm_backward(pdy, px, mean[:, pick], rstd[:, pick], None, None, *args, False)["dx"]
    ref.check(got.dx[:, pick], want, ref.depth_row(D), "dx")
    api.rms_adaln_backward(dy, x, sc, nv, eps=EPS, dx=y)
    want = ref.norm_backward(pdy, px, None, None, None, None, *args, True)["dx"]
    ref.check(y[:, pick], want, ref.depth_row(D), "dx of the RMS norm")

    rng, p = _rng(), 0.25
    keep = torch.stack([ref.keep_mask(D, *RNG, p, DEV, first=int(r) * D) for r in pick])[None]
    d = torch.where(keep, px.double(), 0.0) / (1 - ref.p32(p)) * ref.spread(sc, nvp, 7)
    api.dropout_residual(dy, x, sc, nv, p, rng, out=y)
    ref.check(y[:, pick], (d + pdy.double(), d.abs() + pdy.double().abs()), 4, "out")
    api.dropout_residual_backward(x, dy, sc, nv, p, rng, dbranch=y)
    ref.check(y[:, pick], (d, d.abs()), 4, "dbranch")

    pos = (torch.arange(L, device=DEV, dtype=torch.int32) % 4099)[None]
    plan, pairs = api.RopeAxes(hd, (36,)), ref.pair_map((36,), 10000.0, False, False)
    ppos, hx, hdy = pos[:, None, pick], x.view(1, L, H, hd), dy.view(1, L, H, hd)
    api.rope_axes(hx, None, pos, plan, qk_norm=True, eps=EPS, q_out=y.view(1, L, H, hd))
    want = ref.rope(hx[:, pick], ppos, pairs, False, True, None, EPS)
    ref.check(y.view(1, L, H, hd)[:, pick], want, 32, "rotated")
    api.rope_axes_backward(hdy, None, pos, plan, hx, qk_norm=True, eps=EPS,
                           dq=y.view(1, L, H, hd))
    want, _ = ref.rope_backward(hdy[:, pick], hx[:, pick], ppos, pairs, False, True, None, EPS)
    ref.check(y.view(1, L, H, hd)[:, pick], want, 48, "dq")
