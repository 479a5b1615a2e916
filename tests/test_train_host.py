"""Training operators without a GPU: the references' own correctness (published
generator vectors, derivatives from differences), the plan, and the calls that
the C ABI and the tensor wrappers refuse (fake, never-dereferenced addresses)."""
import ctypes
import pathlib
import random
import re

import pytest
import torch

from tests import train_reference as ref
from video_diffusion_transformer_rms_b200 import _abi, api
from video_diffusion_transformer_rms_b200.build import build

INV, MIS, UNS = _abi.SOL_ERR_INVALID_ARG, _abi.SOL_ERR_MISALIGNED, _abi.SOL_ERR_UNSUPPORTED
BF, F32 = _abi.SOL_BF16, _abi.SOL_F32


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


# ---------------------------------------------------------------------------
# references
# ---------------------------------------------------------------------------

def test_generator_matches_published_vectors():
    # Philox4x32-10 known answers published with the generator
    for ctr, key, out in (
            ([0] * 4, [0] * 2, [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
            ([0xffffffff] * 4, [0xffffffff] * 2,
             [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
            ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
             [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1])):
        assert ref.philox(ctr, key) == out


def test_mask_reference_places_the_words():
    seed, offset, p = 0xA4093822299F31D0, 0x0370734413198A2E, 0.3
    first, n = 2 ** 35 + 5, 23
    got = ref.keep_mask(n, seed, offset, p, "cpu", first=first)
    for i in range(n):
        e = first + i
        ctr = [e // 4 & 0xFFFFFFFF, e // 4 >> 32, offset & 0xFFFFFFFF, offset >> 32]
        w = ref.philox(ctr, [seed & 0xFFFFFFFF, seed >> 32])[e % 4]
        assert bool(got[i]) == (w >= round(p * 2 ** 32))


def test_readme_recipe_draws_a_mask_of_its_own_for_every_step_and_layer():
    # the counter holds offset + site: steps and sites must not add up to the same
    text = (pathlib.Path(__file__).parent.parent / "README.md").read_text()
    rng_of = re.search(r"^rng = (torch\.tensor\(.*\))  +#", text, re.M).group(1)
    sites = set(re.findall(r"rng, site=(.*)\)", text))
    assert len(sites) == 1            # the gradient's is the forward call's
    masks, n_layers = set(), 5
    for step in range(4):
        for layer in range(n_layers):
            env = dict(torch=torch, seed=7, step=step, layer=layer, n_layers=n_layers)
            seed, offset = eval(rng_of.replace('"cuda"', '"cpu"'), env).tolist()
            keep = ref.keep_mask(512, seed, offset + eval(min(sites), env), 0.5, "cpu")
            masks.add(bytes(keep.numpy()))
    assert len(masks) == 4 * n_layers


def _scalars(seed, B=2, L=3, D=8):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradients_against_differences(rms):
    rnd = _scalars(1)
    B, L, D, nv, eps = 2, 3, 8, 2, 1e-3
    v = dict(x=rnd(B, L, D), gamma=rnd(D), beta=rnd(D), scale=rnd(B, 2, D), shift=rnd(B, 2, D))
    dy = rnd(B, L, D)

    def loss(**u):
        t = {**v, **u}
        if rms:
            y = t["x"] / torch.sqrt((t["x"] ** 2).mean(-1, keepdim=True) + eps) * t["gamma"]
            y = y * (1 + ref.spread(t["scale"], nv, L)) + ref.spread(t["shift"], nv, L)
        else:
            y = ref.layer_norm(t["x"], t["gamma"], t["beta"], t["scale"], t["shift"], nv,
                               eps)[0][0]
        return (y * dy).sum()

    x = v["x"]
    mean = x.mean(-1)
    rstd = 1 / torch.sqrt(x.var(-1, correction=0) + eps)
    got = ref.norm_backward(dy, x, mean, rstd, v["gamma"], None if rms else v["beta"], v["scale"],
                            None, nv, eps, rms)
    for name, grad in (("x", "dx"), ("gamma", "dgamma"), ("beta", "dbeta"), ("scale", "dscale"),
                       ("shift", "dshift")):
        if rms and name == "beta":
            continue
        d = rnd(*v[name].shape)
        ref.assert_derivative(lambda t: loss(**{name: t}), v[name], d, (got[grad][0] * d).sum())


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rope_gradients_against_differences(half, norm):
    rnd = _scalars(2)
    B, L, H, hd, sec = 2, 3, 2, 12, (2, 3)
    x, gamma, dy = rnd(B, L, H, hd), rnd(hd), rnd(B, L, H, hd)
    pos = torch.arange(2 * B * L).view(2, B, L)
    pairs = ref.pair_map(sec, 100.0, False, True)

    def loss(x_, gamma_):
        return (ref.rope(x_, pos, pairs, half, norm, gamma_, 1e-3)[0] * dy).sum()

    (dx, _), dg = ref.rope_backward(dy, x, pos, pairs, half, norm, gamma, 1e-3)
    d = rnd(*x.shape)
    ref.assert_derivative(lambda t: loss(t, gamma), x, d, (dx * d).sum())
    if norm:
        e = rnd(hd)
        ref.assert_derivative(lambda t: loss(x, t), gamma, e, (dg[0] * e).sum())


# ---------------------------------------------------------------------------
# the rotary plan
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("sec,hd", [((16, 24, 24), 128), ((24, 20, 20), 128), ((5,), 16),
                                    ((1, 0, 11), 80), ((7, 20, 5), 96), ((1,) * 8, 16)])
@pytest.mark.parametrize("per_axis", [False, True])
@pytest.mark.parametrize("inter", [False, True])
def test_plan_pairs(sec, hd, per_axis, inter):
    plan = api.RopeAxes(hd, sec, theta=1e6, per_axis_freq=per_axis, interleaved=inter).desc
    want = ref.pair_map(sec, 1e6, per_axis, inter)
    assert plan.rot_dim == 2 * sum(sec) and plan.n_axes == len(sec)
    for i, (a, f) in enumerate(want):
        assert plan.axis[i] == a
        assert plan.freq[i] == pytest.approx(f, rel=1e-14)


@pytest.mark.parametrize("kw", [
    dict(hd=0), dict(hd=258, sec=(4,)), dict(rot=0, sec=(0,)), dict(rot=130), dict(rot=63),
    dict(sec=(16, 24, 25)), dict(sec=(-1, 33, 32)), dict(sec=(1,) * 9, rot=18), dict(theta=0.0),
    dict(theta=float("inf")), dict(theta=float("nan")), dict(per=2), dict(inter=-1),
    dict(half=3), dict(sec=None), dict(plan=None)])
def test_plan_refusals(kw):
    a = dict(hd=128, rot=128, sec=(16, 24, 24), theta=1e4, per=0, inter=0, half=0,
             plan=_abi.RopePlan())
    a.update(kw)
    n = len(a["sec"]) if a["sec"] is not None else 3
    st = _abi.sol_rope_plan_init(a["plan"], a["hd"], a["rot"], n, a["sec"], a["theta"], a["per"],
                                 a["inter"], a["half"])
    assert st == INV and _abi.last_error()


# ---------------------------------------------------------------------------
# refusals of the C ABI
# ---------------------------------------------------------------------------

A = 0x7F0000000000
G = 1 << 30


def ln(x=A, y=A + G, mean=A + 2 * G, rstd=A + 3 * G, g=None, b=None, sc=A + 4 * G,
       sh=A + 5 * G, B=2, L=4, nv=2, D=64, eps=1e-6, dt=BF):
    return _abi.sol_layer_norm(x, y, mean, rstd, g, b, sc, sh, B, L, nv, D, eps, dt, None)


def ln_bwd(dy=A, x=A + G, mean=A + 2 * G, rstd=A + 3 * G, g=A + 4 * G, b=A + 5 * G,
           sc=A + 6 * G, dres=None, dx=A + 7 * G, dg=A + 8 * G, db=A + 9 * G, dsc=A + 10 * G,
           dsh=A + 11 * G, B=2, L=4, nv=2, D=64, ws=A + 12 * G, wb=1 << 30, dt=BF):
    return _abi.sol_layer_norm_backward(dy, x, mean, rstd, g, b, sc, dres, dx, dg, db, dsc, dsh,
                                        B, L, nv, D, ws, wb, dt, None)


def rms_bwd(dy=A, x=A + G, sc=A + 6 * G, g=None, dres=None, dx=A + 7 * G, dsc=A + 10 * G,
            dsh=A + 11 * G, dg=None, B=2, L=4, nv=2, D=64, eps=1e-6, ws=A + 12 * G, wb=1 << 30,
            dt=BF):
    return _abi.sol_rms_adaln_backward(dy, x, sc, g, dres, dx, dsc, dsh, dg, B, L, nv, D, eps, ws,
                                       wb, dt, None)


def drop(h=A, br=A + G, gate=A + 2 * G, out=A + 3 * G, rng=A + 4 * G, site=0, p=0.5, B=2, L=4,
         nv=2, D=64, dt=BF):
    return _abi.sol_dropout_residual(h, br, gate, out, rng, site, p, B, L, nv, D, dt, None)


def drop_bwd(do=A, br=A + G, gate=A + 2 * G, db=A + 3 * G, dgate=A + 5 * G, rng=A + 4 * G,
             site=0, p=0.5, B=2, L=4, nv=2, D=64, ws=A + 6 * G, wb=1 << 30, dt=BF):
    return _abi.sol_dropout_residual_backward(do, br, gate, db, dgate, rng, site, p, B, L, nv, D,
                                              ws, wb, dt, None)


ROWS_REFUSED = [
    (dict(dt=7), INV), (dict(B=-1), INV), (dict(L=-1), INV), (dict(D=0), INV), (dict(nv=5), INV),
    (dict(nv=-1), INV), (dict(L=2 ** 31, nv=0), UNS), (dict(B=2 ** 20, L=2 ** 12, nv=0), UNS), (dict(B=2 ** 30, L=1, nv=0), UNS),
    (dict(D=16392), UNS), (dict(D=8196, dt=F32), UNS), (dict(D=60), MIS), (dict(D=62, dt=F32), MIS),
]


@pytest.mark.parametrize("kw,status", ROWS_REFUSED)
@pytest.mark.parametrize("call", [ln, ln_bwd, rms_bwd, drop, drop_bwd])
def test_sizes_refused(call, kw, status):
    assert call(**kw) == status
    assert _abi.last_error()


@pytest.mark.parametrize("call,kw,status", [
    (ln, dict(x=None), INV), (ln, dict(y=None), INV), (ln, dict(rstd=None), INV),
    (ln, dict(mean=None), INV), (ln, dict(sc=None), INV), (ln, dict(sh=None), INV),
    (ln, dict(eps=-1.0), INV), (ln, dict(eps=float("nan")), INV), (ln, dict(x=A + 8), MIS),
    (ln, dict(mean=A + 2 * G + 2), MIS), (ln, dict(g=A + 8), MIS), (ln, dict(y=A + 16), INV),
    (ln, dict(mean=A), INV), (ln, dict(rstd=A + 2 * G + 16), INV), (ln, dict(g=A + G), INV),
    (ln, dict(sc=A + G + 1008), INV),
    (ln_bwd, dict(dy=None), INV), (ln_bwd, dict(x=None), INV), (ln_bwd, dict(mean=None), INV),
    (ln_bwd, dict(dx=None), INV), (ln_bwd, dict(sc=None), INV),        # dscale without scale
    (ln_bwd, dict(ws=None), INV), (ln_bwd, dict(wb=6143), INV), (ln_bwd, dict(ws=A + 8), MIS),
    (ln_bwd, dict(dg=A + 8 * G + 4), MIS), (ln_bwd, dict(rstd=A + 3 * G + 2), MIS),
    (ln_bwd, dict(dx=A + 16), INV), (ln_bwd, dict(dx=A + 2 * G), INV),
    (ln_bwd, dict(db=A + 8 * G), INV), (ln_bwd, dict(dsh=A + 1008), INV),
    (ln_bwd, dict(ws=A + 7 * G), INV), (ln_bwd, dict(dres=A + 7 * G + 16), INV),
    (rms_bwd, dict(sc=None, dsc=None, dsh=None), INV), (rms_bwd, dict(eps=-1.0), INV),
    (rms_bwd, dict(wb=0), INV), (rms_bwd, dict(dx=A + 6 * G), INV),
    (drop, dict(br=None), INV), (drop, dict(out=None), INV), (drop, dict(rng=None), INV),
    (drop, dict(p=-0.1), INV), (drop, dict(p=1.5), INV), (drop, dict(p=float("nan")), INV),
    (drop, dict(rng=A + 4), MIS), (drop, dict(gate=A + 8), MIS), (drop, dict(out=A + 16), INV),
    (drop, dict(out=A + 2 * G), INV), (drop, dict(rng=A + 3 * G + 8), INV),
    (drop_bwd, dict(br=None), INV), (drop_bwd, dict(gate=None), INV), (drop_bwd, dict(db=None), INV),
    (drop_bwd, dict(ws=None), INV), (drop_bwd, dict(wb=16), INV), (drop_bwd, dict(db=A + G + 16), INV),
    (drop_bwd, dict(dgate=A), INV), (drop_bwd, dict(ws=A + 5 * G), INV),
])
def test_arguments_refused(call, kw, status):
    assert call(**kw) == status
    assert _abi.last_error()


def test_workspace_sizes():
    # 8 rows: 8 shares and 4 keys, two sums of 64 floats
    assert _abi.sol_norm_backward_workspace_bytes(2, 4, 64) == 12 * 2 * 64 * 4
    assert _abi.sol_dropout_backward_workspace_bytes(2, 4, 64) == 12 * 64 * 4
    assert _abi.sol_norm_backward_workspace_bytes(1, 10 ** 6, 64) == 594 * 2 * 64 * 4
    for bad in ((-1, 4, 64), (2, -4, 64), (2, 4, 0), (2 ** 20, 2 ** 20, 64), (2, 4, 2 ** 40)):
        assert _abi.sol_norm_backward_workspace_bytes(*bad) == 0
        assert _abi.sol_dropout_backward_workspace_bytes(*bad) == 0
    assert _abi.sol_rope_backward_workspace_bytes(1) == 0
    assert _abi.sol_rope_backward_workspace_bytes(258) == 0
    assert _abi.sol_rope_backward_workspace_bytes(128) > 0


def H(p, n=2, sb=4 * 256, sr=256, sh=128):
    return _abi.Heads(p, n, sb, sr, sh)


def P(p=A + 20 * G, type=0, reserved=0, sa=8, sb=4):
    return _abi.Positions(p, type, reserved, sa, sb)


def plan(hd=128, sec=(16, 24, 24), **kw):
    return api.RopeAxes(hd, sec, **kw).desc


_DEFAULT = object()


def rope(pl=_DEFAULT, pos=_DEFAULT, q=_DEFAULT, k=_DEFAULT, qo=_DEFAULT, ko=_DEFAULT, gq=None,
         gk=None, norm=0, B=2, L=4, eps=1e-6, dt=BF):
    d = lambda v, x: x if v is _DEFAULT else v  # noqa: E731
    return _abi.sol_rope_axes(d(pl, plan()), d(pos, P()), d(q, H(A)), d(k, H(A + G)),
                              d(qo, H(A + 2 * G)), d(ko, H(A + 3 * G)), gq, gk, norm, B, L, eps,
                              dt, None)


def rope_bwd(pl=_DEFAULT, pos=_DEFAULT, dqo=_DEFAULT, dko=_DEFAULT, q=_DEFAULT, k=_DEFAULT,
             dq=_DEFAULT, dk=_DEFAULT, gq=A + 8 * G, gk=A + 9 * G, dgq=A + 10 * G,
             dgk=A + 11 * G, norm=1, B=2, L=4, eps=1e-6, ws=A + 12 * G, wb=1 << 30, dt=BF):
    d = lambda v, x: x if v is _DEFAULT else v  # noqa: E731
    return _abi.sol_rope_axes_backward(
        d(pl, plan()), d(pos, P()), d(dqo, H(A)), d(dko, H(A + G)), d(q, H(A + 2 * G)),
        d(k, H(A + 3 * G)), d(dq, H(A + 4 * G)), d(dk, H(A + 5 * G)), gq, gk, dgq, dgk, norm, B,
        L, eps, ws, wb, dt, None)


def _bad_plan(**kw):
    p = plan()
    for n, v in kw.items():
        setattr(p, n, v)
    return p


def _plan_with(i, axis=None, freq=None):
    p = plan()
    if axis is not None:
        p.axis[i] = axis
    if freq is not None:
        p.freq[i] = freq
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(pl=None), INV), (dict(pl=_abi.RopePlan()), INV), (dict(dt=5), INV),
    (dict(norm=2), INV), (dict(B=-1), INV), (dict(B=2 ** 20, L=2 ** 20), UNS),
    (dict(pos=None), INV), (dict(pos=P(type=3)), INV), (dict(pos=P(reserved=1)), INV),
    (dict(pos=P(sa=-1)), INV), (dict(pos=P(p=None)), INV), (dict(pos=P(p=A + 2)), MIS),
    (dict(pos=P(p=A + 4, type=1)), MIS), (dict(pos=P(p=A + 2 * G + 64)), INV),
    (dict(q=None), INV), (dict(qo=None), INV), (dict(k=None), INV), (dict(ko=None), INV),
    (dict(q=H(None)), INV), (dict(q=H(A, n=3)), INV), (dict(q=H(A, sr=-256)), INV),
    (dict(q=H(A, sb=2 ** 62)), INV), (dict(q=H(A + 8)), MIS), (dict(q=H(A, sr=260)), MIS),
    (dict(q=H(A, n=0), qo=H(A + 2 * G, n=0)), UNS),
    (dict(q=H(A, n=1025, sr=2 ** 18), qo=H(A + 2 * G, n=1025, sr=2 ** 18)), UNS),
    (dict(qo=H(A + 16)), INV), (dict(qo=H(A, sr=512)), INV), (dict(ko=H(A + 2 * G + 256)), INV),
    (dict(qo=H(A + G)), INV), (dict(ko=H(A)), INV), (dict(gq=A + 8 * G), INV),
    (dict(norm=1, eps=-1.0), INV), (dict(norm=1, gq=A + 8), MIS), (dict(norm=1, gq=A + 2 * G), INV),
    (dict(k=None, ko=None, norm=1, gk=A + 9 * G), INV),
    (dict(pl=_bad_plan(rot_dim=130)), INV), (dict(pl=_bad_plan(half_split=2)), INV),
    (dict(pl=_bad_plan(n_axes=0)), INV), (dict(pl=_plan_with(63, axis=3)), INV),
    (dict(pl=_plan_with(0, freq=float("nan"))), INV),
    (dict(pl=plan(132, (66,))), UNS), (dict(pl=plan(256, (128,)), dt=F32), UNS),
    (dict(pl=plan(128, (20,), half_split=True)), UNS),
])
def test_rope_refused(kw, status):
    assert rope(**kw) == status
    assert _abi.last_error()


# outputs whose own elements overlap, in place too; positions out of range
@pytest.mark.parametrize("kw", [
    dict(qo=H(A + 2 * G, sh=0)), dict(qo=H(A + 2 * G, sh=64)), dict(qo=H(A + 2 * G, sr=128)),
    dict(qo=H(A + 2 * G, sr=0)), dict(qo=H(A + 2 * G, sb=256)), dict(ko=H(A + 3 * G, sb=0)),
    dict(qo=H(A + 2 * G, sb=128, sr=128, sh=1024)), dict(q=H(A, sb=0), qo=H(A, sb=0)),
    dict(pos=P(sa=2 ** 62)), dict(pos=P(sb=2 ** 62)), dict(pos=P(sb=2 ** 40), B=2 ** 29, L=1),
])
def test_rope_refuses_overlapping_outputs_and_far_positions(kw):
    assert rope(**kw) == INV
    assert _abi.last_error()


def test_rope_empty_and_reordered_axes_are_not_refused():
    # no rows: nothing to overlap; and axes in another order of strides are in order
    assert rope(qo=H(A + 2 * G, sh=0), L=0) == 0
    assert rope(qo=H(A + 2 * G, sb=1024, sr=128, sh=512), ko=H(A + 3 * G, n=3)) == INV
    assert "heads" in _abi.last_error() and "overlap" not in _abi.last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dqo=None), INV), (dict(dq=None), INV), (dict(q=None), INV), (dict(k=None), INV),
    (dict(dk=None), INV), (dict(norm=0), INV),
    (dict(norm=0, gq=None, gk=None, dgq=None, dgk=None), INV),         # q without the norm
    (dict(norm=0, gq=None, gk=None, q=None, k=None), INV),             # dgamma without the norm
    (dict(ws=None), INV), (dict(wb=1024), INV), (dict(ws=A + 8), MIS), (dict(dgq=A + 4), MIS),
    (dict(dgq=A + 4 * G), INV), (dict(dgk=A + 10 * G), INV), (dict(ws=A + 10 * G), INV),
    (dict(dgq=A + 8 * G), INV), (dict(dq=H(A + G)), INV), (dict(dq=H(A + 3 * G)), INV),
    (dict(dk=None, dko=None, k=None), INV),                            # dgamma_k without k
    (dict(dk=None, dko=None, k=None, dgk=None), INV),                  # gamma_k without k
])
def test_rope_backward_refused(kw, status):
    assert rope_bwd(**kw) == status
    assert _abi.last_error()


# Arrays that lie in each other's gaps share no byte.  Nothing is launched: dgamma_q is
# given gamma_q's address, which is refused once every heads array has passed.

def _lay(shape, order, pick=None):
    """Strides (b, row, head) and offset of a [B, L, H, hd] view of a tensor whose axes
    lie in memory in `order` ('b', 'r', 'h', 'c', and 's' for slices, of which `pick`
    is taken)."""
    step, s, n = {}, 1, dict(shape)
    for ax in reversed(order):
        step[ax] = s
        s *= n[ax]
    return step["b"], step["r"], step["h"], (pick or 0) * step.get("s", 0)


def _in_gaps(q, k, B, L, hd, over=None):
    """Status and message of the gradient in place over dq_out = q's and dk_out = k's
    layout, (stride_b, stride_row, stride_head, offset, heads) each; `over`: dk_out is
    written over other heads than its own."""
    at = lambda v, base=A: H(base + 2 * v[3], v[4], *v[:3])  # noqa: E731
    st = rope_bwd(pl=plan(hd, (hd // 2,)), pos=P(sa=0, sb=0), dqo=at(q), dko=at(k),
                  q=at(q, A + 2 * G), k=at(k, A + 2 * G), dq=at(q), dk=at(over or k), B=B, L=L,
                  dgq=A + 8 * G)
    return st, _abi.last_error()


@pytest.mark.parametrize("B", [1, 2, 5])
@pytest.mark.parametrize("L", [1, 7, 300])
@pytest.mark.parametrize("Hq,Hk", [(3, 3), (4, 1), (1, 2), (1, 1)])
def test_rope_takes_slices_of_one_tensor(B, L, Hq, Hk):
    hd, n = 64, dict(b=B, r=L, h=Hq + Hk, c=64)
    layouts = []
    # q and k as heads of one buffer, [B, Hq + Hk, L, hd] and the other orders
    for order in ("bhrc", "brhc", "hbrc", "rbhc", "hrbc", "rhbc"):
        sb, sr, sh, _ = _lay(n, order)
        layouts.append(((sb, sr, sh, 0, Hq), (sb, sr, sh, Hq * sh, Hk)))
    if Hq == Hk:      # q, k, v as slices: [B, 3, H, L, hd], [B, L, H, 3, hd] and others
        n = dict(b=B, r=L, h=Hq, c=64, s=3)
        for order in ("bshrc", "brhsc", "sbrhc", "bhsrc", "brshc", "rbshc", "bhrsc"):
            for i, j in ((0, 1), (1, 0), (0, 2)):
                layouts.append(tuple((*_lay(n, order, p), Hq) for p in (i, j)))
    for q, k in layouts:
        st, msg = _in_gaps(q, k, B, L, hd)
        assert st == INV and "dgamma_q overlaps gamma_q" in msg, (q, k, msg)
        # one vector off, the outputs meet
        if (B, L, Hq + Hk) != (1, 1, 2):
            st, msg = _in_gaps(q, k, B, L, hd, over=(*q[:3], q[3] + 8, Hk))
            assert st == INV and "dgamma" not in msg, (q, k, msg)


def _touched(v, B, L, hd):
    """The 16-byte units of a heads array (bf16, offsets and strides in elements)."""
    sb, sr, sh, off, n = v
    return {(off + b * sb + r * sr + h * sh) // 8 + c for b in range(B) for r in range(L)
            for h in range(n) for c in range(hd // 8)}


def _nested(v, B, L, hd):
    """Whether each axis steps over all below it, as an output's must."""
    extent = hd
    for step, n in sorted(zip(v[:3], (B, L, v[4]))):
        if n > 1:
            if step < extent:
                return False
            extent += (n - 1) * step
    return True


def test_rope_overlap_of_random_layouts_is_exact():
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        B, L, hd = rng.randint(1, 3), rng.randint(1, 4), 8 * rng.randint(1, 2)
        two = []
        for _ in "qk":
            n = rng.randint(1, 3)
            # nested strides in any order with gaps, in units of 8 elements
            axes, step, s = [("b", B), ("r", L), ("h", n)], {}, hd // 8
            rng.shuffle(axes)
            for ax, count in axes:
                s += rng.choice((0, 0, 0, 1, 2, 5))
                step[ax] = 8 * s
                s *= count
            two.append((step["b"], step["r"], step["h"], 8 * rng.randint(0, 30), n))
        if rng.random() < 0.5:        # slices of one tensor have the same strides
            two[1] = (*two[0][:3], *two[1][3:])
        q, k = two
        units = [_touched(v, B, L, hd) for v in two]
        if not all(_nested(v, B, L, hd) for v in two):
            continue                  # k's heads under q's strides: refused as such
        st, msg = _in_gaps(q, k, B, L, hd)
        apart = not units[0] & units[1]
        assert st == INV and ("dgamma_q overlaps gamma_q" in msg) == apart, (two, B, L, hd, msg)
        seen[apart] += 1
    assert min(seen.values()) > 300


def test_rope_small_arrays_in_the_gaps_of_heads():
    # gamma_q, positions and dgamma_k between the heads of dq's rows
    wide = H(A + 4 * G, sr=1024, sb=4096)        # 256 of 1,024 elements a row
    gap = A + 4 * G + 600
    for kw in (dict(gq=gap + 8, dgq=gap + 8), dict(pos=P(gap + 8, sa=0, sb=0), dgq=A + 8 * G),
               dict(dgk=gap + 8, dgq=A + 8 * G)):
        assert rope_bwd(dq=wide, **kw) == INV
        assert "dgamma_q overlaps gamma_q" in _abi.last_error(), kw
    for kw in (dict(gq=A + 4 * G + 496), dict(pos=P(A + 4 * G + 508, sa=0, sb=0)),
               dict(dgk=A + 4 * G + 2048)):
        assert rope_bwd(dq=wide, **kw) == INV
        assert "output overlaps" in _abi.last_error(), kw


def test_rope_layouts_that_cannot_be_told_apart_in_time_are_refused():
    # steps that nest in nothing: the check gives up, it does not hang
    q = (2 ** 19 + 8, 2 ** 19, 2 ** 19 + 16, 0, 1000)
    k = (2 ** 19 + 24, 2 ** 19 + 32, 2 ** 19 + 40, 64, 1000)
    st, msg = _in_gaps(q, k, 1000, 1000, 64)
    assert st == INV and "overlap" in msg


# ---------------------------------------------------------------------------
# refusals of the tensor wrappers
# ---------------------------------------------------------------------------

Z = torch.zeros


def test_wrappers_check_shapes_and_types():
    x, v, m = Z(2, 4, 16), Z(16), Z(2, 2, 16)
    for call, match in (
            (lambda: api.layer_norm(x.transpose(0, 1)), "contiguous"),
            (lambda: api.layer_norm(x, Z(8)), "gamma"),
            (lambda: api.layer_norm(x, v, v, Z(2, 16), m), "scale"),
            (lambda: api.layer_norm(x, out=Z(2, 4, 8)), "out"),
            (lambda: api.layer_norm(x), "CUDA"),
            (lambda: api.layer_norm_backward(x, x, Z(2, 3), Z(2, 4)), "mean"),
            (lambda: api.layer_norm_backward(x, x, Z(2, 4), Z(2, 4), dres=Z(2, 4, 8)), "dres"),
            (lambda: api.rms_adaln_backward(x, x, Z(2, 1, 16), 2), "scale"),
            (lambda: api.rms_adaln_backward(Z(2, 3, 16), x, m, 2), "dy"),
            (lambda: api.dropout(x.transpose(0, 1), 0.5, None), "contiguous"),
            (lambda: api.dropout(x, 0.5, None), "rng"),
            (lambda: api.dropout(x, 0.5, Z(3, dtype=torch.int64)), "rng"),
            (lambda: api.dropout(x, 0.0, None), "CUDA"),
            (lambda: api.dropout_residual(Z(2, 4, 8), x, m, 2, 0.0, None), "h must"),
            (lambda: api.dropout_residual_backward(x, None, m, 2, 0.0, None), "branch"),
            (lambda: api.dropout_residual_backward(x, x, Z(1, 2, 16), 2, 0.0, None), "gate"),
    ):
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(TypeError, match="share one dtype"):
        api.layer_norm(x, v.double())
    with pytest.raises(TypeError, match="float32"):
        api.layer_norm_backward(x, x, Z(2, 4).half(), Z(2, 4))
    with pytest.raises(TypeError, match="int64"):
        api.dropout(x, 0.5, Z(2))


def test_rope_wrappers_check_shapes_and_types():
    pl = api.RopeAxes(16, (3, 5))
    q, pos = Z(2, 4, 3, 16), Z(2, 2, 4, dtype=torch.int32)
    for call, match in (
            (lambda: api.rope_axes(Z(2, 4, 48), None, pos, pl), "heads"),
            (lambda: api.rope_axes(Z(2, 4, 3, 32), None, pos, pl), "plan"),
            (lambda: api.rope_axes(q, None, pos, pl, gamma_q=Z(8)), "gamma_q"),
            (lambda: api.rope_axes(q, None, pos, pl, k_out=q), "k_out"),
            (lambda: api.rope_axes(q, q, pos, pl), "CUDA"),
            (lambda: api.rope_axes_backward(q, None, pos, pl, qk_norm=True), "qk_norm"),
            (lambda: api.rope_axes_backward(q, None, pos, pl, dk=q), "dk"),
            (lambda: api._heads(Z(2, 4, 16, 3).transpose(2, 3), 2, 4, 16, "q", q), "unit"),
            (lambda: api._heads(Z(1, 4, 3, 16).expand(2, 4, 3, 16), 2, 4, 16, "q_out", q, 3,
                                True), "expanded|CUDA"),
            (lambda: api._positions(Z(3, 2, 4, dtype=torch.int32), 2, 4, 2, q), "pos must"),
            (lambda: api._positions(Z(2, 4, 2, dtype=torch.int32).transpose(1, 2), 2, 4, 2, q),
             "pos must"),
    ):
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(TypeError, match="int32"):
        api._positions(Z(2, 2, 4, dtype=torch.float64), 2, 4, 2, q)
    with pytest.raises(_abi.SolError, match="sections"):
        api.RopeAxes(16, (9, -1))
    assert ctypes.sizeof(_abi.RopePlan) == 4 * 4 + 128 + 128 * 8


# ---------------------------------------------------------------------------
# the shares and slots of the row sums (the arithmetic of sol_train.h and
# segment_sums.cuh, followed here step by step)
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("B,L,nv", [(1, 1, 0), (1, 56, 48), (3, 37, 20), (5, 1, 1), (2, 300, 0),
                                    (4, 9, 9), (500, 3, 1), (1, 9001, 8000), (700, 2, 1)])
@pytest.mark.parametrize("ctas", [1, 7, 118, 296, 592])
def test_row_sum_slots(B, L, nv, ctas):
    rows, keys = B * L, 2 * B
    ctas = min(ctas, rows)
    share, longer = divmod(rows, ctas)
    begin = [c * share + min(c, longer) for c in range(ctas + 1)]
    assert begin[0] == 0 and begin[-1] == rows and all(a < b for a, b in zip(begin, begin[1:]))

    def share_of(r):
        head = longer * (share + 1)
        return r // (share + 1) if r < head else longer + (r - head) // share

    written = {}
    for c in range(ctas):
        assert share_of(begin[c]) == c == share_of(begin[c + 1] - 1)
        for k in {2 * (r // L) + (r % L >= nv) for r in range(begin[c], begin[c + 1])}:
            assert c + k < min(rows, 592) + keys and c + k not in written
            written[c + k] = (c, k)
    for k in range(keys):      # a key's sum is read from the slots that were written for it
        r0, r1 = (k >> 1) * L + (nv if k & 1 else 0), (k >> 1) * L + (L if k & 1 else nv)
        read = set(range(share_of(r0), share_of(r1 - 1) + 1)) if r0 < r1 else set()
        assert read == {c for c, kk in written.values() if kk == k}
