"""The training operators of the per-token path, as cases to be measured.

Three families, each with its backward pass:

* layer norm (plain affine, or with the adaptive scale/shift of a joint
  video+audio block), its gradient, and the gradient of the RMS-AdaLN;
* rotary positions with several axes at explicit position ids, with or
  without the per-head RMS norm of q and k in front, and their gradient;
* dropout with a counter-based generator in front of the gated residual, and
  its gradient; the mask is generated again in the backward pass.

`own = False` computes each operator from elementary torch operations in fp32
(fp64 for angles and for the long sums of the vector gradients), rounded once.
`own = True` calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}
_POS = {"i32": torch.int32, "i64": torch.int64, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # -- layer norm ------------------------------------------------------
        # the smallest block of the configurations: 48 video + 8 audio tokens, fp32
        dict(name="ln_tiny_f32", op="ln", B=1, L=56, n_video=48, D=256, dtype="f32", mod=False),
        # the 5 s 1344x768 clip: 31x48x84 latent tokens + 1,560 audio tokens
        dict(name="ln_adaln_clip5s", op="ln", B=1, L=126552, n_video=124992, D=5120,
             dtype="bf16", mod=True),
        # the same small block in a training step, where launch latency counts
        dict(name="ln_grad_tiny_f32", op="ln_grad", B=1, L=56, n_video=48, D=256, dtype="f32",
             mod=False, dres=False),
        # a preview clip (8x24x42 + 200 tokens): gradient of the RMS-AdaLN, residual
        # gradient added
        dict(name="rms_grad_medium", op="rms_grad", B=1, L=8264, n_video=8064, D=5120,
             dtype="bf16", mod=True, dres=True),
        # gradient of the adaptive layer norm over the whole clip
        dict(name="ln_grad_clip5s", op="ln_grad", B=1, L=126552, n_video=124992, D=5120,
             dtype="bf16", mod=True, dres=False),
        # -- rotary positions ------------------------------------------------
        # one token for each of two streams, grouped heads, half-split pairs
        dict(name="rope_token", op="rope", B=2, L=1, Hq=40, Hk=8, hd=128, rot=128,
             sec="16+24+24", dtype="bf16", pos="i64", theta=10000.0, per_axis=False,
             interleaved=False, half=True, norm=False, merged=False),
        # merged QKV of the clip, 40 heads, norm and rotation in one pass
        dict(name="rope_norm_clip5s", op="rope", B=1, L=126552, Hq=40, Hk=40, hd=128, rot=128,
             sec="16+24+24", dtype="bf16", pos="i32", theta=10000.0, per_axis=False,
             interleaved=False, half=False, norm=True, merged=True),
        # packed images of several sizes: two axes, fractional (rescaled) positions,
        # a ladder per axis, odd row count, a head of 72; gradient
        dict(name="rope_grad_images_f32", op="rope_grad", B=1, L=4099, Hq=16, Hk=16, hd=72,
             rot=72, sec="18+18", dtype="f32", pos="f32", theta=10000.0, per_axis=True,
             interleaved=False, half=False, norm=False, merged=False),
        # gradient through rotation and norm over the clip, axes dealt in turn
        dict(name="rope_norm_grad_clip5s", op="rope_grad", B=1, L=126552, Hq=40, Hk=40, hd=128,
             rot=128, sec="24+20+20", dtype="bf16", pos="i32", theta=1000000.0,
             per_axis=False, interleaved=True, half=True, norm=True, merged=True),
        # -- dropout ---------------------------------------------------------
        dict(name="dropout_tiny_f32", op="drop", B=1, L=56, n_video=48, D=256, dtype="f32",
             p=0.1, resid=True),
        dict(name="dropout_clip5s", op="drop", B=1, L=126552, n_video=124992, D=5120,
             dtype="bf16", p=0.1, resid=True),
        # two samples of the preview clip, odd audio length
        dict(name="dropout_grad_medium", op="drop_grad", B=2, L=8265, n_video=8064, D=5120,
             dtype="bf16", p=0.25, resid=True),
    ]


_MAX_ELEMENTS = 126552 * 5120          # of one activation of the largest listed cases


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln", "ln", "ln_grad", "ln_grad", "rms_grad", "rope", "rope", "rope_grad",
                     "rope_grad", "drop", "drop", "drop_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("rope", "rope_grad"):
        E = 8 if dtype == "bf16" else 4
        hd = rng.choice([64, 72, 80, 96, 128, 128, 160, 256] if dtype == "bf16"
                        else [32, 64, 72, 96, 128, 128])
        half = rng.random() < 0.5
        unit = 2 * E if half else 2
        rot = hd if rng.random() < 0.7 else unit * rng.randint(1, hd // unit)
        rot -= rot % unit
        n_axes = min(rng.randint(1, 4), rot // 2)
        cuts = sorted(rng.sample(range(1, rot // 2), n_axes - 1)) if n_axes > 1 else []
        edges = [0] + cuts + [rot // 2]
        sec = "+".join(str(edges[i + 1] - edges[i]) for i in range(n_axes))
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        Hq = Hk * rng.choice([1, 1, 2, 3, 5])
        tokens = max(1, min(126552, _MAX_ELEMENTS // ((Hq + Hk) * hd)) // (1 if dtype == "bf16"
                                                                          else 2))
        B = rng.choice([1, 1, 2, 3])
        L = max(1, _log(rng, 1, tokens) // B)
        return dict(op=op, B=B, L=L, Hq=Hq, Hk=Hk, hd=hd, rot=rot, sec=sec, dtype=dtype,
                    pos=rng.choice(["i32", "i64", "f32"]),
                    theta=rng.choice([10000.0, 500000.0, 1000000.0]),
                    per_axis=rng.random() < 0.4, interleaved=rng.random() < 0.4, half=half,
                    norm=rng.random() < 0.6, merged=rng.random() < 0.5)
    E = 8 if dtype == "bf16" else 4
    D = E * max(1, _log(rng, 64, 8192) // E)
    rows = _log(rng, 1, min(126552, _MAX_ELEMENTS // D // (1 if dtype == "bf16" else 2)))
    B = rng.choice([1, 1, 2, 3, 5])
    L = max(1, rows // B)
    n_video = rng.choice([L, rng.randint(0, L), rng.randint(0, L)])
    c = dict(op=op, B=B, L=L, n_video=n_video, D=D, dtype=dtype)
    if op in ("drop", "drop_grad"):
        c.update(p=rng.choice([0.05, 0.1, 0.25, 0.5]),
                 resid=True if op == "drop_grad" else rng.random() < 0.7)
    else:
        c.update(mod=True if op == "rms_grad" else rng.random() < 0.5)
        if op != "ln":
            c.update(dres=rng.random() < 0.5)
    return c


def _sec(case):
    """Rotary pairs of each axis."""
    return tuple(int(v) for v in case["sec"].split("+"))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _act(g, shape, dt, outliers=True):
    """N(0, 1); 1% of the channels 20 times as large, as activations have them."""
    t = torch.randn(shape, generator=g, device=DEV)
    if outliers:
        n = round(0.01 * shape[-1])
        if n:
            t[..., torch.randperm(shape[-1], generator=g, device=DEV)[:n]] *= 20.0
    return t.to(dt)


def _vec(g, shape, mean, std, dt):
    return (mean + std * torch.randn(shape, generator=g, device=DEV)).to(dt)


def _positions(case, g):
    """[n_axes, B, L]: grid coordinates of a clip or of packed images, some far
    into a long stream; fractional ones where the case has real positions."""
    n, B, L = len(_sec(case)), case["B"], case["L"]
    r = torch.arange(L, device=DEV)
    W, H = 84, 48
    axes = [r // (W * H), (r // W) % H, r % W, r]
    p = torch.stack([axes[a] for a in range(n)]) if n > 1 else r[None]
    p = p[:, None, :].expand(n, B, L).clone()
    p += torch.randint(0, 4096, (n, B, 1), generator=g, device=DEV)
    if case["pos"] == "f32":
        return (p.double() * 0.5 + torch.rand((n, B, 1), generator=g, device=DEV)).float()
    return p.to(_POS[case["pos"]])


def _inputs(case, seed):
    g = _gen(seed)
    dt = _DT[case["dtype"]]
    op = case["op"]
    if op in ("rope", "rope_grad"):
        B, L, Hq, Hk, hd = (case[k] for k in ("B", "L", "Hq", "Hk", "hd"))
        s = dict(pos=_positions(case, g))

        def pair():
            if case["merged"]:       # q and k as columns of one projection [B, L, (Hq + 2 Hk) hd]
                qkv = _act(g, (B, L, (Hq + 2 * Hk) * hd), dt)
                q = qkv[..., :Hq * hd].view(B, L, Hq, hd)
                return q, qkv[..., Hq * hd:(Hq + Hk) * hd].view(B, L, Hk, hd)
            return _act(g, (B, L, Hq, hd), dt, False), _act(g, (B, L, Hk, hd), dt, False)

        s["q"], s["k"] = pair()
        s["gamma_q"] = _vec(g, (hd,), 1.0, 0.1, dt) if case["norm"] else None
        s["gamma_k"] = _vec(g, (hd,), 1.0, 0.1, dt) if case["norm"] else None
        if op == "rope_grad":
            s["dq_out"] = _act(g, (B, L, Hq, hd), dt, False)
            s["dk_out"] = _act(g, (B, L, Hk, hd), dt, False)
        return s
    B, L, D = case["B"], case["L"], case["D"]
    if op in ("drop", "drop_grad"):
        s = dict(branch=_act(g, (B, L, D), dt), h=None, gate=None)
        if case["resid"]:
            s["gate"] = _vec(g, (B, 2, D), 0.0, 0.1, dt)
            s["h" if op == "drop" else "dout"] = _act(g, (B, L, D), dt, op == "drop")
        s["rng"] = torch.randint(-2**62, 2**62, (2,), generator=g, device=DEV)
        return s
    s = dict(x=_act(g, (B, L, D), dt))
    # a common offset of the row, which the mean takes out again
    if op != "rms_grad":
        s["x"] += torch.randn((B, L, 1), generator=g, device=DEV).to(dt)
    s["gamma"] = _vec(g, (D,), 1.0, 0.1, dt)
    s["beta"] = _vec(g, (D,), 0.0, 0.1, dt) if op != "rms_grad" else None
    s["scale"] = _vec(g, (B, 2, D), 0.0, 0.5, dt) if case["mod"] else None
    s["shift"] = _vec(g, (B, 2, D), 0.0, 0.5, dt) if case["mod"] else None
    if op != "ln":
        s["dy"] = _act(g, (B, L, D), dt, False)
        s["dres"] = _act(g, (B, L, D), dt, False) if case["dres"] else None
    return s


EPS = 1e-6
SITE = 3       # the dropout's place in the block


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "ln_grad":      # what the forward pass left behind
        x = s["x"].float()
        mean = x.mean(-1)
        s["mean"] = mean
        s["rstd"] = 1.0 / torch.sqrt((x - mean[..., None]).square().mean(-1) + EPS)
    if case["op"] in ("rope", "rope_grad"):
        if own:
            from video_diffusion_transformer_rms_b200 import api
            s["plan"] = api.RopeAxes(case["hd"], _sec(case), theta=case["theta"],
                                     per_axis_freq=case["per_axis"],
                                     interleaved=case["interleaved"], half_split=case["half"])
        else:
            s["plan"] = _plan(case)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plan(case):
    """(axis, frequency) of every rotary pair."""
    sec, n = _sec(case), len(_sec(case))
    axis, left, a = [], list(sec), 0
    while sum(left):
        if left[a]:
            axis.append(a)
            left[a] -= 1
        if case["interleaved"] or not left[a]:
            a = (a + 1) % n
    seen, freq = [0] * n, []
    for i, a in enumerate(axis):
        e = seen[a] / sec[a] if case["per_axis"] else 2 * i / case["rot"]
        freq.append(case["theta"] ** -e)
        seen[a] += 1
    return (torch.tensor(axis, device=DEV),
            torch.tensor(freq, dtype=torch.float64, device=DEV))


def _rows(v, n_video, L):
    """Per-(sample, modality) vectors [B, 2, D] spread over the rows."""
    B, _, D = v.shape
    v = v.float()
    return torch.cat([v[:, 0:1].expand(B, n_video, D), v[:, 1:2].expand(B, L - n_video, D)], 1)


def _sums(t, n_video):
    """Sums over the rows of each (sample, modality): [B, 2, D]."""
    return torch.stack([t[:, :n_video].sum(1, dtype=torch.float64),
                        t[:, n_video:].sum(1, dtype=torch.float64)], 1).float()


def _ln(s):
    c = s["case"]
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True)
    x = x - mean
    rstd = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    y = x * rstd * s["gamma"].float() + s["beta"].float()
    if c["mod"]:
        y = y * (1.0 + _rows(s["scale"], c["n_video"], c["L"]))
        y = y + _rows(s["shift"], c["n_video"], c["L"])
    return y.to(s["x"].dtype), mean[..., 0], rstd[..., 0]


def _norm_grad(s):
    c = s["case"]
    x = s["x"].float()
    dy = s["dy"].float()
    gamma = s["gamma"].float()
    if c["op"] == "rms_grad":
        rstd = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
        xh = x * rstd
        n = xh * gamma
    else:
        rstd = s["rstd"][..., None]
        xh = (x - s["mean"][..., None]) * rstd
        n = xh * gamma + s["beta"].float()
    dn = dy
    dscale = dshift = None
    if c["mod"]:
        dscale, dshift = _sums(dy * n, c["n_video"]), _sums(dy, c["n_video"])
        dn = dy * (1.0 + _rows(s["scale"], c["n_video"], c["L"]))
    del n
    dgamma = (dn * xh).sum((0, 1), dtype=torch.float64).float()
    dbeta = None if c["op"] == "rms_grad" else dn.sum((0, 1), dtype=torch.float64).float()
    g = dn * gamma
    dx = g - xh * (g * xh).mean(-1, keepdim=True)
    if c["op"] != "rms_grad":
        dx = dx - g.mean(-1, keepdim=True)
    dx = dx * rstd
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return _present(dx.to(s["x"].dtype), dgamma, dbeta, dscale, dshift)


def _present(*ts):
    return tuple(t for t in ts if t is not None)


def _cos_sin(s):
    axis, freq = s["plan"]
    ang = s["pos"].double()[axis].permute(1, 2, 0) * freq          # [B, L, rot / 2]
    return ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]


def _rotate(t, cos, sin, c):
    P, rot = c["rot"] // 2, c["rot"]
    if c["half"]:
        a, b = t[..., :P], t[..., P:rot]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, t[..., rot:]], -1)
    a, b = t[..., 0:rot:2], t[..., 1:rot:2]
    r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([r, t[..., rot:]], -1)


def _rope(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    out = []
    for n in ("q", "k"):
        t = s[n].float()
        if c["norm"]:
            t = t * (1.0 / torch.sqrt(t.square().mean(-1, keepdim=True) + EPS))
            t = t * s["gamma_" + n].float()
        out.append(_rotate(t, cos, sin, c).to(s[n].dtype))
    return tuple(out)


def _rope_grad(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    grads, dgammas = [], []
    for n in ("q", "k"):
        d = _rotate(s["d" + n + "_out"].float(), cos, -sin, c)
        if c["norm"]:
            x = s[n].float()
            rstd = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
            xh = x * rstd
            dgammas.append((d * xh).sum((0, 1, 2), dtype=torch.float64).float())
            g = d * s["gamma_" + n].float()
            d = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
        grads.append(d.to(s[n].dtype))
    return tuple(grads + dgammas)


_M32 = 0xFFFFFFFF


def _random_words(rng, n):
    """n 32-bit words: word e is word e % 4 of Philox4x32-10 (Salmon et al.,
    2011) at counter (e / 4, offset + site), key seed."""
    key, off = rng[0], rng[1] + SITE
    c0 = torch.arange((n + 3) // 4, device=DEV)
    c1 = c0 >> 32
    c0 = c0 & _M32
    c2 = (off & _M32).expand_as(c0)
    c3 = ((off >> 32) & _M32).expand_as(c0)
    k0, k1 = key & _M32, (key >> 32) & _M32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0 = ((b >> 32) & _M32) ^ c1 ^ k0
        c1 = b & _M32
        c2 = ((a >> 32) & _M32) ^ c3 ^ k1
        c3 = a & _M32
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    return torch.stack([c0, c1, c2, c3], -1).flatten()[:n]


def _p32(p):
    return torch.tensor(p, dtype=torch.float32).item()


def _dropped(t, rng, p):
    """t / (1 - p) where the element is kept, 0 where not."""
    p = _p32(p)
    keep = _random_words(rng, t.numel()).view(t.shape) >= round(p * 2.0 ** 32)
    return torch.where(keep, t * (1.0 / (1.0 - p)), torch.zeros((), device=DEV))


def _drop(s):
    c = s["case"]
    y = _dropped(s["branch"].float(), s["rng"], c["p"])
    if c["resid"]:
        y = s["h"].float() + _rows(s["gate"], c["n_video"], c["L"]) * y
    return y.to(s["branch"].dtype)


def _drop_grad(s):
    c = s["case"]
    d = _dropped(s["dout"].float(), s["rng"], c["p"])
    dgate = _sums(d * s["branch"].float(), c["n_video"])
    return (d * _rows(s["gate"], c["n_video"], c["L"])).to(s["branch"].dtype), dgate


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"ln": _ln, "ln_grad": _norm_grad, "rms_grad": _norm_grad, "rope": _rope,
            "rope_grad": _rope_grad, "drop": _drop, "drop_grad": _drop_grad}[
                state["case"]["op"]](state)


def _run_own(s):
    from video_diffusion_transformer_rms_b200 import api
    c = s["case"]
    op = c["op"]
    if op == "ln":
        return api.layer_norm(s["x"], s["gamma"], s["beta"], s["scale"], s["shift"],
                              n_video=c["n_video"], eps=EPS)
    if op == "ln_grad":
        return _present(*api.layer_norm_backward(
            s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"], s["beta"], s["scale"],
            n_video=c["n_video"], dres=s["dres"]))
    if op == "rms_grad":
        dx, dscale, dshift, dgamma = api.rms_adaln_backward(
            s["dy"], s["x"], s["scale"], c["n_video"], gamma=s["gamma"], eps=EPS,
            dres=s["dres"])
        return dx, dgamma, dscale, dshift
    if op == "rope":
        return api.rope_axes(s["q"], s["k"], s["pos"], s["plan"], s["gamma_q"], s["gamma_k"],
                             qk_norm=c["norm"], eps=EPS)
    if op == "rope_grad":
        return _present(*api.rope_axes_backward(
            s["dq_out"], s["dk_out"], s["pos"], s["plan"], s["q"], s["k"], s["gamma_q"],
            s["gamma_k"], qk_norm=c["norm"], eps=EPS))
    if op == "drop":
        if c["resid"]:
            return api.dropout_residual(s["h"], s["branch"], s["gate"], c["n_video"], c["p"],
                                        s["rng"], site=SITE)
        return api.dropout(s["branch"], c["p"], s["rng"], site=SITE)
    return api.dropout_residual_backward(s["dout"], s["branch"], s["gate"], c["n_video"], c["p"],
                                         s["rng"], site=SITE)


def work(case):
    """Bytes read and written once, and the arithmetic that cannot be left out."""
    es, op = _ES[case["dtype"]], case["op"]
    if op in ("rope", "rope_grad"):
        rows = case["B"] * case["L"]
        n = rows * (case["Hq"] + case["Hk"]) * case["hd"]
        pos = rows * len(_sec(case)) * (8 if case["pos"] == "i64" else 4)
        acts = 2 + (op == "rope_grad" and case["norm"])
        return {"bytes": acts * n * es + pos + 4 * case["hd"] * es * case["norm"],
                "flops": n * (3 + case["norm"] * (4 if op == "rope" else 11))}
    B, D = case["B"], case["D"]
    n = B * case["L"] * D
    vec, rows = D * es, B * case["L"]
    if op == "drop":
        acts = 2 + case["resid"]
        return {"bytes": acts * n * es + 2 * B * vec * case["resid"], "flops": 4 * n}
    if op == "drop_grad":
        return {"bytes": 3 * n * es + 2 * B * (vec + 4 * D), "flops": 6 * n}
    if op == "ln":
        return {"bytes": 2 * n * es + 2 * vec + 8 * rows + 4 * B * vec * case["mod"],
                "flops": n * (8 + 2 * case["mod"])}
    stats = 8 * rows * (op == "ln_grad")
    return {"bytes": (3 + case["dres"]) * n * es + stats + 2 * vec + 8 * D
            + 2 * B * (vec + 8 * D) * case["mod"],
            "flops": n * (14 + 2 * case["mod"])}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits, a block of rows at a time
# ---------------------------------------------------------------------------

_BLOCK = 1 << 24       # elements held in fp64 at a time


def _blocks(rows, width):
    step = max(1, _BLOCK // max(1, width))
    return [(i, min(rows, i + step)) for i in range(0, rows, step)]


def _segments(case):
    """(first row, past the last, sample, modality) of the flattened rows."""
    L, nv = case["L"], case["n_video"]
    out = []
    for b in range(case["B"]):
        out += [(b * L, b * L + nv, b, 0), (b * L + nv, (b + 1) * L, b, 1)]
    return out


def _exact_norm(case, s):
    """The norm as a function of its inputs, row block by row block; gradients
    from the derivative of the normalisation written as a projection."""
    D, op = case["D"], case["op"]
    rows = case["B"] * case["L"]
    f = torch.float64
    x, dt = s["x"].view(rows, D), s["x"].dtype
    g = s["gamma"].to(f)
    be = s["beta"].to(f) if s["beta"] is not None else torch.zeros(D, dtype=f, device=DEV)
    center = op != "rms_grad"
    # an output of 16 bits is kept in 32, far below its own rounding
    y = torch.empty((rows, D), dtype=f if dt == torch.float32 else torch.float32, device=DEV)
    mean = torch.empty(rows, dtype=f, device=DEV)
    rstd = torch.empty(rows, dtype=f, device=DEV)
    dg, db = torch.zeros(D, dtype=f, device=DEV), torch.zeros(D, dtype=f, device=DEV)
    dsc = torch.zeros((case["B"], 2, D), dtype=f, device=DEV)
    dsh = torch.zeros_like(dsc)
    for r0, r1, b, m in _segments(case):
        fac = 1.0 + s["scale"][b, m].to(f) if case["mod"] else torch.ones_like(g)
        add = s["shift"][b, m].to(f) if case["mod"] else torch.zeros_like(g)
        for i, j in _blocks(r1 - r0, D):
            i, j = r0 + i, r0 + j
            v = x[i:j].to(f)
            mu = v.sum(1) / D if center else torch.zeros(j - i, dtype=f, device=DEV)
            v = v - mu[:, None]
            rs = ((v * v).sum(1) / D + EPS).rsqrt()
            if op == "ln_grad":      # the given statistics, as the operator takes them
                mu = s["mean"].view(rows)[i:j].to(f)
                rs = s["rstd"].view(rows)[i:j].to(f)
                v = x[i:j].to(f) - mu[:, None]
            u = v * rs[:, None]
            if op == "ln":
                y[i:j] = ((u * g + be) * fac + add).to(y.dtype)
                mean[i:j], rstd[i:j] = mu, rs
                continue
            d = s["dy"].view(rows, D)[i:j].to(f)
            dsh[b, m] += d.sum(0)
            dsc[b, m] += (d * (u * g + be)).sum(0)
            d = d * fac
            dg += (d * u).sum(0)
            db += d.sum(0)
            d = d * g
            t = u * ((d * u).sum(1) / D)[:, None]
            if center:
                t = t + (d.sum(1) / D)[:, None]
            d = (d - t) * rs[:, None]
            if s["dres"] is not None:
                d = d + s["dres"].view(rows, D)[i:j].to(f)
            y[i:j] = d.to(y.dtype)
    y = y.view(case["B"], case["L"], D)
    if op == "ln":
        return y, mean.view(case["B"], -1), rstd.view(case["B"], -1)
    return _present(y, dg, db if center else None, dsc if case["mod"] else None,
                    dsh if case["mod"] else None)


def _exact_rope(case, s):
    """Every pair as a complex number, multiplied by exp(i angle)."""
    f = torch.float64
    B, L, hd, rot = case["B"], case["L"], case["hd"], case["rot"]
    P, n = rot // 2, len(_sec(case))
    # the pairs dealt to the axes, contiguous or in turn
    order = []
    if case["interleaved"]:
        for j in range(max(_sec(case))):
            order += [(a, j) for a in range(n) if j < _sec(case)[a]]
    else:
        order = [(a, j) for a in range(n) for j in range(_sec(case)[a])]
    w = torch.tensor([math.exp(-math.log(case["theta"])
                               * (j / _sec(case)[a] if case["per_axis"] else i / P))
                      for i, (a, j) in enumerate(order)], dtype=f, device=DEV)
    which = [a for a, _ in order]
    first = list(range(P)) if case["half"] else list(range(0, rot, 2))
    second = list(range(P, rot)) if case["half"] else list(range(1, rot, 2))
    grad = case["op"] == "rope_grad"
    pos = s["pos"].reshape(n, B * L).to(f)
    od = torch.float32 if case["dtype"] == "bf16" else f
    outs, extra = [], []
    for name in ("q", "k"):
        src = (s["d" + name + "_out"] if grad else s[name])
        H = src.shape[2]
        src = src.reshape(B * L, H, hd)
        x = s[name].reshape(B * L, H, hd)
        out = torch.empty((B * L, H, hd), dtype=od, device=DEV)
        ga = s["gamma_" + name].to(f) if case["norm"] else None
        dga = torch.zeros(hd, dtype=f, device=DEV)
        for i, j in _blocks(B * L, H * hd):
            t = src[i:j].to(f)
            phi = torch.stack([pos[a, i:j] for a in which], 1) * w
            if grad:
                phi = -phi
            if case["norm"]:
                xb = x[i:j].to(f)
                r = ((xb * xb).sum(-1, keepdim=True) / hd + EPS).rsqrt()
                if not grad:
                    t = xb * r * ga
            z = torch.complex(t[..., first], t[..., second]) * torch.polar(
                torch.ones_like(phi), phi)[:, None]
            t = t.clone()
            t[..., first], t[..., second] = z.real, z.imag
            if grad and case["norm"]:
                u = xb * r
                dga += (t * u).sum((0, 1))
                t = t * ga
                t = (t - u * (t * u).sum(-1, keepdim=True) / hd) * r
            out[i:j] = t.to(od)
        outs.append(out.view(B, L, H, hd))
        if grad and case["norm"]:
            extra.append(dga)
    return tuple(outs + extra)


def _exact_words(first, count, rng, site):
    """Philox4x32-10 for elements first .. first + count (first a multiple of
    4), products from 16-bit halves so that nothing wraps."""
    def mul(x, m):
        lo, hi = x * (m & 0xFFFF), x * (m >> 16)                   # both below 2^48
        s = lo + ((hi & 0xFFFF) << 16)
        return (hi >> 16) + (s >> 32), s & _M32
    seed, offset = (int(v) % 2**64 for v in rng.tolist())
    offset = (offset + site) % 2**64
    i = torch.arange(first // 4, (first + count + 3) // 4, device=DEV)
    x = [i % 2**32, i // 2**32, torch.full_like(i, offset % 2**32),
         torch.full_like(i, offset // 2**32)]
    key = [seed % 2**32, seed // 2**32]
    for r in range(10):
        ka, kb = (key[0] + r * 0x9E3779B9) % 2**32, (key[1] + r * 0xBB67AE85) % 2**32
        h0, l0 = mul(x[0], 0xD2511F53)
        h1, l1 = mul(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ ka, l1, h0 ^ x[3] ^ kb, l0]
    return torch.stack(x, 1).view(-1)[:count]


def _exact_drop(case, s):
    f = torch.float64
    D, rows = case["D"], case["B"] * case["L"]
    p = _p32(case["p"])
    thr = int(round(p * 4294967296.0))
    grad = case["op"] == "drop_grad"
    br = s["branch"].view(rows, D)
    out = torch.empty((rows, D), dtype=torch.float32 if case["dtype"] == "bf16" else f,
                      device=DEV)
    dgate = torch.zeros((case["B"], 2, D), dtype=f, device=DEV)
    for r0, r1, b, m in _segments(case):
        gate = s["gate"][b, m].to(f) if case["resid"] else torch.ones(D, dtype=f, device=DEV)
        for i, j in _blocks(r1 - r0, D):
            i, j = r0 + i, r0 + j
            w = _exact_words(i * D, (j - i) * D, s["rng"], SITE).view(j - i, D)
            keep = (w >= thr).to(f) / (1.0 - p)
            if grad:
                d = s["dout"].view(rows, D)[i:j].to(f) * keep
                dgate[b, m] += (d * br[i:j].to(f)).sum(0)
                out[i:j] = (d * gate).to(out.dtype)
            else:
                o = br[i:j].to(f) * keep * gate
                if case["resid"]:
                    o = o + s["h"].view(rows, D)[i:j].to(f)
                out[i:j] = o.to(out.dtype)
    out = out.view(case["B"], case["L"], D)
    return (out, dgate) if grad else out


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "ln_grad":
        x = s["x"].float()
        s["mean"] = x.mean(-1)
        s["rstd"] = 1.0 / torch.sqrt((x - s["mean"][..., None]).square().mean(-1) + EPS)
    if case["op"] in ("rope", "rope_grad"):
        return _exact_rope(case, s)
    return _exact_drop(case, s) if case["op"] in ("drop", "drop_grad") else _exact_norm(case, s)
