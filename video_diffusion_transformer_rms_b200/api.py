"""Tensor-level calls on top of the C ABI: take torch CUDA tensors, pass
their pointers, shapes and the current stream to libsol.  Marshalling only
(PyTorch allocates outputs when the caller does not pass them); the
arithmetic runs in libsol's kernels.

No call is recorded by autograd: a result does not require a gradient even where
an input does, and nothing warns of it.  The gradients are the _backward calls;
a caller that trains through autograd wraps the pairs in torch.autograd.Function.
"""
import contextlib
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import _abi

_DT = {torch.float32: _abi.SOL_F32, torch.bfloat16: _abi.SOL_BF16}


def _dtype(*ts) -> int:
    dts = {t.dtype for t in ts if t is not None}
    if len(dts) != 1:
        raise TypeError(f"all tensors must share one dtype, got {dts}")
    dt = dts.pop()
    if dt not in _DT:
        raise TypeError(f"dtype {dt} is not supported (float32 or bfloat16)")
    return _DT[dt]


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libsol takes CUDA tensors")
    return t.data_ptr()


def _expect(t: Optional[torch.Tensor], shape, name: str, like: torch.Tensor):
    """The library sees only pointers, so every tensor handed to it must be
    contiguous, of exactly this shape, and on the device of `like`."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}, got "
                         f"{tuple(t.shape)}{'' if t.is_contiguous() else ' (not contiguous)'}")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, the inputs on {like.device}")


def _stream(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def rms_adaln(x: torch.Tensor, scale: torch.Tensor, shift: torch.Tensor, n_video: int,
              gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
              out: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """y = RMSNorm(x) * gamma * (1 + scale[b, m]) + shift[b, m]; x: [B, L, D],
    scale/shift: [B, 2, D]."""
    if x.dim() != 3 or not x.is_contiguous():
        raise ValueError("x must be a contiguous [B, L, D] tensor")
    B, L, D = x.shape
    for t, shape, name in ((scale, (B, 2, D), "scale"), (shift, (B, 2, D), "shift"),
                           (gamma, (D,), "gamma"), (out, (B, L, D), "out")):
        _expect(t, shape, name, x)
    y = torch.empty_like(x) if out is None else out
    _abi.check(_abi.sol_rms_adaln(_ptr(x), _ptr(y), _ptr(scale), _ptr(shift), _ptr(gamma),
                                  B, L, n_video, D, eps, _dtype(x, y, scale, shift, gamma),
                                  _stream(stream)))
    return y


def gate_residual(h: torch.Tensor, branch: torch.Tensor, gate: torch.Tensor, n_video: int,
                  out: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out = h + gate[b, m] * branch; h/branch: [B, L, D], gate: [B, 2, D]."""
    if h.dim() != 3 or not h.is_contiguous():
        raise ValueError("h must be a contiguous [B, L, D] tensor")
    B, L, D = h.shape
    for t, shape, name in ((branch, (B, L, D), "branch"), (gate, (B, 2, D), "gate"),
                           (out, (B, L, D), "out")):
        _expect(t, shape, name, h)
    o = torch.empty_like(h) if out is None else out
    _abi.check(_abi.sol_gate_residual(_ptr(h), _ptr(branch), _ptr(gate), _ptr(o), B, L,
                                      n_video, D, _dtype(h, branch, gate, o), _stream(stream)))
    return o


def gate_residual_rms_adaln(h: torch.Tensor, branch: torch.Tensor, gate: torch.Tensor,
                            scale: torch.Tensor, shift: torch.Tensor, n_video: int,
                            gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
                            h_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None
                            ) -> Tuple[torch.Tensor, torch.Tensor]:
    """h_out = h + gate[b, m] * branch; y = RMS-AdaLN(h_out) with scale/shift;
    returns (h_out, y).  Pass h_out=h to update the residual stream in place."""
    if h.dim() != 3 or not h.is_contiguous():
        raise ValueError("h must be a contiguous [B, L, D] tensor")
    B, L, D = h.shape
    for t, shape, name in ((branch, (B, L, D), "branch"), (gate, (B, 2, D), "gate"),
                           (scale, (B, 2, D), "scale"), (shift, (B, 2, D), "shift"),
                           (gamma, (D,), "gamma"), (h_out, (B, L, D), "h_out"),
                           (y, (B, L, D), "y")):
        _expect(t, shape, name, h)
    ho = torch.empty_like(h) if h_out is None else h_out
    yo = torch.empty_like(h) if y is None else y
    _abi.check(_abi.sol_gate_residual_rms_adaln(
        _ptr(h), _ptr(branch), _ptr(gate), _ptr(ho), _ptr(yo), _ptr(scale), _ptr(shift),
        _ptr(gamma), B, L, n_video, D, eps, _dtype(h, branch, gate, ho, yo, scale, shift, gamma),
        _stream(stream)))
    return ho, yo


def residual_change(cur: torch.Tensor, prev: torch.Tensor,
                    prev_out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """First-Block-Cache change of a [B, L, D] residual against the previous
    step's: returns a [B + 1, 3] float64 CUDA tensor of (sum |cur - prev|,
    sum |prev|, their ratio) per sample and, in the last row, for the batch.
    With prev_out (may be prev itself) the cache is refreshed to cur in the
    same pass.  The workspace is allocated by PyTorch unless given."""
    if cur.dim() != 3 or not cur.is_contiguous():
        raise ValueError("cur must be a contiguous [B, L, D] tensor")
    B, L, D = cur.shape
    for t, shape, name in ((prev, (B, L, D), "prev"), (prev_out, (B, L, D), "prev_out"),
                           (out, (B + 1, 3), "out")):
        _expect(t, shape, name, cur)
    if out is not None and out.dtype != torch.float64:
        raise TypeError("out must be float64")
    if workspace is not None:
        _expect(workspace, (workspace.numel(),), "workspace", cur)
    need = _abi.sol_residual_change_workspace_bytes(B)
    ws = workspace if workspace is not None else torch.empty(
        max(need, 16), dtype=torch.uint8, device=cur.device)
    o = out if out is not None else torch.empty((B + 1, 3), dtype=torch.float64,
                                                device=cur.device)
    _abi.check(_abi.sol_residual_change(
        _ptr(cur), _ptr(prev), _ptr(prev_out), B, L, D, _ptr(o), _ptr(ws),
        ws.numel() * ws.element_size(), _dtype(cur, prev, prev_out), _stream(stream)))
    return o


class RopeTable:
    """A rotary table on the device (sol_rope_table): row p holds cos(p*f_i)
    for every rotary pair i, then sin(p*f_i), fp32, for positions
    0 .. n_pos-1.  Build it once per video shape; pass it as `table=` to
    qknorm_rope3d / qknorm_rope3d_ex."""

    def __init__(self, n_pos: int, head_dim: int, sections: Sequence[int] = (16, 24, 24),
                 theta: float = 10000.0, per_axis_freq: bool = False, device=None,
                 stream: Optional[torch.cuda.Stream] = None):
        nbytes = _abi.sol_rope_table_bytes(n_pos, head_dim)
        if nbytes == 0 and n_pos != 0:
            raise ValueError("n_pos must be >= 0 and head_dim even in [2, 256]")
        self.data = torch.empty(max(nbytes // 4, 4), dtype=torch.float32, device=device)
        self.n_pos, self.head_dim = n_pos, head_dim
        self.sections = tuple(int(x) for x in sections)
        self.theta, self.per_axis_freq = float(theta), bool(per_axis_freq)
        st, sh, sw = self.sections
        self.desc = _abi.RopeTable(self.data.data_ptr(), n_pos, head_dim, st, sh, sw, theta,
                                   int(self.per_axis_freq))
        _abi.check(_abi.sol_rope_table_build(self.desc, _stream(stream)))

    @classmethod
    def for_grid(cls, T: int, H: int, W: int, n_audio: int, head_dim: int, **kw):
        """A table covering every position of a T x H x W video grid plus
        n_audio audio tokens."""
        n = max(n_audio, max(T, H, W) if T * H * W > 0 else 0)
        return cls(n, head_dim, **kw)

    def check(self, head_dim: int, sections: Sequence[int], theta: float,
              per_axis_freq: bool = False):
        if (head_dim != self.head_dim or tuple(sections) != self.sections
                or float(theta) != self.theta or bool(per_axis_freq) != self.per_axis_freq):
            raise ValueError("the rotary table was built for other head_dim, sections, theta "
                             "or frequency rule")


def qknorm_rope3d(qkv: torch.Tensor, T: int, H: int, W: int, n_audio: int, n_heads: int,
                  head_dim: int, sections: Sequence[int] = (16, 24, 24),
                  gamma_q: Optional[torch.Tensor] = None,
                  gamma_k: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  theta: float = 10000.0, q_out: Optional[torch.Tensor] = None,
                  k_out: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None,
                  table: Optional[RopeTable] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-head QKNorm + 3D RoPE of q and k in a merged qkv [B, L, >=2D]
    (row stride qkv.stride(1)); returns (q, k) as [B, L, D] views.  With
    `table` the (cos, sin) come from that rotary table (sol_qknorm_rope3d_tab)
    instead of being computed per row."""
    if qkv.dim() != 3 or qkv.stride(2) != 1 or qkv.stride(0) != qkv.shape[1] * qkv.stride(1):
        raise ValueError("qkv must be [B, L, C] with unit column stride and packed rows")
    B, L, _ = qkv.shape
    D = n_heads * head_dim
    if L != T * H * W + n_audio:
        raise ValueError("L must equal T*H*W + n_audio")
    for t, name in ((gamma_q, "gamma_q"), (gamma_k, "gamma_k")):
        _expect(t, (head_dim,), name, qkv)
    if q_out is None and k_out is None:
        buf = torch.empty((B, L, 2 * D), dtype=qkv.dtype, device=qkv.device)
        q_out, k_out = buf[..., :D], buf[..., D:]
    elif q_out is None or k_out is None:
        raise ValueError("pass both q_out and k_out, or neither")
    if q_out.stride() != k_out.stride() or q_out.stride(2) != 1:
        raise ValueError("q_out and k_out must share a row stride with unit column stride")
    for t, name in ((q_out, "q_out"), (k_out, "k_out")):
        if tuple(t.shape) != (B, L, D) or t.stride(0) != L * t.stride(1):
            raise ValueError(f"{name} must be a [B, L, D] view with packed rows")
        if t.device != qkv.device:
            raise ValueError(f"{name} is on {t.device}, qkv on {qkv.device}")
    ld_out = q_out.stride(1)
    st, sh, sw = sections
    dt = _dtype(qkv, q_out, k_out, gamma_q, gamma_k)
    if table is not None:
        table.check(head_dim, sections, theta)
        if table.data.device != qkv.device:
            raise ValueError(f"the rotary table is on {table.data.device}, qkv on {qkv.device}")
        _abi.check(_abi.sol_qknorm_rope3d_tab(
            _ptr(qkv), qkv.stride(1), _ptr(q_out), _ptr(k_out), ld_out, _ptr(gamma_q),
            _ptr(gamma_k), table.desc, B, T, H, W, n_audio, n_heads, eps, dt, _stream(stream)))
    else:
        _abi.check(_abi.sol_qknorm_rope3d(
            _ptr(qkv), qkv.stride(1), _ptr(q_out), _ptr(k_out), ld_out, _ptr(gamma_q),
            _ptr(gamma_k), B, T, H, W, n_audio, n_heads, head_dim, st, sh, sw, eps, theta, dt,
            _stream(stream)))
    return q_out, k_out


def qknorm_rope3d_ex(qkv: torch.Tensor, T: int, H: int, W: int, n_audio: int, n_heads: int,
                     head_dim: int, sections: Sequence[int] = (16, 24, 24),
                     gamma_q: Optional[torch.Tensor] = None,
                     gamma_k: Optional[torch.Tensor] = None, eps: float = 1e-6,
                     theta: float = 10000.0, layout: str = "bshd", half_split: bool = False,
                     int8: bool = False, per_axis_freq: bool = False, quantize_v: bool = False,
                     stream: Optional[torch.cuda.Stream] = None,
                     table: Optional[RopeTable] = None):
    """QKNorm + 3D RoPE epilogue variants (bf16 input).  layout "bshd" gives
    q, k as [B, L, H, hd]; "bhsd" as attention's [B, H, L, hd].  half_split
    pairs element i with i + hd/2; per_axis_freq gives each rotary section a
    frequency ladder of its own.  int8 returns (q, k, q_scale, k_scale): int8
    codes in the chosen layout and scales fp32 [B, L, H]; with quantize_v
    also (v, v_scale), v quantised as it stands; else (q, k) in bf16.  With
    `table` the (cos, sin) come from that rotary table
    (sol_qknorm_rope3d_ex_tab)."""
    if qkv.dim() != 3 or qkv.stride(2) != 1 or qkv.stride(0) != qkv.shape[1] * qkv.stride(1):
        raise ValueError("qkv must be [B, L, C] with unit column stride and packed rows")
    if quantize_v and not int8:
        raise ValueError("quantize_v needs int8=True")
    B, L, _ = qkv.shape
    if L != T * H * W + n_audio:
        raise ValueError("L must equal T*H*W + n_audio")
    for t, name in ((gamma_q, "gamma_q"), (gamma_k, "gamma_k")):
        _expect(t, (head_dim,), name, qkv)
    odt = torch.int8 if int8 else qkv.dtype
    if layout == "bshd":
        shape = (B, L, n_heads, head_dim)
        strides = (L * n_heads * head_dim, n_heads * head_dim, head_dim)
    elif layout == "bhsd":
        shape = (B, n_heads, L, head_dim)
        strides = (n_heads * L * head_dim, head_dim, L * head_dim)
    else:
        raise ValueError("layout must be 'bshd' or 'bhsd'")
    q = torch.empty(shape, dtype=odt, device=qkv.device)
    k = torch.empty(shape, dtype=odt, device=qkv.device)
    qs = ks = v = vs = None
    if int8:
        qs = torch.empty((B, L, n_heads), dtype=torch.float32, device=qkv.device)
        ks = torch.empty((B, L, n_heads), dtype=torch.float32, device=qkv.device)
    if quantize_v:
        v = torch.empty(shape, dtype=odt, device=qkv.device)
        vs = torch.empty((B, L, n_heads), dtype=torch.float32, device=qkv.device)
    lay = _abi.QkLayout(strides[0], strides[1], strides[2], int(bool(half_split)),
                        int(bool(int8)), _ptr(qs), _ptr(ks), int(bool(per_axis_freq)), 0,
                        _ptr(v), _ptr(vs))
    st, sh, sw = sections
    dt = _dtype(qkv, gamma_q, gamma_k)
    if table is not None:
        table.check(head_dim, sections, theta, per_axis_freq)
        if table.data.device != qkv.device:
            raise ValueError(f"the rotary table is on {table.data.device}, qkv on {qkv.device}")
        _abi.check(_abi.sol_qknorm_rope3d_ex_tab(
            _ptr(qkv), qkv.stride(1), _ptr(q), _ptr(k), lay, _ptr(gamma_q), _ptr(gamma_k),
            table.desc, B, T, H, W, n_audio, n_heads, eps, dt, _stream(stream)))
    else:
        _abi.check(_abi.sol_qknorm_rope3d_ex(
            _ptr(qkv), qkv.stride(1), _ptr(q), _ptr(k), lay, _ptr(gamma_q), _ptr(gamma_k), B, T,
            H, W, n_audio, n_heads, head_dim, st, sh, sw, eps, theta, dt, _stream(stream)))
    if quantize_v:
        return q, k, qs, ks, v, vs
    return (q, k, qs, ks) if int8 else (q, k)


def gemm_gelu(A: torch.Tensor, B: torch.Tensor, bias: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """C = gelu_tanh(A @ B.T + bias) on the tensor cores; A [M, K], B [N, K]
    (a Linear weight), bias [N], all bf16; returns C [M, N] bf16."""
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[1]:
        raise ValueError("A must be [M, K] and B [N, K]")
    if not (A.is_contiguous() and B.is_contiguous()):
        raise ValueError("A and B must be contiguous")
    M, K = A.shape
    N = B.shape[0]
    _expect(B, (N, K), "B", A)
    _expect(bias, (N,), "bias", A)
    _expect(out, (M, N), "out", A)
    C = torch.empty((M, N), dtype=A.dtype, device=A.device) if out is None else out
    need = _abi.sol_gemm_gelu_workspace_bytes(M, N, K)
    ws = torch.empty(need, dtype=torch.uint8, device=A.device) if need else None
    _dtype(A, B, bias, C)
    if A.dtype != torch.bfloat16:
        raise TypeError("sol_gemm_gelu takes bf16 tensors")
    _abi.check(_abi.sol_gemm_gelu(_ptr(A), _ptr(B), _ptr(bias), _ptr(C), M, N, K, _ptr(ws),
                                  need, _stream(stream)))
    return C


# ---------------------------------------------------------------------------
# training operators
# ---------------------------------------------------------------------------

_NO_CONTEXT = contextlib.nullcontext()


# These wrappers are the whole cost of a small call, so an operand is checked
# and turned into its address in one step.

def _arg(t: Optional[torch.Tensor], shape, name: str, like: torch.Tensor, dtype=None):
    """Address of a contiguous operand of this shape, on the device of `like`
    and of its dtype (or of the one given); None for None."""
    if t is None:
        return None
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}, got "
                         f"{tuple(t.shape)}{'' if t.is_contiguous() else ' (not contiguous)'}")
    if t.get_device() != like.get_device():
        raise ValueError(f"{name} is on {t.device}, the inputs on {like.device}")
    if dtype is None:
        if t.dtype is not like.dtype:
            raise TypeError(f"all tensors must share one dtype, got {t.dtype} for {name} and "
                            f"{like.dtype}")
    elif t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype).split('.')[1]}, got {t.dtype}")
    return t.data_ptr()


def _io_dtype(t: torch.Tensor) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"dtype {t.dtype} is not supported (float32 or bfloat16)")
    return dt


def _on(t: torch.Tensor, stream: Optional[torch.cuda.Stream]):
    """The context a call on `t` runs in: t's device is current, and `stream`,
    where one is given, is the current stream, so that outputs and workspaces
    allocated inside belong to the stream that uses them."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("libsol takes CUDA tensors")
    if stream is not None:
        if stream.device != t.device:
            raise ValueError(f"the stream is on {stream.device}, the inputs on {t.device}")
        return torch.cuda.stream(stream)
    if dev != torch._C._cuda_getDevice():
        return torch.cuda.device(dev)
    return _NO_CONTEXT


def _current(t: torch.Tensor) -> int:
    """Handle of the current stream of t's device."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _workspace(given: Optional[torch.Tensor], need: int, like: torch.Tensor) -> torch.Tensor:
    if given is None:
        return torch.empty_strided((need if need > 16 else 16,), (1,), dtype=torch.uint8,
                                   device=like.device)
    _arg(given, given.shape, "workspace", like, given.dtype)
    return given


def _rows3(x: torch.Tensor, n_video: Optional[int], name: str):
    if x.dim() != 3 or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [B, L, D] tensor")
    B, L, D = x.shape
    return B, L, D, L if n_video is None else n_video


def _fp32(shape, stride, like: torch.Tensor) -> torch.Tensor:
    # (the cheapest of PyTorch's allocation calls by about 1 us)
    return torch.empty_strided(shape, stride, dtype=torch.float32, device=like.device)


def _packed(t: torch.Tensor) -> torch.Tensor:
    """An uninitialised contiguous [B, L, H, hd] tensor like t, whose strides may
    be any."""
    B, L, H, hd = t.shape
    return torch.empty_strided((B, L, H, hd), (L * H * hd, H * hd, hd, 1), dtype=t.dtype,
                               device=t.device)


def layer_norm(x: torch.Tensor, gamma: Optional[torch.Tensor] = None,
               beta: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
               shift: Optional[torch.Tensor] = None, n_video: Optional[int] = None,
               eps: float = 1e-6, stats: bool = True, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None
               ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """y = (LayerNorm(x) * gamma + beta) * (1 + scale[b, m]) + shift[b, m];
    x: [B, L, D], gamma/beta: [D] or None, scale/shift: [B, 2, D] or both
    None.  Returns (y, mean, rstd); the statistics, fp32 [B, L], are what
    layer_norm_backward takes, and None with stats=False."""
    B, L, D, nv = _rows3(x, n_video, "x")
    vec, mod = (D,), (B, 2, D)
    args = (_arg(gamma, vec, "gamma", x), _arg(beta, vec, "beta", x),
            _arg(scale, mod, "scale", x), _arg(shift, mod, "shift", x))
    py = _arg(out, x.shape, "out", x)
    dt = _io_dtype(x)
    with _on(x, stream):
        y = out
        if y is None:
            y = torch.empty_like(x)
            py = y.data_ptr()
        mean = rstd = pm = pr = None
        if stats:
            mean, rstd = _fp32((B, L), (L, 1), x), _fp32((B, L), (L, 1), x)
            pm, pr = mean.data_ptr(), rstd.data_ptr()
        _abi.check(_abi.sol_layer_norm(x.data_ptr(), py, pm, pr, *args, B, L, nv, D, eps, dt,
                                       _current(x)))
    return y, mean, rstd


class NormGrads(NamedTuple):
    """Gradients of layer_norm; None where the input was not given.  Those of
    vectors are fp32."""
    dx: torch.Tensor
    dgamma: Optional[torch.Tensor]
    dbeta: Optional[torch.Tensor]
    dscale: Optional[torch.Tensor]
    dshift: Optional[torch.Tensor]


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor, gamma: Optional[torch.Tensor] = None,
                        beta: Optional[torch.Tensor] = None,
                        scale: Optional[torch.Tensor] = None, n_video: Optional[int] = None,
                        dres: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> NormGrads:
    """Gradients of layer_norm(x, gamma, beta, scale, shift) for dy.  mean and
    rstd are those the forward call returned; dres, a gradient of x's shape, is
    added to dx.  dx may be dy, x or dres (in place).  The workspace
    (sol_norm_backward_workspace_bytes) is allocated by PyTorch unless given."""
    B, L, D, nv = _rows3(x, n_video, "x")
    shape, rows, vec, mod = x.shape, (B, L), (D,), (B, 2, D)
    args = (_arg(dy, shape, "dy", x), x.data_ptr(), _arg(mean, rows, "mean", x, torch.float32),
            _arg(rstd, rows, "rstd", x, torch.float32), _arg(gamma, vec, "gamma", x),
            _arg(beta, vec, "beta", x), _arg(scale, mod, "scale", x),
            _arg(dres, shape, "dres", x))
    pd = _arg(dx, shape, "dx", x)
    dt = _io_dtype(x)
    with _on(x, stream):
        if dx is None:
            dx = torch.empty_like(x)
            pd = dx.data_ptr()
        dgamma = dbeta = dscale = dshift = pg = pb = ps = ph = None
        if gamma is not None:
            dgamma = _fp32(vec, (1,), x)
            pg = dgamma.data_ptr()
        if beta is not None:
            dbeta = _fp32(vec, (1,), x)
            pb = dbeta.data_ptr()
        if scale is not None:
            dscale, dshift = _fp32(mod, (2 * D, D, 1), x), _fp32(mod, (2 * D, D, 1), x)
            ps, ph = dscale.data_ptr(), dshift.data_ptr()
        ws = _workspace(workspace, _abi.sol_norm_backward_workspace_bytes(B, L, D), x)
        _abi.check(_abi.sol_layer_norm_backward(
            *args, pd, pg, pb, ps, ph, B, L, nv, D, ws.data_ptr(), ws.nbytes, dt, _current(x)))
    return NormGrads(dx, dgamma, dbeta, dscale, dshift)


def rms_adaln_backward(dy: torch.Tensor, x: torch.Tensor, scale: torch.Tensor, n_video: int,
                       gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
                       dres: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None
                       ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor,
                                  Optional[torch.Tensor]]:
    """Gradients (dx, dscale, dshift, dgamma) of rms_adaln(x, scale, shift,
    n_video, gamma, eps) for dy; those of vectors fp32, dgamma None without
    gamma.  dres, dx and workspace as for layer_norm_backward."""
    B, L, D, nv = _rows3(x, n_video, "x")
    shape = x.shape
    args = (_arg(dy, shape, "dy", x), x.data_ptr(), _arg(scale, (B, 2, D), "scale", x),
            _arg(gamma, (D,), "gamma", x), _arg(dres, shape, "dres", x))
    pd = _arg(dx, shape, "dx", x)
    dt = _io_dtype(x)
    with _on(x, stream):
        if dx is None:
            dx = torch.empty_like(x)
            pd = dx.data_ptr()
        mod, stride = (B, 2, D), (2 * D, D, 1)
        dscale, dshift = _fp32(mod, stride, x), _fp32(mod, stride, x)
        dgamma = None if gamma is None else _fp32((D,), (1,), x)
        ws = _workspace(workspace, _abi.sol_norm_backward_workspace_bytes(B, L, D), x)
        _abi.check(_abi.sol_rms_adaln_backward(
            *args, pd, dscale.data_ptr(), dshift.data_ptr(),
            None if gamma is None else dgamma.data_ptr(), B, L, nv, D, eps, ws.data_ptr(),
            ws.nbytes, dt, _current(x)))
    return dx, dscale, dshift, dgamma


def _rng_arg(rng: Optional[torch.Tensor], p: float, like: torch.Tensor):
    if rng is None:
        if p != 0:
            raise ValueError("rng is needed with p > 0")
        return None
    if rng.dtype is not torch.int64 and rng.dtype is not torch.uint64:
        raise TypeError("rng must be int64 or uint64: (seed, offset)")
    return _arg(rng, (2,), "rng", like, rng.dtype)


def dropout(x: torch.Tensor, p: float, rng: Optional[torch.Tensor], site: int = 0,
            out: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """x / (1 - p) where the generator keeps the element, else 0; x: a contiguous
    tensor whose last dimension is one that layer_norm takes.  The mask is a
    function of (seed, offset + site, the element's index, p), with rng = (seed,
    offset) two int64 on x's device: the gradient is dropout(dout, p, rng,
    site).  Every step moves offset by at least its number of sites, or masks come
    again; ranks and parts of a batch need seeds of their own."""
    if x.dim() < 1 or not x.is_contiguous():
        raise ValueError("x must be a contiguous tensor")
    po = _arg(out, x.shape, "out", x)
    prng = _rng_arg(rng, p, x)
    D = x.shape[-1]
    rows = x.numel() // D if D else 0
    dt = _io_dtype(x)
    with _on(x, stream):
        if out is None:
            out = torch.empty_like(x)
            po = out.data_ptr()
        if rows:
            _abi.check(_abi.sol_dropout_residual(None, x.data_ptr(), None, po, prng,
                                                 site % 2**64, p, 1, rows, rows, D, dt,
                                                 _current(x)))
    return out


def dropout_residual(h: Optional[torch.Tensor], branch: torch.Tensor,
                     gate: Optional[torch.Tensor], n_video: Optional[int], p: float,
                     rng: Optional[torch.Tensor], site: int = 0,
                     out: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out = h + gate[b, m] * dropout(branch); h/branch: [B, L, D], gate:
    [B, 2, D] (None for 1; h None for 0).  rng and site as for dropout; no mask
    is stored.  out may be h or branch (in place)."""
    B, L, D, nv = _rows3(branch, n_video, "branch")
    ph = _arg(h, branch.shape, "h", branch)
    pg = _arg(gate, (B, 2, D), "gate", branch)
    po = _arg(out, branch.shape, "out", branch)
    prng = _rng_arg(rng, p, branch)
    dt = _io_dtype(branch)
    with _on(branch, stream):
        if out is None:
            out = torch.empty_like(branch)
            po = out.data_ptr()
        _abi.check(_abi.sol_dropout_residual(ph, branch.data_ptr(), pg, po, prng, site % 2**64,
                                             p, B, L, nv, D, dt, _current(branch)))
    return out


def dropout_residual_backward(dout: torch.Tensor, branch: Optional[torch.Tensor],
                              gate: Optional[torch.Tensor], n_video: Optional[int], p: float,
                              rng: Optional[torch.Tensor], site: int = 0,
                              dbranch: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None,
                              stream: Optional[torch.cuda.Stream] = None
                              ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gradients (dbranch, dgate) of dropout_residual for dout (that of h is
    dout itself), the mask computed again from rng, site and p; dgate is fp32,
    and None without gate (branch may be None then).  p = 0 gives the gradients
    of gate_residual.  dbranch may be dout or branch (in place)."""
    B, L, D, nv = _rows3(dout, n_video, "dout")
    if gate is not None and branch is None:
        raise ValueError("branch is needed for the gradient of gate")
    pb = _arg(branch, dout.shape, "branch", dout)
    pg = _arg(gate, (B, 2, D), "gate", dout)
    pd = _arg(dbranch, dout.shape, "dbranch", dout)
    prng = _rng_arg(rng, p, dout)
    dt = _io_dtype(dout)
    with _on(dout, stream):
        if dbranch is None:
            dbranch = torch.empty_like(dout)
            pd = dbranch.data_ptr()
        dgate = pdg = pw = None
        nw = 0
        if gate is not None:
            dgate = _fp32((B, 2, D), (2 * D, D, 1), dout)
            ws = _workspace(workspace, _abi.sol_dropout_backward_workspace_bytes(B, L, D), dout)
            pdg, pw, nw = dgate.data_ptr(), ws.data_ptr(), ws.nbytes
        _abi.check(_abi.sol_dropout_residual_backward(
            dout.data_ptr(), pb, pg, pd, pdg, prng, site % 2**64, p, B, L, nv, D, pw, nw, dt,
            _current(dout)))
    return dbranch, dgate


class RopeAxes:
    """How the heads of rope_axes are rotated (sol_rope_plan): `sections` gives
    each position axis its number of rotary pairs, in consecutive blocks or,
    with interleaved=True, one pair each in turn; the first
    rot_dim = 2 * sum(sections) channels of a head are rotated.  per_axis_freq
    gives every axis a frequency ladder of its own; half_split pairs channel i
    with i + rot_dim / 2.  Build it once; `desc.freq` may be rescaled."""

    def __init__(self, head_dim: int, sections: Sequence[int], theta: float = 10000.0,
                 per_axis_freq: bool = False, interleaved: bool = False,
                 half_split: bool = False):
        self.head_dim, self.n_axes = head_dim, len(sections)
        self.desc = _abi.RopePlan()
        _abi.check(_abi.sol_rope_plan_init(self.desc, head_dim, 2 * sum(sections),
                                           len(sections), sections, theta,
                                           int(bool(per_axis_freq)), int(bool(interleaved)),
                                           int(bool(half_split))))


_POS = {torch.int32: _abi.SOL_POS_I32, torch.int64: _abi.SOL_POS_I64,
        torch.float32: _abi.SOL_POS_F32}


def _heads(t: Optional[torch.Tensor], B: int, L: int, hd: int, name: str, like: torch.Tensor,
           heads: Optional[int] = None, written: bool = False) -> Optional[_abi.Heads]:
    if t is None:
        return None
    n = t.shape[2] if heads is None and t.dim() == 4 else heads
    if t.shape != (B, L, n, hd) or (hd > 1 and t.stride(3) != 1):
        raise ValueError(f"{name} must be [{B}, {L}, {'heads' if n is None else n}, {hd}] with "
                         f"unit channel stride, got {tuple(t.shape)}, strides {t.stride()}")
    if t.get_device() != like.get_device():
        raise ValueError(f"{name} is on {t.device}, q on {like.device}")
    if t.dtype is not like.dtype:
        raise TypeError(f"all tensors must share one dtype, got {t.dtype} for {name} and "
                        f"{like.dtype}")
    sb, sr, sh, _ = t.stride()
    # the stride of an axis of one element says nothing
    if B == 1:
        sb = 0
    if L == 1:
        sr = 0
    if n == 1:
        sh = 0
    if written and L > 0 and ((sb == 0 and B > 1) or (sr == 0 and L > 1) or (sh == 0 and n > 1)):
        raise ValueError(f"{name} must not be an expanded tensor")
    return _abi.Heads(t.data_ptr(), n, sb, sr, sh)


def _positions(pos: torch.Tensor, B: int, L: int, n_axes: int, like: torch.Tensor):
    kind = _POS.get(pos.dtype)
    if kind is None:
        raise TypeError("pos must be int32, int64 or float32")
    shape = pos.shape
    if (shape != (n_axes, B, L) and shape != (n_axes, L)) or (L > 1 and pos.stride(-1) != 1):
        raise ValueError(f"pos must be [{n_axes}, {B}, {L}] or [{n_axes}, {L}] with unit row "
                         f"stride, got {tuple(pos.shape)}")
    if pos.get_device() != like.get_device():
        raise ValueError(f"pos is on {pos.device}, q on {like.device}")
    s = pos.stride()
    return _abi.Positions(pos.data_ptr(), kind, 0, 0 if n_axes == 1 else s[0],
                          s[1] if len(shape) == 3 and B > 1 else 0)


def _rope_shapes(q, k, plan, what):
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError(f"{what} must be [B, L, heads, head_dim]")
    B, L, H, hd = q.shape
    if hd != plan.head_dim:
        raise ValueError(f"{what} has heads of {hd}, the plan of {plan.head_dim}")
    return B, L, H, hd


def rope_axes(q: torch.Tensor, k: Optional[torch.Tensor], pos: torch.Tensor, plan: RopeAxes,
              gamma_q: Optional[torch.Tensor] = None, gamma_k: Optional[torch.Tensor] = None,
              qk_norm: bool = False, eps: float = 1e-6, q_out: Optional[torch.Tensor] = None,
              k_out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
              ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Rotate q [B, L, Hq, hd] and k [B, L, Hk, hd] (any strides: columns of a
    merged projection, a transposed [B, H, L, hd]; k may be None) at positions
    pos [n_axes, B, L], or [n_axes, L] for all samples (int32, int64 or
    float32), behind a per-head RMS norm with qk_norm=True (gamma_q/gamma_k
    [hd] or None).  Returns (q_out, k_out); pass q_out=q, k_out=k to rotate in
    place."""
    B, L, Hq, hd = _rope_shapes(q, k, plan, "q")
    gq, gk = _arg(gamma_q, (hd,), "gamma_q", q), _arg(gamma_k, (hd,), "gamma_k", q)
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    dt = _io_dtype(q)
    hq, p = _heads(q, B, L, hd, "q", q), _positions(pos, B, L, plan.n_axes, q)
    with _on(q, stream):
        if q_out is None:
            q_out = _packed(q)
        hk = ho = None
        if k is not None:
            hk = _heads(k, B, L, hd, "k", q)
            if k_out is None:
                k_out = _packed(k)
            ho = _heads(k_out, B, L, hd, "k_out", q, k.shape[2], True)
        _abi.check(_abi.sol_rope_axes(plan.desc, p, hq, hk,
                                      _heads(q_out, B, L, hd, "q_out", q, Hq, True), ho, gq, gk,
                                      int(qk_norm), B, L, eps, dt, _current(q)))
    return q_out, k_out


class RopeGrads(NamedTuple):
    """Gradients of rope_axes; None where the input was not given.  dgamma_q and
    dgamma_k are fp32."""
    dq: torch.Tensor
    dk: Optional[torch.Tensor]
    dgamma_q: Optional[torch.Tensor]
    dgamma_k: Optional[torch.Tensor]


def rope_axes_backward(dq_out: torch.Tensor, dk_out: Optional[torch.Tensor], pos: torch.Tensor,
                       plan: RopeAxes, q: Optional[torch.Tensor] = None,
                       k: Optional[torch.Tensor] = None, gamma_q: Optional[torch.Tensor] = None,
                       gamma_k: Optional[torch.Tensor] = None, qk_norm: bool = False,
                       eps: float = 1e-6, dq: Optional[torch.Tensor] = None,
                       dk: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> RopeGrads:
    """Gradients of rope_axes(q, k, pos, plan, gamma_q, gamma_k, qk_norm, eps)
    for (dq_out, dk_out).  q and k are read with qk_norm only.  dq and dk may
    be given with any strides (columns of a merged gradient) and may be dq_out
    and dk_out, or q and k (in place)."""
    g = dq_out
    B, L, Hq, hd = _rope_shapes(g, dk_out, plan, "dq_out")
    gq, gk = _arg(gamma_q, (hd,), "gamma_q", g), _arg(gamma_k, (hd,), "gamma_k", g)
    if qk_norm and (q is None or (k is None) != (dk_out is None)):
        raise ValueError("qk_norm needs q, and k together with dk_out")
    if dk_out is None and dk is not None:
        raise ValueError("dk without dk_out")
    dt = _io_dtype(g)
    p = _positions(pos, B, L, plan.n_axes, g)
    hgq, hgk = _heads(g, B, L, hd, "dq_out", g), _heads(dk_out, B, L, hd, "dk_out", g)
    hq = hk = None
    if qk_norm:
        hq = _heads(q, B, L, hd, "q", g, Hq)
        if k is not None:
            hk = _heads(k, B, L, hd, "k", g, dk_out.shape[2])
    with _on(g, stream):
        if dq is None:
            dq = _packed(g)
        hdk = None
        if dk_out is not None:
            if dk is None:
                dk = _packed(dk_out)
            hdk = _heads(dk, B, L, hd, "dk", g, dk_out.shape[2], True)
        dgq = dgk = pgq = pgk = pw = None
        nw = 0
        if gamma_q is not None:
            dgq = _fp32((hd,), (1,), g)
            pgq = dgq.data_ptr()
        if gamma_k is not None:
            dgk = _fp32((hd,), (1,), g)
            pgk = dgk.data_ptr()
        if pgq or pgk:
            ws = _workspace(workspace, _abi.sol_rope_backward_workspace_bytes(hd), g)
            pw, nw = ws.data_ptr(), ws.nbytes
        _abi.check(_abi.sol_rope_axes_backward(
            plan.desc, p, hgq, hgk, hq, hk, _heads(dq, B, L, hd, "dq", g, Hq, True), hdk, gq, gk,
            pgq, pgk, int(qk_norm), B, L, eps, pw, nw, dt, _current(g)))
    return RopeGrads(dq, dk, dgq, dgk)
