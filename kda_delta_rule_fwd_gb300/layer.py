"""The operators around the recurrence: short causal convolution, selective
state-space scan, and the norms before and after a block with its gate and
residual scale.

Argument marshalling only, as in the package's other entry points; the C ABI is
``include/kda_layer.h``.

    y, state = conv_fwd(x, weight, bias, activation="silu")       # prompts
    y = conv_step(x, weight, state, bias, activation="silu")      # single tokens
    y, hT = scan_fwd(x, dt, A, B, C, D=D, dt_bias=b, dt_softplus=True)
    y = scan_step(x, dt, A, B, C, state, D=D, dt_bias=b, dt_softplus=True)
    r, y = norm_fwd(x, weight=w, gate=g, residual=h, out_weight=w2)

Activations may be views with any token stride (column slices of a fused
projection) as long as the channels of one token are contiguous and one stride
leads from each token to the next, from the last of one sequence to the first of
the following too.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _DT, KDA_OK, KDAError, load

_C = ctypes
_GATES = {"sigmoid": 1, "silu": 2}
_F32 = torch.float32


class ConvShape(_C.Structure):
    """Mirror of ``kda_conv_shape``."""
    _fields_ = [("B", _C.c_int32), ("T", _C.c_int32), ("D", _C.c_int32), ("W", _C.c_int32),
                ("num_seqs", _C.c_int32), ("dtype", _C.c_int), ("silu", _C.c_int32),
                ("ldx", _C.c_int64)]


class ScanShape(_C.Structure):
    """Mirror of ``kda_scan_shape``."""
    _fields_ = [("B", _C.c_int32), ("T", _C.c_int32), ("H", _C.c_int32), ("G", _C.c_int32),
                ("ds", _C.c_int32), ("dx", _C.c_int32), ("num_seqs", _C.c_int32),
                ("in_dtype", _C.c_int), ("out_dtype", _C.c_int), ("dt_softplus", _C.c_int32),
                ("ldx", _C.c_int64), ("lddt", _C.c_int64), ("ldb", _C.c_int64),
                ("ldc", _C.c_int64)]


class NormShape(_C.Structure):
    """Mirror of ``kda_norm_shape``."""
    _fields_ = [("tokens", _C.c_int64), ("heads", _C.c_int32), ("d", _C.c_int32),
                ("dtype", _C.c_int), ("res_dtype", _C.c_int), ("gate", _C.c_int),
                ("gate_first", _C.c_int32), ("scale", _C.c_float), ("eps", _C.c_float),
                ("ldx", _C.c_int64), ("ldgate", _C.c_int64)]


def declare(lib):
    """Argument and result types of the entry points (called once by ``load``)."""
    vp, sz, i32 = _C.c_void_p, _C.c_size_t, _C.c_int
    conv, scan, norm = (_C.POINTER(c) for c in (ConvShape, ScanShape, NormShape))
    for name, res, args in (
            ("kda_conv_fwd", i32, [conv] + [vp] * 8 + [sz, vp]),
            ("kda_conv_step", i32, [conv] + [vp] * 7 + [sz, vp]),
            ("kda_conv_bwd_workspace_size", sz, [conv]),
            ("kda_conv_bwd", i32, [conv] + [vp] * 12 + [sz, vp]),
            ("kda_scan_workspace_size", sz, [scan]),
            ("kda_scan_fwd", i32, [scan] + [vp] * 12 + [sz, vp]),
            ("kda_scan_step", i32, [scan] + [vp] * 11 + [sz, vp]),
            ("kda_norm_fwd", i32, [norm] + [vp] * 9),
            ("kda_norm_bwd_workspace_size", sz, [norm]),
            ("kda_norm_bwd", i32, [norm] + [vp] * 15 + [sz, vp])):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args


# ---------------------------------------------------------------------------
# argument checks.  The smallest calls take about as long here as on the device: every check
# is one comparison when it holds, and the structs are built once per set of sizes.
# ---------------------------------------------------------------------------
def _structs(cls):
    @functools.lru_cache(maxsize=1024)
    def of(*sizes):
        for (name, kind), v in zip(cls._fields_, sizes):
            if kind is _C.c_int32 and v >= 1 << 31:  # ctypes would keep the low bits
                raise ValueError(f"{name} = {v} is more than 2^31 - 1")
        return cls(*sizes)
    return of


_conv_struct, _scan_struct, _norm_struct = (_structs(c) for c in (ConvShape, ScanShape, NormShape))
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                  lambda index: torch.cuda.current_stream(index).cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _new(x, dtype):
    """An output of x's shape (empty_like is the cheaper call where x is dense)."""
    if dtype is x.dtype and x.is_contiguous():
        return torch.empty_like(x)
    return torch.empty(x.shape, dtype=dtype, device=x.device)


def _elsewhere(x, stream):
    """Whether the call has to be made under another device or stream than the current ones."""
    index = x.get_device()  # -1 for a CPU tensor, which _under refuses
    return stream is not None or index < 0 or index != _device()


def _under(x, stream):
    """The tensors' device or, where given, the stream (the buffers allocated under it belong to
    it)."""
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    return torch.cuda.device(x.device) if stream is None else torch.cuda.stream(stream)


def _activation(t, name, x, shape=None):
    """A tensor of x's type, on its device, of ``shape`` (default x's)."""
    if t.dtype is not x.dtype or x.dtype not in _DT:
        raise TypeError(f"{name} must be float32 or bfloat16, the same for all activations")
    if t.get_device() != x.get_device():
        raise ValueError(f"{name} is on another device than x")
    if t.shape != (x.shape if shape is None else shape):
        raise ValueError(f"{name} must have shape {tuple(x.shape if shape is None else shape)}, "
                         f"not {tuple(t.shape)}")


def _dense(t, name, dtype, shape, x):
    """None, or a contiguous tensor of the given type and shape on x's device."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.is_contiguous()
                     and t.get_device() == x.get_device()):
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be a contiguous tensor on {x.device}")


def _uniform(t, lead):
    """The one stride between the rows of the first ``lead`` dimensions when what follows is
    contiguous; None when there is none."""
    inner = 1
    for i in range(t.dim() - 1, lead - 1, -1):
        if t.shape[i] != 1:
            if t.stride(i) != inner:
                return None
            inner *= t.shape[i]
    ld = span = None
    for i in range(lead - 1, -1, -1):
        if t.shape[i] != 1:
            if ld is None:
                ld = span = t.stride(i)
            elif t.stride(i) != span:
                return None
            span *= t.shape[i]
    if ld is None:
        return inner
    return ld if ld >= inner else None


def _token_stride(t, name):
    if t.is_contiguous() or t.numel() == 0:
        return 0
    ld = _uniform(t, 2)
    if ld is None:
        raise ValueError(f"{name} needs contiguous channels and one stride between its tokens")
    return ld


def _seqs(cu_seqlens, B, x):
    """(packed count for the shape, sequences) of a batch."""
    if cu_seqlens is None:
        return 0, B
    if cu_seqlens.dtype is not torch.int32 or not cu_seqlens.is_contiguous() \
            or cu_seqlens.get_device() != x.get_device() or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a contiguous int32 tensor [num_seqs + 1] beside x")
    if B != 1:
        raise ValueError("a packed batch has B = 1")
    n = cu_seqlens.numel() - 1
    return n, n


def _counts(num_commit, B, x):
    if num_commit is not None and (num_commit.dtype is not torch.int32 or num_commit.numel() != B
                                   or not num_commit.is_contiguous()
                                   or num_commit.get_device() != x.get_device()):
        raise ValueError("num_commit must be int32 with one count per sequence, beside x")


def _check(rc, where):
    if rc != KDA_OK:
        raise KDAError(rc, where)


def _ws(workspace, x):
    if workspace is None:
        return None, 0
    if workspace.get_device() != x.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor beside x")
    return workspace.data_ptr(), workspace.nbytes


# ---------------------------------------------------------------------------
# short causal convolution
# ---------------------------------------------------------------------------
def _conv_shape(x, weight, bias, activation, cu_seqlens):
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [B, T, D] and weight [D, W]")
    if activation is not None and activation != "silu":
        raise ValueError("activation must be None or 'silu'")
    if x.dtype not in _DT:
        raise TypeError("x must be float32 or bfloat16")
    B, T, D = x.shape
    W = weight.shape[1]
    _dense(weight, "weight", _F32, (D, W), x)
    _dense(bias, "bias", _F32, (D,), x)
    packed, N = _seqs(cu_seqlens, B, x)
    return _conv_struct(B, T, D, W, packed, _DT[x.dtype], activation is not None,
                        _token_stride(x, "x")), N


def conv_fwd(x, weight, bias=None, *, activation=None, cu_seqlens=None, init_state=None, out=None,
             final_state=None, output_final_state=True, workspace=None, stream=None):
    """Short causal convolution over ``x [B,T,D]`` (packed: ``[1,T,D]`` with int32
    ``cu_seqlens``): ``weight [D,W]`` and ``bias [D]`` float32, W = 2..4, the newest input
    last.  ``init_state [N,W-1,D]`` holds the inputs before the first token (None: zeros).
    Returns ``(y, final_state)``, the state None unless requested."""
    if _elsewhere(x, stream):
        with _under(x, stream):
            return conv_fwd(x, weight, bias, activation=activation, cu_seqlens=cu_seqlens,
                            init_state=init_state, out=out, final_state=final_state,
                            output_final_state=output_final_state, workspace=workspace)
    shape, N = _conv_shape(x, weight, bias, activation, cu_seqlens)
    state = (N, shape.W - 1, shape.D)
    _dense(init_state, "init_state", x.dtype, state, x)
    _dense(out, "out", x.dtype, x.shape, x)
    _dense(final_state, "final_state", x.dtype, state, x)
    if out is None:
        out = _new(x, x.dtype)
    if final_state is None and output_final_state:
        final_state = torch.empty(state, dtype=x.dtype, device=x.device)
    _check(load().kda_conv_fwd(shape, x.data_ptr(), weight.data_ptr(), _ptr(bias),
                               _ptr(cu_seqlens), _ptr(init_state), out.data_ptr(),
                               _ptr(final_state), *_ws(workspace, x), _stream(x.get_device())),
           "kda_conv_fwd")
    return out, final_state


def conv_step(x, weight, state, bias=None, *, activation=None, num_commit=None, out=None,
              want_out=True, workspace=None, stream=None):
    """``conv_fwd`` for 1 to 8 tokens of each of B sequences; ``state [B,W-1,D]`` is updated in
    place.  ``num_commit`` (int32 ``[B]``) keeps the state after each sequence's first
    ``num_commit[n]`` tokens.  Returns ``y [B,T,D]``, or None when ``want_out`` is False (only
    with ``num_commit``)."""
    if _elsewhere(x, stream):
        with _under(x, stream):
            return conv_step(x, weight, state, bias, activation=activation, num_commit=num_commit,
                             out=out, want_out=want_out, workspace=workspace)
    shape, N = _conv_shape(x, weight, bias, activation, None)
    _dense(state, "state", x.dtype, (N, shape.W - 1, shape.D), x)
    _dense(out, "out", x.dtype, x.shape, x)
    _counts(num_commit, N, x)
    if out is None and want_out:
        out = _new(x, x.dtype)
    _check(load().kda_conv_step(shape, x.data_ptr(), weight.data_ptr(), _ptr(bias),
                                _ptr(num_commit), state.data_ptr(), _ptr(out), *_ws(workspace, x),
                                _stream(x.get_device())), "kda_conv_step")
    return out


def conv_bwd(x, weight, dy, bias=None, *, activation=None, cu_seqlens=None, init_state=None,
             dfinal=None, want_dinit=False, workspace=None, stream=None):
    """Gradients of ``sum(y * dy) + sum(final_state * dfinal)`` for ``conv_fwd``'s inputs.
    Returns ``(dx, dweight, dbias, dinit)``: dx and dinit in x's type, the parameters'
    gradients float32; dbias None without a bias, dinit None unless wanted."""
    if _elsewhere(x, stream):
        with _under(x, stream):
            return conv_bwd(x, weight, dy, bias, activation=activation, cu_seqlens=cu_seqlens,
                            init_state=init_state, dfinal=dfinal, want_dinit=want_dinit,
                            workspace=workspace)
    shape, N = _conv_shape(x, weight, bias, activation, cu_seqlens)
    state = (N, shape.W - 1, shape.D)
    _dense(dy, "dy", x.dtype, x.shape, x)
    _dense(init_state, "init_state", x.dtype, state, x)
    _dense(dfinal, "dfinal", x.dtype, state, x)
    lib = load()
    dx = _new(x, x.dtype)
    dw = torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    dinit = torch.empty(state, dtype=x.dtype, device=x.device) if want_dinit else None
    if workspace is None:
        workspace = torch.empty(lib.kda_conv_bwd_workspace_size(shape), dtype=torch.uint8,
                                device=x.device)
    _check(lib.kda_conv_bwd(shape, x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(cu_seqlens),
                            _ptr(init_state), dy.data_ptr(), _ptr(dfinal), dx.data_ptr(),
                            dw.data_ptr(), _ptr(db), _ptr(dinit), *_ws(workspace, x),
                            _stream(x.get_device())), "kda_conv_bwd")
    return dx, dw, db, dinit


# ---------------------------------------------------------------------------
# selective state-space scan
# ---------------------------------------------------------------------------
def _scan_shape(x, dt, A, B, C, D, dt_bias, dt_softplus, cu_seqlens, out_dtype):
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [B, T, H, dx], B and C [B, T, G, ds]")
    if out_dtype not in _DT:
        raise TypeError("the output must be float32 or bfloat16")
    n, T, H, dx = x.shape
    G, ds = B.shape[2:]
    _activation(dt, "dt", x, (n, T, H))
    _activation(B, "B", x, (n, T, G, ds))
    _activation(C, "C", x, (n, T, G, ds))
    _dense(A, "A", _F32, (H,), x)
    _dense(D, "D", _F32, (H,), x)
    _dense(dt_bias, "dt_bias", _F32, (H,), x)
    packed, N = _seqs(cu_seqlens, n, x)
    return _scan_struct(n, T, H, G, ds, dx, packed, _DT[x.dtype], _DT[out_dtype],
                        bool(dt_softplus), _token_stride(x, "x"), _token_stride(dt, "dt"),
                        _token_stride(B, "B"), _token_stride(C, "C")), N


def scan_workspace_size(shape: ScanShape) -> int:
    return int(load().kda_scan_workspace_size(shape))


def scan_fwd(x, dt, A, B, C, *, D=None, dt_bias=None, dt_softplus=False, cu_seqlens=None, h0=None,
             out_dtype=torch.float32, out=None, hT=None, output_final_state=True, workspace=None,
             stream=None):
    """Selective state-space scan over ``x [B,T,H,dx]``, ``dt [B,T,H]`` and ``B, C [B,T,G,ds]``
    (packed: ``[1,T,...]`` with int32 ``cu_seqlens``), with the decay rates ``A [H]`` (<= 0), the
    skip weights ``D [H]`` and ``dt_bias [H]`` in float32.  Returns ``(y, hT)``: ``y [B,T,H,dx]``
    in ``out_dtype`` and the final states ``[N,H,ds,dx]`` float32 (None unless requested)."""
    if _elsewhere(x, stream):
        with _under(x, stream):
            return scan_fwd(x, dt, A, B, C, D=D, dt_bias=dt_bias, dt_softplus=dt_softplus,
                            cu_seqlens=cu_seqlens, h0=h0, out_dtype=out_dtype, out=out, hT=hT,
                            output_final_state=output_final_state, workspace=workspace)
    shape, N = _scan_shape(x, dt, A, B, C, D, dt_bias, dt_softplus, cu_seqlens, out_dtype)
    state = (N, shape.H, shape.ds, shape.dx)
    _dense(h0, "h0", _F32, state, x)
    _dense(out, "out", out_dtype, x.shape, x)
    _dense(hT, "hT", _F32, state, x)
    lib = load()
    if out is None:
        out = _new(x, out_dtype)
    if hT is None and output_final_state:
        hT = torch.empty(state, dtype=_F32, device=x.device)
    if workspace is None:
        workspace = torch.empty(lib.kda_scan_workspace_size(shape), dtype=torch.uint8,
                                device=x.device)
    _check(lib.kda_scan_fwd(shape, x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(),
                            C.data_ptr(), _ptr(D), _ptr(dt_bias), _ptr(cu_seqlens), _ptr(h0),
                            out.data_ptr(), _ptr(hT), *_ws(workspace, x), _stream(x.get_device())),
           "kda_scan_fwd")
    return out, hT


def scan_step(x, dt, A, B, C, state, *, D=None, dt_bias=None, dt_softplus=False, num_commit=None,
              out_dtype=torch.float32, out=None, want_out=True, workspace=None, stream=None):
    """``scan_fwd`` for 1 to 8 tokens of each of B sequences; ``state [B,H,ds,dx]`` float32 is
    updated in place.  ``num_commit`` and ``want_out`` as in :func:`conv_step`."""
    if _elsewhere(x, stream):
        with _under(x, stream):
            return scan_step(x, dt, A, B, C, state, D=D, dt_bias=dt_bias, dt_softplus=dt_softplus,
                             num_commit=num_commit, out_dtype=out_dtype, out=out,
                             want_out=want_out, workspace=workspace)
    shape, N = _scan_shape(x, dt, A, B, C, D, dt_bias, dt_softplus, None, out_dtype)
    _dense(state, "state", _F32, (N, shape.H, shape.ds, shape.dx), x)
    _dense(out, "out", out_dtype, x.shape, x)
    _counts(num_commit, N, x)
    if out is None and want_out:
        out = _new(x, out_dtype)
    _check(load().kda_scan_step(shape, x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(),
                                C.data_ptr(), _ptr(D), _ptr(dt_bias), _ptr(num_commit),
                                state.data_ptr(), _ptr(out), *_ws(workspace, x),
                                _stream(x.get_device())), "kda_scan_step")
    return out


# ---------------------------------------------------------------------------
# norms with gate and residual scale
# ---------------------------------------------------------------------------
def _row_strides(x, gate):
    """(heads, token stride of x, of gate) where one of the two is not contiguous: rows of d
    channels with one stride, or tokens of several rows where only the tokens have one."""
    strided = [t is not None and t.numel() > 0 and not t.is_contiguous() for t in (x, gate)]
    for lead in (x.dim() - 1, x.dim() - 2):
        if lead >= 0:
            lds = [_uniform(t, lead) if s else 0 for s, t in zip(strided, (x, gate))]
            if None not in lds:
                return (1 if lead == x.dim() - 1 else x.shape[-2]), *lds
    raise ValueError("x and gate need contiguous channels and one stride between rows")


def _norm_shape(x, weight, gate, gate_act, gate_first, residual, scale, res_scale, out_weight, eps,
                res_dtype):
    if x.dtype not in _DT:
        raise TypeError("x must be float32 or bfloat16")
    if x.dim() < 1:
        raise ValueError("x must be [..., d]")
    d = x.shape[-1]
    act, heads, ldx, ldg = 0, 1, 0, 0
    if gate is not None:
        _activation(gate, "gate", x)
        act = _GATES.get(gate_act, 0)
        if not act:
            raise ValueError("gate_act must be 'sigmoid' or 'silu'")
    _dense(weight, "weight", _F32, (d,), x)
    _dense(res_scale, "res_scale", _F32, (d,), x)
    _dense(out_weight, "out_weight", _F32, (d,), x)
    if res_dtype is None:
        res_dtype = x.dtype if residual is None else residual.dtype
    if res_dtype is not x.dtype and res_dtype is not _F32:
        raise TypeError("the residual must be of x's type or float32")
    _dense(residual, "residual", res_dtype, x.shape, x)
    if not (x.is_contiguous() and (gate is None or gate.is_contiguous())):
        heads, ldx, ldg = _row_strides(x, gate)
    tokens = x.numel() // (heads * d) if d else 0
    return _norm_struct(tokens, heads, d, _DT[x.dtype], _DT[res_dtype], act, bool(gate_first),
                        float(scale), float(eps), ldx, ldg), res_dtype


def norm_fwd(x, *, weight=None, gate=None, gate_act="sigmoid", gate_first=False, residual=None,
             scale=1.0, res_scale=None, out_weight=None, eps=1e-6, res_dtype=None, r=None, y=None,
             want_r=True, stream=None):
    """Norms around a block: with ``z = act(gate)``, ``m = rms(x) * weight * z`` (``gate_first``:
    ``rms(x * z) * weight``; no norm without ``weight``), ``r = residual + scale * res_scale * m``
    and ``y = rms(r) * out_weight``.  Rows are the last dimension; ``weight``, ``res_scale`` and
    ``out_weight`` are float32 ``[d]``; the residual is of x's type or float32.  Returns
    ``(r, y)``: r in the residual's type (None unless wanted; it may be the residual's own
    buffer), y in x's type (None without ``out_weight``)."""
    if _elsewhere(x, stream):
        with _under(x, stream):
            return norm_fwd(x, weight=weight, gate=gate, gate_act=gate_act, gate_first=gate_first,
                            residual=residual, scale=scale, res_scale=res_scale,
                            out_weight=out_weight, eps=eps, res_dtype=res_dtype, r=r, y=y,
                            want_r=want_r)
    shape, res_dtype = _norm_shape(x, weight, gate, gate_act, gate_first, residual, scale,
                                   res_scale, out_weight, eps, res_dtype)
    _dense(r, "r", res_dtype, x.shape, x)
    _dense(y, "y", x.dtype, x.shape, x)
    if r is None and want_r:
        r = _new(x, res_dtype)
    if y is None and out_weight is not None:
        y = _new(x, x.dtype)
    _check(load().kda_norm_fwd(shape, x.data_ptr(), _ptr(weight), _ptr(gate), _ptr(residual),
                               _ptr(res_scale), _ptr(out_weight), _ptr(r), _ptr(y),
                               _stream(x.get_device())), "kda_norm_fwd")
    return r, y


def norm_bwd(x, dr, dy=None, *, weight=None, gate=None, gate_act="sigmoid", gate_first=False,
             residual=None, scale=1.0, res_scale=None, out_weight=None, eps=1e-6, res_dtype=None,
             workspace=None, stream=None):
    """Gradients of ``sum(r * dr) + sum(y * dy)`` for ``norm_fwd``'s inputs (``dr`` or ``dy`` may
    be None).  Returns ``(dx, dgate, dresidual, dweight, dres_scale, dout_weight)``, each None
    where its operand is; the parameters' gradients are float32."""
    if _elsewhere(x, stream):
        with _under(x, stream):
            return norm_bwd(x, dr, dy, weight=weight, gate=gate, gate_act=gate_act,
                            gate_first=gate_first, residual=residual, scale=scale,
                            res_scale=res_scale, out_weight=out_weight, eps=eps,
                            res_dtype=res_dtype, workspace=workspace)
    if res_dtype is None and residual is None and dr is not None:
        res_dtype = dr.dtype
    shape, res_dtype = _norm_shape(x, weight, gate, gate_act, gate_first, residual, scale,
                                   res_scale, out_weight, eps, res_dtype)
    _dense(dr, "dr", res_dtype, x.shape, x)
    _dense(dy, "dy", x.dtype, x.shape, x)
    lib = load()
    new = lambda t: None if t is None else _new(t, t.dtype)
    dx, dgate, dres = new(x), new(gate), new(residual)
    dw, dls, dow = new(weight), new(res_scale), new(out_weight)
    if workspace is None:
        workspace = torch.empty(lib.kda_norm_bwd_workspace_size(shape), dtype=torch.uint8,
                                device=x.device)
    _check(lib.kda_norm_bwd(shape, x.data_ptr(), _ptr(weight), _ptr(gate), _ptr(residual),
                            _ptr(res_scale), _ptr(out_weight), _ptr(dr), _ptr(dy), dx.data_ptr(),
                            _ptr(dgate), _ptr(dres), _ptr(dw), _ptr(dls), _ptr(dow),
                            *_ws(workspace, x), _stream(x.get_device())), "kda_norm_bwd")
    return dx, dgate, dres, dw, dls, dow
