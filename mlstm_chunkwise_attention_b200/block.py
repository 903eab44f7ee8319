"""The operators around the recurrence, for torch tensors (``include/mlstm_block.h``).

* ``causal_conv_forward`` / ``_backward`` / ``_step``: the short causal convolution before the
  cell or the scan;
* ``selective_scan_forward`` / ``_backward`` / ``_step``: the selective state space scan;
* ``group_norm_forward`` / ``_backward``: group norm with an activation or an output gate, after
  the cell (statistics per token and head) or over a whole sequence.

Like ``binding``, these functions allocate through PyTorch and call the CUDA library, which does
all of the computation.  Activations are bfloat16 or float32, channels last ([B, T, D], any batch
and token strides) or head-major ([B, NH, T, d], as the cell takes and returns them); parameters,
their gradients and the scan's states are float32.  Work is enqueued on the current stream of the
tensors' device, or on ``stream``: outputs and workspaces are then allocated for that stream.
"""

import struct

import torch

from .binding import (
    BF16, FP32, STATUS_OK, STATUS_UNSUPPORTED, MLSTMError, Rows, ScanGrads, ScanProblem, load)

ACT_NONE = 0
ACT_SILU = 1
ACT_SIGMOID = 2
SCOPE_TOKEN = 0
SCOPE_SEQUENCE = 1


# --------------------------------------------------------------------------
# argument checks and plumbing
# --------------------------------------------------------------------------

def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return FP32
    raise TypeError(f"unsupported dtype {t.dtype}: use bfloat16 or float32")


# The checks run on every call, of which a small one takes 15 us.  So they ask each tensor for as
# little as they can (get_device() is -1 off the GPU), in line where a call has many tensors, and
# leave what is not plainly right to _activation and _fp32, and the wording to _refuse.
_FP32 = torch.float32


def _activation(name, t, shape, like):
    """An activation of `like`'s dtype and device, last dimension contiguous, of this shape."""
    if not (t.shape == shape and t.dtype == like.dtype and t.get_device() == like.get_device()
            and (t.is_contiguous() or t.stride(-1) == 1 or shape[-1] <= 1) and t.is_cuda):
        _refuse(name, t, shape, like, like.dtype, "contiguous in its last dimension")


def _fp32(name, t, shape, like):
    """A contiguous float32 parameter or state (None passes)."""
    if t is not None and not (t.shape == shape and t.dtype == _FP32 and t.is_contiguous()
                              and t.get_device() == like.get_device()):
        _refuse(name, t, shape, like, _FP32, "contiguous")


def _refuse(name, t, shape, like, dtype, layout):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, expected {like.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {str(dtype).removeprefix('torch.')}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be {layout}")


def _contiguous(name, t, shape, like):
    if t is None:
        return
    _activation(name, t, shape, like)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _dims(name, t, n):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got shape {tuple(t.shape)}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rows(t):
    """[B, T, D] (or [B, D], one token) as mlstm_rows_t."""
    if t is None:
        return Rows(None, 0, 0, 0)
    st = t.stride()
    return Rows(t.data_ptr(), st[0], st[1] if len(st) == 3 else 0, 0)


def _head_rows(t, layout, d):
    """A tensor by heads: [B, NH, T, d] ("heads") or [B, T, NH d] ("last")."""
    if t is None:
        return Rows(None, 0, 0, 0)
    sb, s1, s2 = t.stride()[:3]
    return Rows(t.data_ptr(), sb, s2, s1) if layout == "heads" else Rows(t.data_ptr(), sb, s1, d)


def _on(stream, like, tensors, launch):
    """launch(stream handle), with `like`'s device current.  With an explicit stream, what launch
    allocates belongs to that stream, and the inputs are kept from reuse until its work is done."""
    device = like.get_device()
    if stream is None and device == torch.cuda.current_device():
        # the handle of torch.cuda.current_stream() without building a Stream (3 us of a 15 us call)
        return launch(torch._C._cuda_getCurrentRawStream(device))
    if stream is not None and stream.device != like.device:
        raise ValueError(f"stream is on {stream.device}, tensors on {like.device}")
    with torch.cuda.device(device):
        if stream is None:
            return launch(torch._C._cuda_getCurrentRawStream(device))
        with torch.cuda.stream(stream):
            for t in (like, *tensors):
                if t is not None:
                    t.record_stream(stream)
            return launch(stream.cuda_stream)


def _check(status, where):
    if status != STATUS_OK:
        raise MLSTMError(status, where)


def _like(t):
    """A contiguous tensor like t (None for None)."""
    if t is None:
        return None
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _bytes(n, like):
    return like.new_empty(max(n, 16), dtype=torch.uint8)


# --------------------------------------------------------------------------
# short causal convolution
# --------------------------------------------------------------------------

def _conv_args(x, weight, bias, state, act, tokens):
    _activation("x", x, x.shape, x)
    D = x.shape[-1]
    _dims("weight", weight, 2)
    W = weight.shape[1]
    _fp32("weight", weight, (D, W), x)
    _fp32("bias", bias, (D,), x)
    _contiguous("state", state, (x.shape[0], W - 1, D), x)
    if act not in (ACT_NONE, ACT_SILU):
        raise ValueError("act must be ACT_NONE or ACT_SILU")
    if not 2 <= W <= 4:
        raise MLSTMError(STATUS_UNSUPPORTED, f"causal convolution of {W} taps")
    return x.shape[0], tokens, D, W, _dtype_code(x)


def _heads_of(D, heads):
    if heads is None:
        return 1, D
    if heads <= 0 or D % heads:
        raise ValueError(f"{heads} heads do not divide {D} channels")
    return heads, D // heads


def causal_conv_forward(x, weight, bias=None, *, act=ACT_SILU, state_in=None, want_state=False,
                        heads=None, stream=None):
    """y = act(bias + causal convolution of x) per channel; returns (y, state_out).

    x [B, T, D]; weight [D, W] with 2 to 4 taps, the last one on the current token; state_in
    [B, W - 1, D]: the inputs before the first token (None: zeros).  y is [B, T, D], or with
    ``heads`` head-major, [B, heads, T, D / heads].  state_out: the last W - 1 inputs, for a later
    call or ``causal_conv_step`` (None unless want_state).
    """
    _dims("x", x, 3)
    B, T, D, W, dt = _conv_args(x, weight, bias, state_in, act, x.shape[1])
    NH, d = _heads_of(D, heads)

    def launch(s):
        y = _like(x) if heads is None else x.new_empty((B, NH, T, d))
        state_out = None
        if want_state:
            state_out = _like(state_in) if state_in is not None else x.new_empty((B, W - 1, D))
        _check(load().mlstm_conv_fwd(_rows(x), weight.data_ptr(), _ptr(bias), _ptr(state_in),
                                     _head_rows(y, "last" if heads is None else "heads", d),
                                     _ptr(state_out), B, T, NH, d, W, act, dt, s), "mlstm_conv_fwd")
        return y, state_out

    return _on(stream, x, (weight, bias, state_in), launch)


def causal_conv_backward(x, weight, bias, dy, *, act=ACT_SILU, state_in=None, dstate_out=None,
                         want_dstate=False, stream=None):
    """Gradients of sum(dy y) + sum(dstate_out state_out): dict of dx [B, T, D], dweight, dbias
    (None without a bias) and dstate_in (None unless want_dstate).  dy is laid out like the
    forward's y: [B, T, D], or head-major [B, NH, T, d]."""
    _dims("x", x, 3)
    B, T, D, W, dt = _conv_args(x, weight, bias, state_in, act, x.shape[1])
    NH, d, layout = 1, D, "last"
    if dy.dim() == 4:
        NH, d = _heads_of(D, dy.shape[1])
        layout = "heads"
    _activation("dy", dy, (B, NH, T, d) if layout == "heads" else (B, T, D), x)
    _contiguous("dstate_out", dstate_out, (B, W - 1, D), x)

    def launch(s):
        out = {"dx": _like(x), "dweight": _like(weight), "dbias": _like(bias),
               "dstate_in": x.new_empty((B, W - 1, D)) if want_dstate else None}
        ws = _bytes(load().mlstm_conv_bwd_workspace_size(B, T, NH, d, W, dt), x)
        _check(load().mlstm_conv_bwd(_rows(x), weight.data_ptr(), _ptr(bias), _ptr(state_in),
                                     _head_rows(dy, layout, d), _ptr(dstate_out), _rows(out["dx"]),
                                     out["dweight"].data_ptr(), _ptr(out["dbias"]),
                                     _ptr(out["dstate_in"]), ws.data_ptr(), ws.numel(), B, T, NH, d, W,
                                     act, dt, s), "mlstm_conv_bwd")
        return out

    return _on(stream, x, (weight, bias, state_in, dy, dstate_out), launch)


def causal_conv_step(x, weight, bias, state, *, act=ACT_SILU, heads=None, stream=None):
    """One token: x [B, D]; returns y [B, D] (with ``heads``: [B, heads, D / heads]) and updates
    ``state`` [B, W - 1, D] in place."""
    _dims("x", x, 2)
    if state is None:
        raise ValueError("state is required")
    B, _, D, W, dt = _conv_args(x, weight, bias, state, act, 1)
    NH, d = _heads_of(D, heads)

    def launch(s):
        y = _like(x) if heads is None else x.new_empty((B, NH, d))
        at = state.data_ptr()
        _check(load().mlstm_conv_step(_rows(x), weight.data_ptr(), _ptr(bias), at,
                                      Rows(y.data_ptr(), D, 0, d), at, B, NH, d, W, act, dt, s),
               "mlstm_conv_step")
        return y

    return _on(stream, x, (weight, bias, state), launch)


# --------------------------------------------------------------------------
# selective state space scan
# --------------------------------------------------------------------------

#: mlstm_scan_t: five mlstm_rows_t, four pointers, seven ints (packed at once: a field at a time
#: costs five times as long)
_SCAN_PROBLEM = struct.Struct("@20q4q7i4x")


def _scan_problem(x, dt, A, Bm, Cm, skip, z, dt_bias, softplus, state):
    """mlstm_scan_t of a call on [B, T, D] tensors (or [B, D]: one token)."""
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    _activation("x", x, shape, x)
    D = shape[-1]
    if dt.shape != shape or dt.dtype != dtype or dt.get_device() != dev or not dt.is_contiguous():
        _activation("dt", dt, shape, x)
    if z is not None and (z.shape != shape or z.dtype != dtype or z.get_device() != dev
                          or not z.is_contiguous()):
        _activation("z", z, shape, x)
    if A.dim() != 2:
        _dims("A", A, 2)
    N = A.shape[1]
    _fp32("A", A, (D, N), x)
    for name, t in (("skip", skip), ("dt_bias", dt_bias)):
        if t is not None and (t.shape != (D,) or t.dtype != _FP32 or t.get_device() != dev
                              or not t.is_contiguous()):
            _fp32(name, t, (D,), x)
    G, grouped = 1, Bm.dim() > len(shape)
    if grouped:
        G = Bm.shape[-2]
        if G <= 0 or D % G:
            raise ValueError(f"{G} groups do not divide {D} channels")
    per = (*shape[:-1], G, N) if grouped else (*shape[:-1], N)
    bs, cs = Bm.stride(), Cm.stride()
    if Bm.shape != per or Bm.dtype != dtype or Bm.get_device() != dev or bs[-1] != 1:
        _activation("B", Bm, per, x)
    if Cm.shape != per or Cm.dtype != dtype or Cm.get_device() != dev or cs[-1] != 1:
        _activation("C", Cm, per, x)
    _fp32("state", state, (shape[0], D, N), x)
    xs, ds = x.stride(), dt.stride()
    zp, zs = (0, xs) if z is None else (z.data_ptr(), z.stride())
    if len(xs) == 3:
        T, xt, dtt, zt, bt, ct = shape[1], xs[1], ds[1], zs[1], bs[1], cs[1]
    else:
        T, xt, dtt, zt, bt, ct = 1, 0, 0, 0, 0, 0
    bg, cg = (bs[-2], cs[-2]) if grouped else (0, 0)
    return ScanProblem.from_buffer_copy(_SCAN_PROBLEM.pack(
        x.data_ptr(), xs[0], xt, 0, dt.data_ptr(), ds[0], dtt, 0, zp, zs[0], zt, 0,
        Bm.data_ptr(), bs[0], bt, bg, Cm.data_ptr(), cs[0], ct, cg, A.data_ptr(),
        0 if skip is None else skip.data_ptr(), 0 if dt_bias is None else dt_bias.data_ptr(),
        0 if state is None else state.data_ptr(), shape[0], T, D, G, N, 1 if softplus else 0,
        _dtype_code(x)))


def selective_scan_forward(x, dt, A, B, C, *, skip=None, z=None, dt_bias=None, softplus=True,
                           state_in=None, keep_saved=True, want_state=False, stream=None):
    """y = (sum_n C[n] s[n] + skip x) silu(z) with s[n] <- exp(delta A[n]) s[n] + delta x B[n] and
    delta = softplus(dt + dt_bias); returns (y, saved, state_out).

    x, dt, z [B, T, D]; A [D, N], up to 64 states; B, C [B, T, N], or [B, T, G, N] where each of G
    groups of D / G channels has its own; skip, dt_bias [D]; state_in [B, D, N] (None: zeros).
    ``saved`` is what the backward needs (None unless keep_saved); state_out [B, D, N] is None
    unless want_state.
    """
    _dims("x", x, 3)
    p = _scan_problem(x, dt, A, B, C, skip, z, dt_bias, softplus, state_in)

    def launch(s):
        y = _like(x)
        saved = (_bytes(load().mlstm_scan_saved_size(p.B, p.T, p.D, p.G, p.N, p.dtype), x)
                 if keep_saved else None)
        state_out = x.new_empty((p.B, p.D, p.N), dtype=torch.float32) if want_state else None
        need = load().mlstm_scan_fwd_workspace_size(p.B, p.T, p.D, p.G, p.N, p.dtype)
        ws = _bytes(need, x) if need else None
        _check(load().mlstm_scan_fwd(p, _rows(y), _ptr(saved), _ptr(state_out), _ptr(ws), need, s),
               "mlstm_scan_fwd")
        return y, saved, state_out

    return _on(stream, x, (dt, A, B, C, skip, z, dt_bias, state_in), launch)


def selective_scan_backward(x, dt, A, B, C, dy, saved, *, skip=None, z=None, dt_bias=None,
                            softplus=True, state_in=None, dstate_out=None, want_dstate=False,
                            stream=None):
    """Gradients of sum(dy y) + sum(dstate_out state_out): dict of dx, ddt, dA, dB, dC, dskip,
    ddt_bias, dz and dstate_in (None where the input was not given, or not want_dstate)."""
    _dims("x", x, 3)
    p = _scan_problem(x, dt, A, B, C, skip, z, dt_bias, softplus, state_in)
    _activation("dy", dy, x.shape, x)
    _fp32("dstate_out", dstate_out, (p.B, p.D, p.N), x)
    need = load().mlstm_scan_saved_size(p.B, p.T, p.D, p.G, p.N, p.dtype)
    if (saved is None or saved.device != x.device or not saved.is_contiguous()
            or saved.numel() * saved.element_size() < need):
        raise ValueError(f"saved must hold the {need} bytes of the forward of the same inputs, contiguous")

    def launch(s):
        out = {"dx": _like(x), "ddt": _like(x), "dA": _like(A), "dB": _like(B), "dC": _like(C),
               "dskip": _like(skip), "ddt_bias": _like(dt_bias), "dz": _like(z),
               "dstate_in": A.new_empty((p.B, p.D, p.N)) if want_dstate else None}
        g = ScanGrads(_rows(out["dx"]), _rows(out["ddt"]), _rows(out["dz"]), _group_rows(out["dB"]),
                      _group_rows(out["dC"]), _ptr(out["dA"]), _ptr(out["dskip"]),
                      _ptr(out["ddt_bias"]), _ptr(out["dstate_in"]))
        ws = _bytes(load().mlstm_scan_bwd_workspace_size(p.B, p.T, p.D, p.G, p.N, p.dtype), x)
        _check(load().mlstm_scan_bwd(p, _rows(dy), saved.data_ptr(), _ptr(dstate_out), g, ws.data_ptr(),
                                     ws.numel(), s), "mlstm_scan_bwd")
        return out

    return _on(stream, x, (dt, A, B, C, skip, z, dt_bias, state_in, dy, saved, dstate_out), launch)


def _group_rows(t):
    """The gradient of B or C: [B, T, N] or [B, T, G, N]."""
    return Rows(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2) if t.dim() == 4 else 0)


def selective_scan_step(x, dt, A, B, C, state, *, skip=None, z=None, dt_bias=None, softplus=True,
                        stream=None):
    """One token: x, dt, z [B, D]; B, C [B, N] or [B, G, N]; returns y [B, D] and updates ``state``
    [B, D, N] in place."""
    _dims("x", x, 2)
    if state is None:
        raise ValueError("state is required")
    p = _scan_problem(x, dt, A, B, C, skip, z, dt_bias, softplus, state)

    def launch(s):
        y = _like(x)
        _check(load().mlstm_scan_step(p, _rows(y), state.data_ptr(), s), "mlstm_scan_step")
        return y

    return _on(stream, x, (dt, A, B, C, skip, z, dt_bias, state), launch)


# --------------------------------------------------------------------------
# group norm with an activation or an output gate
# --------------------------------------------------------------------------

def _norm_args(x, weight, bias, gate, act, scope, groups):
    """(layout of x, B, T, NH, d) of a group norm call."""
    if x.dim() == 4:
        B, NH, T, d = x.shape
        if groups is not None and groups != NH:
            raise ValueError(f"x has {NH} heads, groups is {groups}")
        layout = "heads"
    else:
        _dims("x", x, 3)
        B, T, D = x.shape
        if groups is None or groups <= 0 or D % groups:
            raise ValueError(f"{groups} groups do not divide {D} channels")
        NH, d = groups, D // groups
        layout = "last"
    D, dev = NH * d, x.get_device()
    _activation("x", x, x.shape, x)
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None and (t.shape != (D,) or t.dtype != _FP32 or t.get_device() != dev
                              or not t.is_contiguous()):
            _fp32(name, t, (D,), x)
    if gate is not None and (gate.shape != (B, T, D) or gate.dtype != x.dtype
                             or gate.get_device() != dev or not gate.is_contiguous()):
        _activation("gate", gate, (B, T, D), x)
    if act not in (ACT_NONE, ACT_SILU, ACT_SIGMOID):
        raise ValueError("act must be ACT_NONE, ACT_SILU or ACT_SIGMOID")
    if scope not in (SCOPE_TOKEN, SCOPE_SEQUENCE):
        raise ValueError("scope must be SCOPE_TOKEN or SCOPE_SEQUENCE")
    return layout, B, T, NH, d, _dtype_code(x)


def _stats_shape(B, T, NH, scope):
    return (B, T, NH, 2) if scope == SCOPE_TOKEN else (B, NH, 2)


def group_norm_forward(x, weight=None, bias=None, *, gate=None, act=ACT_NONE, scope=SCOPE_TOKEN,
                       groups=None, eps=1e-5, keep_stats=True, stream=None):
    """Group norm, then the activation (or, with ``gate``, times the gate's activation).

    x is head-major [B, NH, T, d], as the cell returns it (a group per head), or [B, T, C] with
    ``groups``; weight, bias [NH d] or None; gate [B, T, NH d].  The mean and variance are over the d
    channels of each token and group (SCOPE_TOKEN, d <= 512) or over all T tokens of the group
    (SCOPE_SEQUENCE).  Returns (y [B, T, NH d], stats): stats are what the backward needs (None
    unless keep_stats).
    """
    layout, B, T, NH, d, dt = _norm_args(x, weight, bias, gate, act, scope, groups)

    def launch(s):
        y = x.new_empty((B, T, NH * d))
        stats = (x.new_empty(_stats_shape(B, T, NH, scope), dtype=torch.float32) if keep_stats
                 else None)
        need, ws = 0, None  # a forward per token needs none
        if scope == SCOPE_SEQUENCE:
            need = load().mlstm_group_norm_workspace_size(B, T, NH, d, scope, dt, 0)
            ws = _bytes(need, x) if need else None
        _check(load().mlstm_group_norm_fwd(_head_rows(x, layout, d), _ptr(weight), _ptr(bias),
                                           _head_rows(gate, "last", d), _head_rows(y, "last", d),
                                           _ptr(stats), _ptr(ws), need, B, T, NH, d, scope, act, eps,
                                           dt, s), "mlstm_group_norm_fwd")
        return y, stats

    return _on(stream, x, (weight, bias, gate), launch)


def group_norm_backward(x, weight, bias, dy, stats, *, gate=None, act=ACT_NONE, scope=SCOPE_TOKEN,
                        groups=None, stream=None):
    """Gradients of sum(dy y): dict of dx (laid out like x), dweight, dbias and dgate (None where
    the input was not given)."""
    layout, B, T, NH, d, dt = _norm_args(x, weight, bias, gate, act, scope, groups)
    _activation("dy", dy, (B, T, NH * d), x)
    if stats is None:
        raise ValueError("stats of the forward are required")
    _fp32("stats", stats, _stats_shape(B, T, NH, scope), x)

    def launch(s):
        out = {"dx": _like(x), "dweight": _like(weight), "dbias": _like(bias), "dgate": _like(gate)}
        need = load().mlstm_group_norm_workspace_size(B, T, NH, d, scope, dt, 1)
        ws = _bytes(need, x) if need else None
        _check(load().mlstm_group_norm_bwd(_head_rows(x, layout, d), _ptr(weight), _ptr(bias),
                                           _head_rows(gate, "last", d), _head_rows(dy, "last", d),
                                           stats.data_ptr(), _head_rows(out["dx"], layout, d),
                                           _head_rows(out["dgate"], "last", d), _ptr(out["dweight"]),
                                           _ptr(out["dbias"]), _ptr(ws), need, B, T, NH, d, scope, act,
                                           dt, s), "mlstm_group_norm_bwd")
        return out

    return _on(stream, x, (weight, bias, gate, dy, stats), launch)
