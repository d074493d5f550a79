"""The operators a recurrent layer runs around its scan, on torch CUDA tensors:
short causal convolution, selective state space scan, rotary positions, and the
single-token steps (layouts and rules of ``include/gdn.h``).

Argument checks and marshalling only, as in the package's other calls; imported
by the package, whose names these are.  Every call takes ``stream`` (a
``torch.cuda.Stream``; the current one of the tensors' device by default).
Prompts come as equal sequences ([B, T, ...]) or packed ([T, ...] with
``seq_offsets`` [B + 1] int32); operands may be strided views whose last
dimension is contiguous (the halves of one projection, say).
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence, Tuple

import torch

import gated_delta_rule_scan_amd as _g

_F32 = torch.float32
_byref = ctypes.byref
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
_TYPES = {torch.bfloat16: _g.GDN_DTYPE_BF16, torch.float32: _g.GDN_DTYPE_F32}


def _type(x, name: str) -> int:
    kind = _TYPES.get(x.dtype)
    if kind is None:
        raise TypeError(f"{name} must be float32 or bfloat16")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return kind


def _param(t, shape: tuple, like, name: str, dtype=_F32) -> Optional[int]:
    """Address of an optional contiguous parameter of the given shape and type."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != like.device:
        raise ValueError(f"{name} must be contiguous {str(dtype)[6:]} {list(shape)} on {like.device}")
    return t.data_ptr()


def _rows(t, shape, dtype, dev, name: str) -> None:
    """Checks that t is rows of the given shape, type and device whose last dimension is contiguous."""
    if t.shape == shape and t.dtype is dtype and t.device == dev and t.stride(-1) == 1:
        return
    if t.shape != shape or t.dtype is not dtype or t.device != dev:
        raise ValueError(f"{name} must be {str(dtype)[6:]} {list(shape)} on {dev}")
    if t.shape[-1] != 1 and t.numel():
        raise ValueError(f"{name}: the last dimension must be contiguous")


def _lead(x, offsets) -> tuple:
    """(sequences, tokens): x is [B, T, D], or [T, D] with offsets."""
    if offsets is None:
        if x.dim() != 3:
            raise ValueError("x must be [B, T, D] (or [T, D] with seq_offsets)")
        return x.shape[0], x.shape[1]
    if x.dim() != 2:
        raise ValueError("x must be [T, D] with seq_offsets")
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.shape[0] < 2 or not offsets.is_contiguous() \
            or offsets.device != x.device:
        raise ValueError(f"seq_offsets must be contiguous int32 [B + 1] on {x.device}")
    return offsets.shape[0] - 1, x.shape[0]


def _strides(t, packed: bool) -> tuple:
    """(sequence stride, token stride) of rows."""
    return (0, t.stride(0)) if packed else (t.stride(0), t.stride(1))


def _states(B, tail: tuple, dtype, x, state_in, state_out, index, want) -> tuple:
    """Checks the state buffers of a prompt and allocates a final state if one is wanted; (slots, state_out)."""
    _param(index, (B,), x, "state_index", torch.int32)
    slots = B
    given = state_in if state_in is not None else state_out
    if given is not None:
        slots = given.shape[0]
        if index is None and slots != B:
            raise ValueError(f"a state of {slots} slots needs state_index for {B} sequences")
    for t, name in ((state_in, "state_in"), (state_out, "state_out")):
        _param(t, (slots,) + tail, x, name, dtype)
    if state_out is None and want:
        if index is not None:
            raise ValueError("state_out must be given with state_index (or want_state=False)")
        state_out = torch.empty((B,) + tail, dtype=dtype, device=x.device)
    return slots, state_out


def _call(fn, problem, device, stream, made, *pointers) -> None:
    """One library call on `device`; `made`: tensors allocated here, which work on another stream than the
    current one keeps alive."""
    index = device.index
    current = _raw_stream(index)
    if stream is None:
        problem.stream = current or None
    else:
        if stream.device != device:
            raise ValueError(f"stream must be one of {device}")
        problem.stream = stream.cuda_stream or None
        if stream.cuda_stream != current:
            for t in made:
                t.record_stream(stream)
    if _current_device() == index:
        st = fn(_byref(problem), *pointers)
    else:
        with torch.cuda.device(device):
            st = fn(_byref(problem), *pointers)
    if st:
        raise _g.GdnError(st)


def _output(out, like, name="out"):
    """(out, made): a new contiguous tensor like `like`, or the caller's, checked."""
    if out is None:
        out = torch.empty_like(like, memory_format=torch.contiguous_format)
        return out, (out,)
    if out.dtype != like.dtype or out.shape != like.shape or out.device != like.device:
        raise ValueError(f"{name} must be {str(like.dtype)[6:]} {list(like.shape)} on {like.device}")
    if out.shape[-1] != 1 and out.stride(-1) != 1 and out.numel():
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return out, ()


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def causal_conv(x, weight, bias=None, state_in=None, activation: str = "silu", seq_offsets=None, state_index=None,
                out=None, state_out=None, want_state: bool = True, stream=None) -> Tuple:
    """Short causal depthwise convolution over time, y[t] = act(bias + sum_j weight[:, j] x[t - (W - 1) + j]).

    x [B, T, D], or [T, D] packed with ``seq_offsets``; weight [D, W] float32, W in 2..4; bias [D] float32 or None;
    ``activation`` "silu" or "none".  ``state_in`` [slots, W - 1, D] (the type of x) holds the W - 1 rows before each
    sequence (None: zeros), ``state_out`` receives the last W - 1 and may be ``state_in``; sequence b uses slot
    ``state_index[b]`` (None: slot b; out of range: no state).
    Returns (out like x, state_out or None)."""
    dt = _type(x, "x")
    B, T = _lead(x, seq_offsets)
    D, W = x.shape[-1], weight.shape[-1]
    _rows(x, x.shape, x.dtype, x.device, "x")
    if activation not in _g.ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(_g.ACTIVATIONS)}")
    w, b = _param(weight, (D, W), x, "weight"), _param(bias, (D,), x, "bias")
    slots, new_state = _states(B, (W - 1, D), x.dtype, x, state_in, state_out, state_index, want_state)
    out, made = _output(out, x)
    packed = seq_offsets is not None
    problem = _g.gdn_conv_problem_t(B, T, D, *_strides(x, packed), *_strides(out, packed), slots, dt, W,
                                    _g.ACTIVATIONS[activation], _ptr(seq_offsets), _ptr(state_index))
    if state_out is None and new_state is not None:
        made += (new_state,)
    _call(_g.lib().gdn_conv_forward, problem, x.device, stream, made, x.data_ptr(), w, b, _ptr(state_in), _ptr(new_state),
          out.data_ptr())
    return out, new_state


def causal_conv_step(x, weight, bias=None, state=None, activation: str = "silu", state_index=None, out=None,
                     stream=None):
    """The convolution of one new token per sequence: x [B, D]; ``state`` [slots, W - 1, D] is read and advanced in
    place.  A row whose ``state_index`` is out of range is skipped: its output row and every state stay as they
    were.  Returns out [B, D]."""
    dt = _type(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [B, D]")
    B, D = x.shape
    W = weight.shape[-1]
    _rows(x, x.shape, x.dtype, x.device, "x")
    if activation not in _g.ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(_g.ACTIVATIONS)}")
    w, b = _param(weight, (D, W), x, "weight"), _param(bias, (D,), x, "bias")
    slots, ps, pi = _step_state(state, (W - 1, D), x.dtype, x.device, state_index, B)
    out, made = _output(out, x)
    problem = _g.gdn_conv_problem_t(B, 1, D, x.stride(0), 0, out.stride(0), 0, slots, dt, W,
                                    _g.ACTIVATIONS[activation], None, pi)
    _call(_g.lib().gdn_conv_step, problem, x.device, stream, made, x.data_ptr(), w, b, ps, out.data_ptr())
    return out


def _step_state(state, tail: tuple, dtype, dev, index, B) -> tuple:
    """(slots, address of the state, address of the index) of a step."""
    if state is None:
        raise ValueError("state must be given")
    ss = state.shape
    if ss[1:] != tail or state.dtype is not dtype or state.device != dev or not state.is_contiguous():
        raise ValueError(f"state must be contiguous {str(dtype)[6:]} {['slots', *tail]} on {dev}")
    if index is None:
        if ss[0] != B:
            raise ValueError(f"a state of {ss[0]} slots needs state_index for {B} sequences")
        return B, state.data_ptr(), None
    if index.dtype is not torch.int32 or index.shape != (B,) or index.device != dev or not index.is_contiguous():
        raise ValueError(f"state_index must be contiguous int32 {[B]} on {dev}")
    return ss[0], state.data_ptr(), index.data_ptr()


def _ssm_operands(x, dt, A, B, C, D, z, dt_bias) -> tuple:
    """Checks a selective scan's operands; (type, channels, N, G, addresses of A, D and dt_bias)."""
    kind = _type(x, "x")
    xs, dtype, dev = x.shape, x.dtype, x.device
    Dch = xs[-1]
    if A.dim() != 2:
        raise ValueError("A must be [D, N]")
    N, bs = A.shape[1], B.shape
    grouped = len(bs) == len(xs) + 1
    G = bs[-2] if grouped else 1
    want = xs[:-1] + ((G, N) if grouped else (N,))
    _rows(x, xs, dtype, dev, "x")
    _rows(dt, xs, dtype, dev, "dt")
    _rows(B, want, dtype, dev, "B")
    _rows(C, want, dtype, dev, "C")
    if z is not None:
        _rows(z, xs, dtype, dev, "z")
    if G != 1:
        if G < 1 or Dch % G:
            raise ValueError(f"{G} groups do not divide {Dch} channels")
        if (B.stride(-2) != N or C.stride(-2) != N) and B.numel():
            raise ValueError("B, C: the last two dimensions must be contiguous")
    return kind, Dch, N, G, _param(A, (Dch, N), x, "A"), _param(D, (Dch,), x, "D"), _param(dt_bias, (Dch,), x, "dt_bias")


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = True, state_in=None,
                   seq_offsets=None, state_index=None, out=None, state_out=None, want_state: bool = True,
                   workspace=None, stream=None) -> Tuple:
    """Selective state space scan: per channel, with dt' = softplus(dt + dt_bias) (dt + dt_bias without
    ``dt_softplus``), h = exp(dt' A) h + dt' x B, y = h . C + D x, out = y silu(z).

    x, dt, z [B, T, Dch] (or [T, Dch] packed with ``seq_offsets``); A [Dch, N] float32 (<= 0), N <= 256; B, C
    [..., G, N] or [..., N], shared by groups of Dch / G channels; D, dt_bias [Dch] float32 or None.  States
    [slots, Dch, N] float32: ``state_in`` (None: zeros), ``state_out`` (may be ``state_in``), ``state_index`` as for
    causal_conv.  ``workspace``: a uint8 tensor (``gdn_ssm_workspace_bytes``); a smaller one, or None, is replaced by
    one allocated here.  Returns (out like x, state_out or None)."""
    kind, Dch, N, G, pA, pD, pbias = _ssm_operands(x, dt, A, B, C, D, z, dt_bias)
    S, T = _lead(x, seq_offsets)
    slots, new_state = _states(S, (Dch, N), torch.float32, x, state_in, state_out, state_index, want_state)
    out, made = _output(out, x)
    packed = seq_offsets is not None
    zs = (0, 0) if z is None else _strides(z, packed)
    problem = _g.gdn_ssm_problem_t(S, T, Dch, N, G, *_strides(x, packed), *_strides(dt, packed), *zs,
                                   *_strides(B, packed), *_strides(C, packed), *_strides(out, packed), slots, kind,
                                   _g.GDN_SSM_OPT_SOFTPLUS if dt_softplus else 0, _ptr(seq_offsets), _ptr(state_index),
                                   _ptr(z), pbias, pD)
    if state_out is None and new_state is not None:
        made += (new_state,)
    size = _g.gdn_ssm_workspace_bytes(problem)
    if size:
        if workspace is None or workspace.numel() < size:
            workspace = torch.empty(size, dtype=torch.uint8, device=x.device)
            made += (workspace,)
        elif workspace.dtype != torch.uint8 or workspace.device != x.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous uint8 tensor on {x.device}")
        problem.workspace, problem.workspace_bytes = workspace.data_ptr(), workspace.numel()
    _call(_g.lib().gdn_ssm_forward, problem, x.device, stream, made, x.data_ptr(), dt.data_ptr(), pA, B.data_ptr(),
          C.data_ptr(), _ptr(state_in), _ptr(new_state), out.data_ptr())
    return out, new_state


def selective_step(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = True, state=None,
                   state_index=None, out=None, stream=None):
    """The selective scan of one new token per sequence: x, dt, z [S, Dch], B, C [S, G, N] or [S, N]; ``state``
    [slots, Dch, N] float32 is read and advanced in place.  A row whose ``state_index`` is out of range is skipped.
    Returns out [S, Dch]."""
    if x.dim() != 2:
        raise ValueError("x must be [S, D]")
    kind, Dch, N, G, pA, pD, pbias = _ssm_operands(x, dt, A, B, C, D, z, dt_bias)
    S = x.shape[0]
    slots, ps, pi = _step_state(state, (Dch, N), _F32, x.device, state_index, S)
    out, made = _output(out, x)
    problem = _g.gdn_ssm_problem_t(S, 1, Dch, N, G, x.stride(0), 0, dt.stride(0), 0, 0 if z is None else z.stride(0),
                                   0, B.stride(0), 0, C.stride(0), 0, out.stride(0), 0, slots, kind,
                                   _g.GDN_SSM_OPT_SOFTPLUS if dt_softplus else 0, None, pi, _ptr(z), pbias, pD)
    _call(_g.lib().gdn_ssm_step, problem, x.device, stream, made, x.data_ptr(), dt.data_ptr(), pA, B.data_ptr(), C.data_ptr(),
          ps, out.data_ptr())
    return out


def rotary_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       original: int = 4096, slow: float = 1.0, fast: float = 32.0,
                       factors: Optional[Sequence[float]] = None) -> Tuple:
    """Rotary frequencies in 64 bits, base^(-2i / rot) for pair i, for contexts ``factor`` times as long as the
    ``original`` one; returns (inv_freq [rot / 2] float64 on the CPU, length scale).

    ``scaling``: "none"; "linear" (every frequency / factor); "base" (the base times factor^(rot / (rot - 2)), so that
    the slowest pair is slowed by the factor and the fastest not at all); "parts" (a pair that turns at least ``fast``
    times over the original context keeps its frequency, one that turns at most ``slow`` times is slowed by the
    factor, those between are blended linearly in their turns); "pairs" (pair i / factors[i]).  The length scale, for
    ``rotary``'s ``scale``, is 0.1 ln(factor) + 1 for "parts" and 1 otherwise; pass another to ``rotary`` to leave
    it out."""
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if scaling not in ("none", "linear", "base", "parts", "pairs"):
        raise ValueError("scaling must be 'none', 'linear', 'base', 'parts' or 'pairs'")
    if not factor >= 1.0:
        raise ValueError("factor must be at least 1")
    if scaling == "base":
        if rot < 4:
            raise ValueError("scaling 'base' needs rot of at least 4")
        base = base * factor ** (rot / (rot - 2))
    f = torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    if scaling == "linear":
        f = f / factor
    elif scaling == "pairs":
        if factors is None or len(factors) != rot // 2:
            raise ValueError(f"factors must be {rot // 2} numbers")
        f = f / torch.tensor([float(x) for x in factors], dtype=torch.float64)
    elif scaling == "parts":
        if not fast > slow:
            raise ValueError("fast must exceed slow")
        keep = ((original * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        return f * (keep + (1.0 - keep) / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rotary(q, k, inv_freq, positions=None, interleaved: bool = False, sections: Optional[Sequence[int]] = None,
           scale: float = 1.0, inverse: bool = False, position0: int = 0, q_out=None, k_out=None, stream=None) -> Tuple:
    """Rotary positions on q [B, T, Hq, d] and k [B, T, Hk, d] (or None): pair i of every head is turned by
    position * inv_freq[i] and scaled; channels from 2 len(inv_freq) on pass through.

    Pairs are (x[i], x[i + rot / 2]), with ``interleaved`` (x[2i], x[2i + 1]).  inv_freq [rot / 2] float64 (see
    ``rotary_frequencies``).  ``positions`` [B, T] or [axes, B, T], int32 or int64 (None: position0 + t); with several
    axes ``sections`` gives the pairs that follow each axis.  ``inverse`` turns back: the gradient of the call.
    ``q_out`` and ``k_out`` may be q and k (in place).  Returns (q_out, k_out or None)."""
    dt = _type(q, "q")
    if q.dim() != 4:
        raise ValueError("q must be [B, T, H, d]")
    B, T, Hq, d = q.shape
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be [rot / 2]")
    pairs = inv_freq.shape[0]
    pf = _param(inv_freq, (pairs,), q, "inv_freq", torch.float64)
    Hk = 0
    for t, name in ((q, "q"), (k, "k")):
        if t is None:
            continue
        if t.dtype != q.dtype or t.device != q.device or t.dim() != 4 or t.shape[:2] != q.shape[:2] or t.shape[3] != d:
            raise ValueError(f"{name} must be [{B}, {T}, H, {d}] of the type and on the device of q")
        if d != 1 and t.stride(3) != 1 and t.numel():
            raise ValueError(f"{name}: the last dimension must be contiguous")
    q_out, made = _output(q_out, q, "q_out")
    if k is not None:
        Hk = k.shape[2]
        k_out, mk = _output(k_out, k, "k_out")
        made += mk
    elif k_out is not None:
        raise ValueError("k_out without k")
    axes, bits = 1, 0
    if positions is not None:
        if positions.dtype not in (torch.int32, torch.int64) or positions.device != q.device \
                or not positions.is_contiguous():
            raise ValueError(f"positions must be contiguous int32 or int64 on {q.device}")
        if positions.dim() == 3:
            axes = positions.shape[0]
        if positions.shape[-2:] != (B, T) or positions.dim() not in (2, 3):
            raise ValueError(f"positions must be [{B}, {T}] or [axes, {B}, {T}]")
        bits = 64 if positions.dtype == torch.int64 else 32
    if sections is None:
        if axes != 1:
            raise ValueError("several axes need sections")
        sections = (pairs,)
    if len(sections) != axes or axes > 4:
        raise ValueError(f"sections must give the pairs of each of {axes} axes (at most 4)")
    problem = _g.gdn_rotary_problem_t(B, T, Hq, Hk, d, 2 * pairs, *q.stride()[:3],
                                      *((0, 0, 0) if k is None else k.stride()[:3]), *q_out.stride()[:3],
                                      *((0, 0, 0) if k is None else k_out.stride()[:3]), position0, dt,
                                      (_g.GDN_ROTARY_OPT_INTERLEAVED if interleaved else 0)
                                      | (_g.GDN_ROTARY_OPT_INVERSE if inverse else 0), bits, axes, tuple(sections), scale)
    _call(_g.lib().gdn_rotary, problem, q.device, stream, made, q.data_ptr(), _ptr(k), pf, _ptr(positions), q_out.data_ptr(),
          None if k is None else k_out.data_ptr())
    return q_out, k_out


def delta_step(q, k, v, log_alpha, beta, state, state_index=None, erase: bool = True, exclusive: bool = False,
               gate=None, norm_weight=None, norm_eps: float = 1e-6, out=None, stream=None):
    """One token of ``forward`` (forward direction) for each of B sequences: q, k [B, H, dk], v [B, H, dv];
    log_alpha, beta [B, H] float32; ``state`` [slots, H, dv, dk] float32 is read and advanced in place, sequence b in
    slot ``state_index[b]`` (None: slot b; out of range: the row is skipped).  ``erase``, ``exclusive`` (o read
    before the token's own write), ``gate`` [B, H, dv], ``norm_weight`` [dv] and ``norm_eps`` as for ``forward``.
    Returns out [B, H, dv] float32."""
    dtype, dev, qs = q.dtype, q.device, q.shape
    dt = _type(q, "q")
    if len(qs) != 3 or v.dim() != 3:
        raise ValueError("q, k must be [B, H, dk] and v [B, H, dv]")
    B, H, dk = qs
    dv = v.shape[2]
    vs, gs = (B, H, dv), (B, H)
    if not (k.shape == qs and v.shape == vs and k.dtype is dtype and v.dtype is dtype and k.device == dev
            and v.device == dev and q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError(f"q, k, v must be contiguous {str(dtype)[6:]} {list(qs)}, {list(qs)}, {list(vs)} on {dev}")
    if not (log_alpha.shape == gs and beta.shape == gs and log_alpha.dtype is _F32 and beta.dtype is _F32
            and log_alpha.device == dev and beta.device == dev and log_alpha.is_contiguous() and beta.is_contiguous()):
        raise ValueError(f"log_alpha and beta must be contiguous float32 {list(gs)} on {dev}")
    slots, ps, pi = _step_state(state, (H, dv, dk), _F32, dev, state_index, B)
    pg, pw = None, None
    if gate is not None:
        pg, pw = _param(gate, (B, H, dv), q, "gate", dtype), _param(norm_weight, (dv,), q, "norm_weight")
        if pw is None:
            raise ValueError(f"norm_weight must be float32 [{dv}] when gate is given")
    made = ()
    if out is None:
        out = torch.empty_like(v, dtype=_F32)
        made = (out,)
    else:
        _param(out, (B, H, dv), q, "out")
    problem = _g.gdn_step_problem_t(B, H, dk, dv, slots, dt, (0 if erase else _g.GDN_OPT_NO_ERASE)
                                    | (_g.GDN_OPT_EXCLUSIVE_FORWARD if exclusive else 0), pi, pg, pw, norm_eps)
    _call(_g.lib().gdn_step, problem, dev, stream, made, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_alpha.data_ptr(),
          beta.data_ptr(), ps, out.data_ptr())
    return out


def register_ops() -> None:
    """The calls as torch.library custom ops (torch.ops.gdn.causal_conv, causal_conv_step, selective_scan,
    selective_step, rotary, delta_step) with fake implementations for tracing; the steps mutate ``state``."""
    op = torch.library.custom_op

    @op("gdn::causal_conv", mutates_args=(), device_types="cuda",
        schema="(Tensor x, Tensor weight, Tensor? bias, Tensor? state_in, str activation, Tensor? seq_offsets) "
               "-> (Tensor, Tensor)")
    def _conv(x, weight, bias, state_in, activation, seq_offsets):
        return causal_conv(x, weight, bias, state_in, activation, seq_offsets)

    @_conv.register_fake
    def _(x, weight, bias, state_in, activation, seq_offsets):
        B = x.shape[0] if seq_offsets is None else seq_offsets.shape[0] - 1
        return x.new_empty(x.shape), x.new_empty((B, weight.shape[1] - 1, x.shape[-1]))

    @op("gdn::causal_conv_step", mutates_args=("state",), device_types="cuda",
        schema="(Tensor x, Tensor weight, Tensor? bias, Tensor(a!) state, str activation, Tensor? state_index) -> Tensor")
    def _conv_step(x, weight, bias, state, activation, state_index):
        return causal_conv_step(x, weight, bias, state, activation, state_index)

    @_conv_step.register_fake
    def _(x, weight, bias, state, activation, state_index):
        return x.new_empty(x.shape)

    @op("gdn::selective_scan", mutates_args=(), device_types="cuda",
        schema="(Tensor x, Tensor dt, Tensor A, Tensor B, Tensor C, Tensor? D, Tensor? z, Tensor? dt_bias, "
               "bool dt_softplus, Tensor? state_in, Tensor? seq_offsets) -> (Tensor, Tensor)")
    def _scan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, state_in, seq_offsets):
        return selective_scan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, state_in, seq_offsets)

    @_scan.register_fake
    def _(x, dt, A, B, C, D, z, dt_bias, dt_softplus, state_in, seq_offsets):
        S = x.shape[0] if seq_offsets is None else seq_offsets.shape[0] - 1
        return x.new_empty(x.shape), x.new_empty((S,) + tuple(A.shape), dtype=torch.float32)

    @op("gdn::selective_step", mutates_args=("state",), device_types="cuda",
        schema="(Tensor x, Tensor dt, Tensor A, Tensor B, Tensor C, Tensor? D, Tensor? z, Tensor? dt_bias, "
               "bool dt_softplus, Tensor(a!) state, Tensor? state_index) -> Tensor")
    def _step(x, dt, A, B, C, D, z, dt_bias, dt_softplus, state, state_index):
        return selective_step(x, dt, A, B, C, D, z, dt_bias, dt_softplus, state, state_index)

    @_step.register_fake
    def _(x, dt, A, B, C, D, z, dt_bias, dt_softplus, state, state_index):
        return x.new_empty(x.shape)

    @op("gdn::rotary", mutates_args=(), device_types="cuda",
        schema="(Tensor q, Tensor k, Tensor inv_freq, Tensor? positions, bool interleaved, int[]? sections, float scale, "
               "bool inverse, int position0) -> (Tensor, Tensor)")
    def _rotary(q, k, inv_freq, positions, interleaved, sections, scale, inverse, position0):
        return rotary(q, k, inv_freq, positions, interleaved, sections, scale, inverse, position0)

    @_rotary.register_fake
    def _(q, k, inv_freq, positions, interleaved, sections, scale, inverse, position0):
        return q.new_empty(q.shape), k.new_empty(k.shape)

    @op("gdn::delta_step", mutates_args=("state",), device_types="cuda",
        schema="(Tensor q, Tensor k, Tensor v, Tensor log_alpha, Tensor beta, Tensor(a!) state, Tensor? state_index, "
               "bool erase, bool exclusive, Tensor? gate, Tensor? norm_weight, float norm_eps) -> Tensor")
    def _delta(q, k, v, log_alpha, beta, state, state_index, erase, exclusive, gate, norm_weight, norm_eps):
        return delta_step(q, k, v, log_alpha, beta, state, state_index, erase, exclusive, gate, norm_weight, norm_eps)

    @_delta.register_fake
    def _(q, k, v, log_alpha, beta, state, state_index, erase, exclusive, gate, norm_weight, norm_eps):
        return q.new_empty(v.shape, dtype=torch.float32)
