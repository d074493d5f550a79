"""The operators a recurrent layer runs around its scan, on torch CUDA tensors:
short causal convolution, selective state space scan, rotary positions, and the
single-token steps (layouts and rules of ``include/gdn.h``).

Argument checks and marshalling only, as in the package's other calls, here in
native code (``csrc/gdn_binding.cpp``): the steps run a few microseconds, and
the same checks in Python took longer than the launch.  Imported by the
package, whose names these are.  Every call takes ``stream`` (a
``torch.cuda.Stream``; the current one of the tensors' device by default): its
work, and the memory of what it allocates, belong to that stream.  With one that
is not the current one the caller orders the two, as for any work: inputs are
ready on ``stream``, and the current stream waits for it before it uses results.
Prompts come as equal sequences ([B, T, ...]) or packed ([T, ...] with
``seq_offsets`` [B + 1] int32); operands may be strided views whose last
dimension is contiguous (the halves of one projection, say).  Rows of the
output that belong to no sequence (behind the last one of a packed batch; a
step's row whose ``state_index`` is out of range) are zero in an output made by
the call, and stay as they were in one that is given.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence, Tuple

import torch

import gated_delta_rule_scan_amd as _g

_bound = None


def _native():
    """The native binding, with the entry points of the loaded library."""
    global _bound
    if _bound is not _g._lib or _bound is None:
        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError("the native binding is missing: build it with `python -m gated_delta_rule_scan_amd.build`") \
                from e

        lib = _g.lib()
        address = lambda name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
        _binding.init(_g.GdnError, *(address(n) for n in (
            "gdn_conv_forward", "gdn_conv_step", "gdn_ssm_workspace_bytes", "gdn_ssm_forward", "gdn_ssm_step",
            "gdn_rotary", "gdn_step", "gdn_kv_write", "gdn_kv_read", "gdn_attention_workspace_bytes", "gdn_attention_step",
            "gdn_norm_forward", "gdn_norm_workspace_bytes", "gdn_norm_backward")))
        _native.binding, _bound = _binding, lib
    return _native.binding


def _activation(name: str) -> int:
    act = _g.ACTIVATIONS.get(name)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(_g.ACTIVATIONS)}")
    return act


def causal_conv(x, weight, bias=None, state_in=None, activation: str = "silu", seq_offsets=None, state_index=None,
                out=None, state_out=None, want_state: bool = True, stream=None) -> Tuple:
    """Short causal depthwise convolution over time, y[t] = act(bias + sum_j weight[:, j] x[t - (W - 1) + j]).

    x [B, T, D], or [T, D] packed with ``seq_offsets``; weight [D, W] float32, W in 2..4; bias [D] float32 or None;
    ``activation`` "silu" or "none".  ``state_in`` [slots, W - 1, D] (the type of x) holds the W - 1 rows before each
    sequence (None: zeros), ``state_out`` receives the last W - 1 and may be ``state_in``; sequence b uses slot
    ``state_index[b]`` (None: slot b; out of range: no state).
    Returns (out like x, state_out or None)."""
    return _native().causal_conv(x, weight, bias, state_in, _activation(activation), seq_offsets, state_index, out,
                                 state_out, bool(want_state), stream)


def causal_conv_step(x, weight, bias=None, state=None, activation: str = "silu", state_index=None, out=None,
                     stream=None):
    """The convolution of one new token per sequence: x [B, D]; ``state`` [slots, W - 1, D] is read and advanced in
    place.  A row whose ``state_index`` is out of range is skipped: no state changes, and its output row is zero (in
    a given ``out``: as it was).  Returns out [B, D]."""
    return _native().causal_conv_step(x, weight, bias, state, _activation(activation), state_index, out, stream)


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
    return _native().selective_scan(x, dt, A, B, C, D, z, dt_bias, bool(dt_softplus), state_in, seq_offsets, state_index,
                                    out, state_out, bool(want_state), workspace, stream)


def selective_step(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = True, state=None,
                   state_index=None, out=None, stream=None):
    """The selective scan of one new token per sequence: x, dt, z [S, Dch], B, C [S, G, N] or [S, N]; ``state``
    [slots, Dch, N] float32 is read and advanced in place.  A row whose ``state_index`` is out of range is skipped.
    Returns out [S, Dch]."""
    return _native().selective_step(x, dt, A, B, C, D, z, dt_bias, bool(dt_softplus), state, state_index, out, stream)


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
    options = (_g.GDN_ROTARY_OPT_INTERLEAVED if interleaved else 0) | (_g.GDN_ROTARY_OPT_INVERSE if inverse else 0)
    return _native().rotary(q, k, inv_freq, positions, options, sections, scale, position0, q_out, k_out, stream)


def delta_step(q, k, v, log_alpha, beta, state, state_index=None, erase: bool = True, exclusive: bool = False,
               gate=None, norm_weight=None, norm_eps: float = 1e-6, out=None, stream=None):
    """One token of ``forward`` (forward direction) for each of B sequences: q, k [B, H, dk], v [B, H, dv];
    log_alpha, beta [B, H] float32; ``state`` [slots, H, dv, dk] float32 is read and advanced in place, sequence b in
    slot ``state_index[b]`` (None: slot b; out of range: the row is skipped).  ``erase``, ``exclusive`` (o read
    before the token's own write), ``gate`` [B, H, dv], ``norm_weight`` [dv] and ``norm_eps`` as for ``forward``.
    Returns out [B, H, dv] float32."""
    options = (0 if erase else _g.GDN_OPT_NO_ERASE) | (_g.GDN_OPT_EXCLUSIVE_FORWARD if exclusive else 0)
    return _native().delta_step(q, k, v, log_alpha, beta, state, state_index, options, gate, norm_weight, norm_eps, out,
                                stream)


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
