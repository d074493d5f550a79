"""What a hybrid model runs beside its recurrent layers, on torch CUDA tensors:
a paged cache of keys and values (as they are, or in 8 or 4 bits), a new
token's attention over it, and the seam between two blocks (norm, gate,
residual, norm) with its gradients (layouts and rules of ``include/gdn.h``).

Checked and launched in native code like the operators of ``layer.py``, whose
rules for ``stream``, packed batches (``seq_offsets``), strided views and rows
of no sequence hold here too.  ``residual_norm`` takes part in autograd; the
cache and its attention serve, and their results have no graph.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

import gated_delta_rule_scan_amd as _g

from .layer import _native


class KVCache(NamedTuple):
    """Pools of pages: k, v [pages, heads, page, d]; with 8 or 4 bits a channel also the scale bytes of every 32
    channels, k_scales, v_scales [pages, heads, page, d / 32].  The calls take any such tuple."""

    k: torch.Tensor
    v: torch.Tensor
    k_scales: Optional[torch.Tensor] = None
    v_scales: Optional[torch.Tensor] = None


def kv_cache(pages: int, heads: int, page: int, d: int, format: str = "bfloat16", device="cuda") -> KVCache:
    """A cache of zeros: ``pages`` pages of ``page`` tokens (a power of two, 16 to 1024), ``heads`` heads of ``d`` (64,
    128 or 256) channels.  ``format``: "float32", "bfloat16", "mxfp8" (e4m3, 1.03 bytes a channel) or "mxfp4" (e2m1,
    0.53 bytes); the last two scale every 32 channels by a power of two of their own."""
    if format not in ("float32", "bfloat16", "mxfp8", "mxfp4"):
        raise ValueError("format must be 'float32', 'bfloat16', 'mxfp8' or 'mxfp4'")
    if d not in (64, 128, 256):
        raise ValueError("d must be 64, 128 or 256")
    if page < 16 or page > 1024 or page & (page - 1):
        raise ValueError("page must be a power of two, 16 to 1024")

    def zeros(width, dtype):
        return torch.zeros((pages, heads, page, width), dtype=dtype, device=device)

    if format in ("float32", "bfloat16"):
        dtype = getattr(torch, format)
        return KVCache(zeros(d, dtype), zeros(d, dtype))
    pools = [zeros(d, torch.uint8).view(torch.float8_e4m3fn) if format == "mxfp8" else zeros(d // 2, torch.uint8)
             for _ in range(2)]
    return KVCache(*pools, zeros(d // 32, torch.uint8), zeros(d // 32, torch.uint8))


def kv_write(k, v, cache, page_table, start=None, seq_offsets=None, stream=None) -> None:
    """Rows of keys and values into a paged cache, quantised as its format has it.

    k, v [B, T, heads, d], [B, heads, d] (one token each) or [T, heads, d] packed with ``seq_offsets``; a cache in
    float32 or bfloat16 takes rows of its own type.  page_table [B, pages of a sequence] int32: token t of sequence b
    goes to position ``start[b]`` + t (``start`` [B] int32; None: 0), row position % page of page page_table[b, position
    / page].  A position beyond the table, or one whose page number is no page, is not written.  No two tokens of a call may
    have the same place."""
    _native().kv_write(k, v, cache, page_table, start, seq_offsets, stream)


def kv_read(cache, page_table, tokens: int, start=None, seq_offsets=None, dtype=None, k_out=None, v_out=None,
            stream=None) -> Tuple:
    """Rows of keys and values out of a paged cache: of every sequence ``tokens`` from position ``start[b]`` on, as
    (k, v) [B, tokens, heads, d]; or with ``seq_offsets``, of sequence b as many as the offsets say, packed
    [tokens, heads, d].  ``dtype`` float32 or bfloat16: that of the outputs, or else the cache's, or bfloat16; a cache in
    float32 or bfloat16 gives its own type.  Rows of tokens without a place are zero in outputs made by the call and
    stay as they were in given ones."""
    codes = {None: -1, torch.float32: _g.GDN_DTYPE_F32, torch.bfloat16: _g.GDN_DTYPE_BF16}
    if dtype not in codes:
        raise TypeError("dtype must be float32 or bfloat16")
    return _native().kv_read(cache, page_table, tokens, start, seq_offsets, codes[dtype], k_out, v_out, stream)


def attention_step(q, cache, page_table, lengths, scale: Optional[float] = None, window: int = 0, sinks: int = 0, out=None,
                   lse=None, workspace=None, stream=None):
    """Attention of one new token per sequence over a paged cache: q [B, Hq, d], heads of the cache shared by Hq / heads
    query heads each, softmax(scale q . k) v over the first ``lengths[b]`` positions (the new token's own, written
    before, included), with ``window`` only the last ``window`` of them and the first ``sinks``.  lengths [B] int32;
    ``scale`` None: d^-1/2.  Positions without a page are left out; where nothing is left the output is zero.  ``lse``
    [B, Hq] float32 receives log(sum(exp(scale q . k))) (nothing left: minus infinity).  ``workspace``: a uint8 tensor
    (``gdn_attention_workspace_bytes``); a smaller one, or None, is replaced by one allocated here.  Returns out like q."""
    return _native().attention_step(q, cache, page_table, lengths, scale, window, sinks, out, lse, workspace, stream)


def residual_norm(x, y=None, gate=None, post_weight=None, weight=None, residual_scale: float = 1.0, eps: float = 1e-6,
                  seq_offsets=None, out=None, norm_out=None, stream=None) -> Tuple:
    """The seam between two blocks, per row: u = post_weight rms(y) (None: y), h = residual_scale x + gate u, n = weight
    rms(h), with rms(z) = z / sqrt(mean(z^2) + eps).

    x, y [B, T, D], [B, D] (a token each) or [T, D] packed with ``seq_offsets``; ``gate`` [D], or [B, D] (a gate for
    every sequence), float32; ``weight``, ``post_weight`` [D] float32.  ``out`` (of h) may be x.  Returns (h, n), n None
    without ``weight``; without y, out and a residual scale h is x itself.

    Where x, y or a parameter requires gradients (and they are enabled) the results have a graph, whose backward pass is
    ``residual_norm_backward``; ``out``, ``norm_out`` and ``stream`` are refused then."""
    got = _native().residual_norm(x, y, gate, post_weight, weight, residual_scale, eps, seq_offsets, out, norm_out, stream)
    if got is not None:
        return got
    got = _ResidualNorm.apply(x, y, gate, post_weight, weight, residual_scale, eps, seq_offsets)
    return got if len(got) == 2 else (*got, None) if weight is None else (x, *got)


class _ResidualNorm(torch.autograd.Function):
    """h and n of ``residual_norm``, those of them that it computes."""

    @staticmethod
    def forward(ctx, x, y, gate, post_weight, weight, residual_scale, eps, seq_offsets):
        h, n = _native().residual_norm(x, y, gate, post_weight, weight, residual_scale, eps, seq_offsets, None, None, None)
        ctx.save_for_backward(x, y, gate, post_weight, weight, seq_offsets)
        ctx.numbers, ctx.h = (residual_scale, eps), h is not x
        ctx.set_materialize_grads(False)
        return tuple(t for t in (h if ctx.h else None, n) if t is not None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, *grads):
        x, y, gate, post_weight, weight, seq_offsets = ctx.saved_tensors
        dh = grads[0] if ctx.h else None
        dn = None if weight is None else grads[-1]
        if dh is None and dn is None:
            return (None,) * 8
        got = residual_norm_backward(dh, dn, x, y, gate, post_weight, None if dn is None else weight, *ctx.numbers, seq_offsets)
        return (*(g if need else None for g, need in zip(got, ctx.needs_input_grad)), None, None, None)


def residual_norm_backward(dh, dn, x, y=None, gate=None, post_weight=None, weight=None, residual_scale: float = 1.0,
                           eps: float = 1e-6, seq_offsets=None, dx=None, dy=None, workspace=None, stream=None) -> Tuple:
    """The gradients of ``residual_norm``: dh, dn those of its outputs (dh None: zero; dn goes with ``weight``), the
    others its arguments; where their rows are not contiguous (a sum's gradient is one value, expanded) they are copied
    first.  ``dx`` may be dh.  ``workspace``: a uint8 tensor (``gdn_norm_workspace_bytes``); a smaller
    one, or None, is replaced by one allocated here.  Returns (dx, dy, dgate, dpost_weight, dweight), each None where the
    argument was; the last three float32."""
    return _native().residual_norm_backward(dh, dn, x, y, gate, post_weight, weight, residual_scale, eps, seq_offsets, dx,
                                            dy, workspace, stream)


def register_ops() -> None:
    """The calls as torch.library custom ops (torch.ops.gdn.kv_write, kv_read, attention_step, residual_norm,
    residual_norm_backward) with fake implementations for tracing; kv_write mutates the cache.  residual_norm's op
    needs y and weight; it alone has an autograd formula."""
    op = torch.library.custom_op
    cache = "Tensor k_cache, Tensor v_cache, Tensor? k_scales, Tensor? v_scales"

    def of(k, v, ks, vs):
        return (k, v) if ks is None else (k, v, ks, vs)

    @op("gdn::kv_write", mutates_args=("k_cache", "v_cache", "k_scales", "v_scales"), device_types="cuda",
        schema="(Tensor k, Tensor v, Tensor(a!) k_cache, Tensor(b!) v_cache, Tensor(c!)? k_scales, Tensor(d!)? v_scales, "
               "Tensor page_table, Tensor? start, Tensor? seq_offsets) -> ()")
    def _write(k, v, k_cache, v_cache, k_scales, v_scales, page_table, start, seq_offsets):
        kv_write(k, v, of(k_cache, v_cache, k_scales, v_scales), page_table, start, seq_offsets)

    @_write.register_fake
    def _(k, v, k_cache, v_cache, k_scales, v_scales, page_table, start, seq_offsets):
        return None

    @op("gdn::kv_read", mutates_args=(), device_types="cuda",
        schema=f"({cache}, Tensor page_table, int tokens, Tensor? start, Tensor? seq_offsets, ScalarType dtype) "
               "-> (Tensor, Tensor)")
    def _read(k_cache, v_cache, k_scales, v_scales, page_table, tokens, start, seq_offsets, dtype):
        return kv_read(of(k_cache, v_cache, k_scales, v_scales), page_table, tokens, start, seq_offsets, dtype)

    @_read.register_fake
    def _(k_cache, v_cache, k_scales, v_scales, page_table, tokens, start, seq_offsets, dtype):
        d = k_cache.shape[3] * (2 if k_cache.dtype == torch.uint8 else 1)
        lead = (page_table.shape[0], tokens) if seq_offsets is None else (tokens,)
        return tuple(k_cache.new_empty((*lead, k_cache.shape[1], d), dtype=dtype) for _ in range(2))

    @op("gdn::attention_step", mutates_args=(), device_types="cuda",
        schema=f"(Tensor q, {cache}, Tensor page_table, Tensor lengths, float? scale, int window, int sinks) "
               "-> (Tensor, Tensor)")
    def _attend(q, k_cache, v_cache, k_scales, v_scales, page_table, lengths, scale, window, sinks):
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        y = attention_step(q, of(k_cache, v_cache, k_scales, v_scales), page_table, lengths, scale, window, sinks, lse=lse)
        return y, lse

    @_attend.register_fake
    def _(q, k_cache, v_cache, k_scales, v_scales, page_table, lengths, scale, window, sinks):
        return q.new_empty(q.shape), q.new_empty(q.shape[:2], dtype=torch.float32)

    @op("gdn::residual_norm", mutates_args=(), device_types="cuda",
        schema="(Tensor x, Tensor y, Tensor? gate, Tensor? post_weight, Tensor weight, float residual_scale, float eps, "
               "Tensor? seq_offsets) -> (Tensor, Tensor)")
    def _norm(x, y, gate, post_weight, weight, residual_scale, eps, seq_offsets):
        with torch.no_grad():  # (the graph is the op's)
            return residual_norm(x, y, gate, post_weight, weight, residual_scale, eps, seq_offsets)

    @_norm.register_fake
    def _(x, y, gate, post_weight, weight, residual_scale, eps, seq_offsets):
        return x.new_empty(x.shape), x.new_empty(x.shape)

    def _keep(ctx, inputs, output):
        *tensors, ctx.residual_scale, ctx.eps, offsets = inputs
        ctx.save_for_backward(*tensors, offsets)

    def _gradients(ctx, dh, dn):
        *tensors, offsets = ctx.saved_tensors
        got = torch.ops.gdn.residual_norm_backward(dh, dn, *tensors, ctx.residual_scale, ctx.eps, offsets)
        return (*(None if t is None else g for g, t in zip(got, tensors)), None, None, None)

    _norm.register_autograd(_gradients, setup_context=_keep)

    @op("gdn::residual_norm_backward", mutates_args=(), device_types="cuda",
        schema="(Tensor? dh, Tensor dn, Tensor x, Tensor y, Tensor? gate, Tensor? post_weight, Tensor weight, "
               "float residual_scale, float eps, Tensor? seq_offsets) -> (Tensor, Tensor, Tensor, Tensor, Tensor)")
    def _back(dh, dn, x, y, gate, post_weight, weight, residual_scale, eps, seq_offsets):
        got = residual_norm_backward(dh, dn, x, y, gate, post_weight, weight, residual_scale, eps, seq_offsets)
        return tuple(x.new_empty(0, dtype=torch.float32) if t is None else t for t in got)

    @_back.register_fake
    def _(dh, dn, x, y, gate, post_weight, weight, residual_scale, eps, seq_offsets):
        e = lambda t: x.new_empty((0,) if t is None else t.shape, dtype=torch.float32)
        return x.new_empty(x.shape), x.new_empty(x.shape), e(gate), e(post_weight), e(weight)
