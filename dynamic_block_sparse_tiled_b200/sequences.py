"""Sequences of different lengths: rotary positions, a paged KV cache, exact
attention over packed prompts (with its gradients) and over the cache.

The functions take torch tensors through the compiled binding
(``csrc/seq_binding.cpp``) to the C ABI of ``include/blasst.h``
(``blasst_rotary``, ``blasst_append``, ``blasst_packed_fwd``,
``blasst_packed_bwd``, ``blasst_paged_fwd``), which documents layouts, masks
and the checks made on the device. Packed tokens are ``[T, heads, d]``; any
token and head strides are taken as long as ``d`` is contiguous. Lengths and
page tables stay on the device: a call neither synchronises nor reads them, and
a captured call may be replayed after they have changed.

Autograd records none of the calls. Tensors that require a gradient are refused
(ValueError) unless gradients are off, as they are under ``torch.no_grad()`` and
within a ``torch.autograd.Function``, whose backward then calls
``rotary_backward`` and ``attention_packed_backward``.
"""
from __future__ import annotations

import math

__all__ = [
    "rope_frequencies", "rotary", "rotary_backward", "paged_append", "attention_packed",
    "attention_packed_backward", "attention_paged", "blasst_seq_workspace_bytes",
    "blasst_packed_bwd_workspace_bytes",
]

_ops = None


def _native():
    """The compiled torch binding (raises if it has not been built)."""
    global _ops
    if _ops is None:
        import torch  # noqa: F401  (its libraries have to be loaded first)
        from . import load_library
        load_library()
        try:
            from . import _seq_binding
        except ImportError as e:
            raise RuntimeError(
                "the compiled binding _seq_binding is missing; build it with `python -m "
                "dynamic_block_sparse_tiled_b200.build` (there is no CPU fallback)") from e
        _ops = _seq_binding
    return _ops


def _raw(stream):
    """None (the current stream), or a stream's handle."""
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def blasst_seq_workspace_bytes(d: int) -> int:
    """The C entry point of the same name (current device)."""
    from . import load_library
    return int(load_library().blasst_seq_workspace_bytes(int(d)))


def blasst_packed_bwd_workspace_bytes(Tq: int, Hq: int, Hkv: int) -> int:
    """The C entry point of the same name."""
    from . import load_library
    return int(load_library().blasst_packed_bwd_workspace_bytes(int(Tq), int(Hq), int(Hkv)))


# ------------------------------------------------------------------- rotary
def rope_frequencies(rot, *, base=10000.0, scaling="none", factor=1.0, original_len=0,
                     low=None, high=None, device="cuda"):
    """Angle per position of each pair, float64 [rot / 2], and the factor for
    the turned dims. f_i = base^(-2 i / rot), then by ``scaling``:

      none    f_i;
      linear  f_i / factor (positions interpolated);
      ntk     base * factor^(rot / (rot - 2)) in the place of base;
      blend   (YaRN) pairs that turn at least ``high`` (32) times over
              ``original_len`` positions are kept, those of at most ``low`` (1)
              turns divided by factor, a straight line over the pair's index
              (from 0 on at the earliest) between; factor for the dims
              0.1 ln(factor) + 1;
      bands   as blend over the number of turns, from ``low`` (1) to ``high`` (4),
              and a factor of 1 for the dims.
    """
    import torch
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if not base > 1.0 or not factor > 0.0:
        raise ValueError("base must be over 1 and factor over 0")
    if scaling == "ntk":
        if rot < 4:
            raise ValueError("ntk scaling needs rot >= 4")
        base = base * factor ** (rot / (rot - 2))
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot)
    mscale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling in ("blend", "bands"):
        if original_len <= 0:
            raise ValueError(f"{scaling} scaling needs original_len")
        lo = 1.0 if low is None else float(low)
        hi = (32.0 if scaling == "blend" else 4.0) if high is None else float(high)
        if not 0.0 < lo < hi:
            raise ValueError("low must be over 0 and under high")
        if scaling == "blend":
            # pair index at which a pair turns n times over original_len positions; where the
            # last pair turns more than lo times, the line ends behind the table
            at = lambda n: rot * math.log(original_len / (n * 2.0 * math.pi)) / (2.0 * math.log(base))  # noqa: E731
            first, last = max(math.floor(at(hi)), 0), math.ceil(at(lo))
            keep = 1.0 - ((i - first) / max(last - first, 1e-3)).clamp(0.0, 1.0)
            if factor > 1.0:
                mscale = 0.1 * math.log(factor) + 1.0
        else:
            turns = original_len * f / (2.0 * math.pi)
            keep = ((turns - lo) / (hi - lo)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device), mscale


def rotary(x, inv_freq, positions=None, *, interleaved=False, mscale=1.0, out=None, stream=None):
    """blasst_rotary: x [T, H, d] (packed) or [B, H, L, d] turned by
    ``positions`` ([T], or [L] / [B, L]; None: 0, 1, ...) times ``inv_freq``
    (``rope_frequencies``; its length gives the turned dims). ``out`` may be x."""
    return (_ops or _native()).rotary(x, inv_freq, positions, interleaved, mscale, out, _raw(stream),
                                      False)


def rotary_backward(dy, inv_freq, positions=None, *, interleaved=False, mscale=1.0, out=None,
                    stream=None):
    """Gradient of ``rotary`` with respect to x: the transposed turn of dy."""
    return (_ops or _native()).rotary(dy, inv_freq, positions, interleaved, mscale, out,
                                      _raw(stream), True)


def paged_append(q, k, v, k_pages, v_pages, page_table, kv_lens, cu_q, *, inv_freq=None,
                 interleaved=False, mscale=1.0, q_out=None, stream=None):
    """blasst_append: writes the new tokens' k (turned) and v [T, Hkv, d] into
    the pages and returns q [T, Hq, d] turned (into ``q_out``, which may be q).
    ``kv_lens`` counts each sequence's tokens with the new ones. Without
    ``inv_freq`` nothing is turned."""
    return (_ops or _native()).paged_append(q, k, v, k_pages, v_pages, page_table, kv_lens, cu_q,
                                            inv_freq, interleaved, mscale, q_out, _raw(stream))


# ---------------------------------------------------------------- attention
def attention_packed(q, k, v, cu_q, cu_k=None, *, causal=True, scale=0.0, workspace=None,
                     stream=None):
    """blasst_packed_fwd: exact attention of packed sequences, q [Tq, Hq, d],
    k, v [Tk, Hkv, d], ``cu_k`` None for cu_q. Returns (o [Tq, Hq, d],
    lse [Tq, Hq] fp32); tokens of no sequence are left unwritten."""
    return (_ops or _native()).attention_packed(q, k, v, cu_q, cu_k, causal, scale, workspace,
                                                _raw(stream))


def attention_packed_backward(q, k, v, o, lse, dout, cu_q, cu_k=None, *, causal=True, scale=0.0,
                              workspace=None, stream=None):
    """blasst_packed_bwd: gradients (dq, dk, dv) of ``attention_packed`` in the
    inputs' type, from its outputs o and lse and the gradient dout of o. Tokens
    of no sequence are left unwritten."""
    return (_ops or _native()).attention_packed_backward(q, k, v, o, lse, dout, cu_q, cu_k, causal,
                                                         scale, workspace, _raw(stream))


def attention_paged(q, k_pages, v_pages, page_table, kv_lens, cu_q, *, causal=True, scale=0.0,
                    workspace=None, stream=None):
    """blasst_paged_fwd: exact attention of new tokens q [T, Hq, d] (one or more
    per sequence) over the paged cache, which holds them already (``paged_append``).
    Returns (o [T, Hq, d], lse [T, Hq] fp32)."""
    return (_ops or _native()).attention_paged(q, k_pages, v_pages, page_table, kv_lens, cu_q,
                                               causal, scale, workspace, _raw(stream))
