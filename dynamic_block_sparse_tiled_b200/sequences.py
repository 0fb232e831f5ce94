"""Sequences of different lengths: rotary positions, a paged KV cache, exact
attention over packed prompts (with its gradients) and over the cache.

The functions marshal torch tensors into the C ABI of ``include/blasst.h``
(``blasst_rotary``, ``blasst_append``, ``blasst_packed_fwd``,
``blasst_packed_bwd``, ``blasst_paged_fwd``), which documents layouts, masks
and the checks made on the device. Packed tokens are ``[T, heads, d]``; any
token and head strides are taken as long as ``d`` is contiguous. Lengths and
page tables stay on the device: a call neither synchronises nor reads them, and
a captured call may be replayed after they have changed.
"""
from __future__ import annotations

import ctypes as C
import math

__all__ = [
    "rope_frequencies", "rotary", "rotary_backward", "paged_append", "attention_packed",
    "attention_packed_backward", "attention_paged", "blasst_seq_workspace_bytes",
    "blasst_packed_bwd_workspace_bytes",
]

_VP, _I, _LL, _F, _SZ = C.c_void_p, C.c_int, C.c_longlong, C.c_float, C.c_size_t


class RotaryArgs(C.Structure):
    _fields_ = ([(n, _VP) for n in ("x", "y", "positions", "freq")] +
                [(n, _I) for n in ("pos64", "B", "L", "H", "d", "rot")] +
                [(n, _LL) for n in ("x_sb", "x_sl", "x_sh", "y_sb", "y_sl", "y_sh", "pos_sb")] +
                [("interleaved", _I), ("inverse", _I), ("scale", _F), ("dtype", _I), ("stream", _VP)])


class AppendArgs(C.Structure):
    _fields_ = ([(n, _VP) for n in ("q", "q_out", "k", "v", "k_pages", "v_pages", "page_table",
                                    "kv_lens", "cu_q", "freq")] +
                [(n, _I) for n in ("n_seq", "T", "Hq", "Hkv", "d", "rot", "n_pages", "page_size",
                                   "table_width")] +
                [(n, _LL) for n in ("table_stride", "q_st", "q_sh", "qo_st", "qo_sh", "k_st", "k_sh",
                                    "v_st", "v_sh", "kp_sp", "kp_st", "kp_sh", "vp_sp", "vp_st",
                                    "vp_sh")] +
                [("interleaved", _I), ("scale", _F), ("dtype", _I), ("stream", _VP)])


class PackedArgs(C.Structure):
    _fields_ = ([(n, _VP) for n in ("q", "k", "v", "o", "lse", "cu_q", "cu_k")] +
                [(n, _I) for n in ("n_seq", "Tq", "Tk", "Hq", "Hkv", "d")] +
                [(n, _LL) for n in ("q_st", "q_sh", "k_st", "k_sh", "v_st", "v_sh")] +
                [("causal", _I), ("scale", _F), ("dtype", _I), ("workspace", _VP),
                 ("workspace_bytes", _SZ), ("stream", _VP)])


class PackedBwdArgs(C.Structure):
    _fields_ = ([(n, _VP) for n in ("q", "k", "v", "o", "dout", "lse", "dq", "dk", "dv", "cu_q",
                                    "cu_k")] +
                [(n, _I) for n in ("n_seq", "Tq", "Tk", "Hq", "Hkv", "d")] +
                [(n, _LL) for n in ("q_st", "q_sh", "k_st", "k_sh", "v_st", "v_sh", "o_st", "o_sh",
                                    "do_st", "do_sh")] +
                [("causal", _I), ("scale", _F), ("dtype", _I), ("workspace", _VP),
                 ("workspace_bytes", _SZ), ("stream", _VP)])


class PagedArgs(C.Structure):
    _fields_ = ([(n, _VP) for n in ("q", "k_pages", "v_pages", "o", "lse", "page_table", "kv_lens",
                                    "cu_q")] +
                [(n, _I) for n in ("n_seq", "Tq", "Hq", "Hkv", "d", "n_pages", "page_size",
                                   "table_width")] +
                [(n, _LL) for n in ("table_stride", "q_st", "q_sh", "kp_sp", "kp_st", "kp_sh",
                                    "vp_sp", "vp_st", "vp_sh")] +
                [("causal", _I), ("scale", _F), ("dtype", _I), ("workspace", _VP),
                 ("workspace_bytes", _SZ), ("stream", _VP)])


ENTRY_POINTS = {"blasst_rotary": RotaryArgs, "blasst_append": AppendArgs,
                "blasst_packed_fwd": PackedArgs, "blasst_packed_bwd": PackedBwdArgs,
                "blasst_paged_fwd": PagedArgs}

_dtypes = {}  # torch dtype -> blasst_dtype
_calls = {}   # entry point -> bound C function


def _bind():
    import torch
    from . import BLASST_BF16, BLASST_FP16, BLASST_FP32, load_library
    lib = load_library()
    for name, args in ENTRY_POINTS.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = [C.POINTER(args)], _I
        _calls[name] = f
    lib.blasst_seq_workspace_bytes.argtypes = [_I]
    lib.blasst_seq_workspace_bytes.restype = _SZ
    lib.blasst_packed_bwd_workspace_bytes.argtypes = [_I] * 3
    lib.blasst_packed_bwd_workspace_bytes.restype = _SZ
    _dtypes.update({torch.bfloat16: BLASST_BF16, torch.float32: BLASST_FP32,
                    torch.float16: BLASST_FP16})
    return lib


def _call(name, args):
    from . import _check
    _check(_calls[name](C.byref(args)), name)


def _on(fn):
    """Runs `fn` with its first tensor's device current (the C entry points
    launch on the current device) and refuses tensors of different devices."""
    import functools

    @functools.wraps(fn)
    def call(first, *rest, **kw):
        import torch
        if not _calls:
            _bind()
        if not first.is_cuda:
            raise ValueError("tensors passed to the CUDA library must live on a CUDA device")
        dev = first.get_device()
        for t in rest + tuple(kw.values()):
            if isinstance(t, torch.Tensor) and t.get_device() != dev:
                raise ValueError("tensors must live on one CUDA device")
        if dev == torch.cuda.current_device():
            return fn(first, *rest, **kw)
        with torch.cuda.device(dev):
            return fn(first, *rest, **kw)
    return call


def _stream_of(stream, *made):
    """The raw stream; tensors made here are handed to it (they were allocated
    for the current stream)."""
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    s = torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream
    for t in made:
        if t is not None:
            t.record_stream(s)
    return s.cuda_stream


def _dtype(t, *others):
    if t.dtype not in _dtypes:
        raise ValueError(f"dtype {t.dtype} is not supported")
    for o in others:
        if o.dtype != t.dtype:
            raise ValueError("tensors must have one dtype")
    return _dtypes[t.dtype]


def _rows(t, name, dims=3):
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t


def _strides(t):
    """(token, head) strides; a dimension of one entry gets a stride that fits
    (torch allows any there)."""
    st, sh = t.stride(0), t.stride(1)
    if t.shape[1] == 1:
        sh = t.shape[2]
    if t.shape[0] <= 1:
        st = max(sh * t.shape[1], t.shape[2])
    return st, sh


def _page_strides(t):
    sp, st, sh = t.stride(0), t.stride(1), t.stride(2)
    d = t.shape[3]
    if t.shape[2] == 1:
        sh = d
    if t.shape[1] == 1:
        st = d
    if t.shape[0] == 1:
        sp = t.shape[1] * t.shape[2] * d
    return sp, st, sh


def _index(t, name, n=None):
    import torch
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous one-dimensional int32 tensor")
    if n is not None and t.shape[0] != n:
        raise ValueError(f"{name} must have {n} entries")
    return t.data_ptr()


def _table(t, n):
    import torch
    if t.dtype != torch.int32 or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("page_table must be a two-dimensional int32 tensor with contiguous rows")
    if t.shape[0] != n:
        raise ValueError(f"page_table must have {n} rows")
    return t.data_ptr(), t.shape[1], t.stride(0) if t.shape[0] > 1 else t.shape[1]


def blasst_seq_workspace_bytes(d: int) -> int:
    """The C entry point of the same name (current device)."""
    if not _calls:
        _bind()
    from . import load_library
    return int(load_library().blasst_seq_workspace_bytes(int(d)))


def blasst_packed_bwd_workspace_bytes(Tq: int, Hq: int, Hkv: int) -> int:
    """The C entry point of the same name."""
    if not _calls:
        _bind()
    from . import load_library
    return int(load_library().blasst_packed_bwd_workspace_bytes(int(Tq), int(Hq), int(Hkv)))


_ws_bytes = {}  # (device, d) -> bytes


def _workspace(workspace, d, like):
    import torch
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        return workspace, workspace.numel() * workspace.element_size(), None
    key = (like.get_device(), d)
    n = _ws_bytes.get(key)
    if n is None:
        n = _ws_bytes[key] = max(16, blasst_seq_workspace_bytes(d))
    w = torch.empty(n, dtype=torch.uint8, device=like.device)
    return w, n, w


# ------------------------------------------------------------------- rotary
def rope_frequencies(rot, *, base=10000.0, scaling="none", factor=1.0, original_len=0,
                     low=None, high=None, device="cuda"):
    """Angle per position of each pair, float64 [rot / 2], and the factor for
    the turned dims. f_i = base^(-2 i / rot), then by ``scaling``:

      none    f_i;
      linear  f_i / factor (positions interpolated);
      ntk     base * factor^(rot / (rot - 2)) in the place of base;
      blend   pairs that turn at least ``high`` (32) times over ``original_len``
              positions are kept, those of at most ``low`` (1) turns divided by
              factor, a straight line over the pair's index between; factor for
              the dims 0.1 ln(factor) + 1;
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
            # pair index at which a pair turns n times over original_len positions
            at = lambda n: rot * math.log(original_len / (n * 2.0 * math.pi)) / (2.0 * math.log(base))  # noqa: E731
            first, last = max(math.floor(at(hi)), 0), min(math.ceil(at(lo)), rot // 2 - 1)
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


def _freq(inv_freq):
    import torch
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous one-dimensional float64 tensor")
    return inv_freq.data_ptr(), 2 * inv_freq.shape[0]


def _rotary(x, inv_freq, positions, interleaved, mscale, out, stream, inverse):
    import torch
    packed = x.dim() == 3
    _rows(x, "x", 3 if packed else 4)
    y = torch.empty_like(x, memory_format=torch.contiguous_format) if out is None else out
    _rows(y, "out", x.dim())
    if y.shape != x.shape:
        raise ValueError("out must have the shape of x")
    dt = _dtype(x, y)
    if packed:
        B, (L, H, d) = 1, x.shape
        xs, ys = (0, x.stride(0), x.stride(1)), (0, y.stride(0), y.stride(1))
    else:
        B, H, L, d = x.shape
        xs, ys = (x.stride(0), x.stride(2), x.stride(1)), (y.stride(0), y.stride(2), y.stride(1))
    pp, p64, psb = None, 0, 0
    if positions is not None:
        if positions.dtype not in (torch.int32, torch.int64):
            raise ValueError("positions must be int32 or int64")
        if tuple(positions.shape) not in ((L,), (B, L)):
            raise ValueError("positions must be [tokens], or [batch, tokens]")
        if L > 1 and positions.stride(-1) != 1:
            raise ValueError("positions must be contiguous in the last dimension")
        pp, p64 = positions.data_ptr(), int(positions.dtype == torch.int64)
        psb = positions.stride(0) if positions.dim() == 2 else 0
    fp, rot = _freq(inv_freq)
    s = _stream_of(stream, y if out is None else None)
    _call("blasst_rotary", RotaryArgs(x.data_ptr(), y.data_ptr(), pp, fp, p64, B, L, H, d, rot, *xs,
                                      *ys, psb, int(interleaved), inverse, mscale, dt, s))
    return y


def rotary(x, inv_freq, positions=None, *, interleaved=False, mscale=1.0, out=None, stream=None):
    """blasst_rotary: x [T, H, d] (packed) or [B, H, L, d] turned by
    ``positions`` ([T], or [L] / [B, L]; None: 0, 1, ...) times ``inv_freq``
    (``rope_frequencies``; its length gives the turned dims). ``out`` may be x."""
    return _rotary_on(x, inv_freq, positions, interleaved, mscale, out, stream, 0)


def rotary_backward(dy, inv_freq, positions=None, *, interleaved=False, mscale=1.0, out=None,
                    stream=None):
    """Gradient of ``rotary`` with respect to x: the transposed turn of dy."""
    return _rotary_on(dy, inv_freq, positions, interleaved, mscale, out, stream, 1)


_rotary_on = _on(_rotary)


def _paged_sizes(k_pages, v_pages, cu_q):
    _rows(k_pages, "k_pages", 4)
    _rows(v_pages, "v_pages", 4)
    if k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must have one shape")
    return cu_q.shape[0] - 1


@_on
def paged_append(q, k, v, k_pages, v_pages, page_table, kv_lens, cu_q, *, inv_freq=None,
                 interleaved=False, mscale=1.0, q_out=None, stream=None):
    """blasst_append: writes the new tokens' k (turned) and v [T, Hkv, d] into
    the pages and returns q [T, Hq, d] turned (into ``q_out``, which may be q).
    ``kv_lens`` counts each sequence's tokens with the new ones. Without
    ``inv_freq`` nothing is turned."""
    import torch
    n = _paged_sizes(k_pages, v_pages, cu_q)
    _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
    dt = _dtype(q, k, v, k_pages, v_pages)
    T, Hq, d = q.shape
    P, page, Hkv, _ = k_pages.shape
    if k.shape != (T, Hkv, d) or v.shape != (T, Hkv, d) or k_pages.shape[3] != d:
        raise ValueError("k and v must be [T, Hkv, d], the pages [pages, page, Hkv, d]")
    o = torch.empty_like(q, memory_format=torch.contiguous_format) if q_out is None else q_out
    _rows(o, "q_out")
    if o.shape != q.shape or o.dtype != q.dtype:
        raise ValueError("q_out must have q's shape and dtype")
    fp, rot = _freq(inv_freq) if inv_freq is not None else (None, 0)
    tp, width, ts = _table(page_table, n)
    s = _stream_of(stream, o if q_out is None else None)
    _call("blasst_append", AppendArgs(
        q.data_ptr(), o.data_ptr(), k.data_ptr(), v.data_ptr(), k_pages.data_ptr(),
        v_pages.data_ptr(), tp, _index(kv_lens, "kv_lens", n), _index(cu_q, "cu_q"), fp, n, T, Hq,
        Hkv, d, rot, P, page, width, ts, *_strides(q), *_strides(o), *_strides(k), *_strides(v),
        *_page_strides(k_pages), *_page_strides(v_pages), int(interleaved), mscale, dt, s))
    return o


# ---------------------------------------------------------------- attention
@_on
def attention_packed(q, k, v, cu_q, cu_k=None, *, causal=True, scale=0.0, workspace=None,
                     stream=None):
    """blasst_packed_fwd: exact attention of packed sequences, q [Tq, Hq, d],
    k, v [Tk, Hkv, d], ``cu_k`` None for cu_q. Returns (o [Tq, Hq, d],
    lse [Tq, Hq] fp32); tokens of no sequence are left unwritten."""
    import torch
    _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
    dt = _dtype(q, k, v)
    Tq, Hq, d = q.shape
    Tk, Hkv, dk = k.shape
    if dk != d or v.shape != k.shape:
        raise ValueError("k and v must be [Tk, Hkv, d] with q's d")
    n = cu_q.shape[0] - 1
    if cu_k is None:
        cu_k = cu_q
    o = torch.empty((Tq, Hq, d), dtype=q.dtype, device=q.device)
    lse = torch.empty((Tq, Hq), dtype=torch.float32, device=q.device)
    ws, nbytes, made = _workspace(workspace, d, q)
    s = _stream_of(stream, o, lse, made)
    _call("blasst_packed_fwd", PackedArgs(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
        _index(cu_q, "cu_q"), _index(cu_k, "cu_k", n + 1), n, Tq, Tk, Hq, Hkv, d, *_strides(q),
        *_strides(k), *_strides(v), int(bool(causal)), scale, dt, ws.data_ptr(), nbytes, s))
    return o, lse


@_on
def attention_packed_backward(q, k, v, o, lse, dout, cu_q, cu_k=None, *, causal=True, scale=0.0,
                              workspace=None, stream=None):
    """blasst_packed_bwd: gradients (dq, dk, dv) of ``attention_packed`` in the
    inputs' type, from its outputs o and lse and the gradient dout of o. Tokens
    of no sequence are left unwritten."""
    import torch
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _rows(t, name)
    dt = _dtype(q, k, v, o, dout)
    Tq, Hq, d = q.shape
    Tk, Hkv, dk_ = k.shape
    if dk_ != d or v.shape != k.shape:
        raise ValueError("k and v must be [Tk, Hkv, d] with q's d")
    if o.shape != q.shape or dout.shape != q.shape:
        raise ValueError("o and dout must have q's shape")
    if lse.dtype != torch.float32 or lse.shape != q.shape[:2] or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 tensor [Tq, Hq]")
    n = cu_q.shape[0] - 1
    if cu_k is None:
        cu_k = cu_q
    dq = torch.empty((Tq, Hq, d), dtype=q.dtype, device=q.device)
    dk = torch.empty((Tk, Hkv, d), dtype=q.dtype, device=q.device)
    dv = torch.empty((Tk, Hkv, d), dtype=q.dtype, device=q.device)
    made = None
    if workspace is None:
        nbytes = max(16, blasst_packed_bwd_workspace_bytes(Tq, Hq, Hkv))
        workspace = made = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    s = _stream_of(stream, dq, dk, dv, made)
    _call("blasst_packed_bwd", PackedBwdArgs(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(), lse.data_ptr(),
        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _index(cu_q, "cu_q"),
        _index(cu_k, "cu_k", n + 1), n, Tq, Tk, Hq, Hkv, d, *_strides(q), *_strides(k), *_strides(v),
        *_strides(o), *_strides(dout), int(bool(causal)), scale, dt, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), s))
    return dq, dk, dv


@_on
def attention_paged(q, k_pages, v_pages, page_table, kv_lens, cu_q, *, causal=True, scale=0.0,
                    workspace=None, stream=None):
    """blasst_paged_fwd: exact attention of new tokens q [T, Hq, d] (one or more
    per sequence) over the paged cache, which holds them already (``paged_append``).
    Returns (o [T, Hq, d], lse [T, Hq] fp32)."""
    import torch
    n = _paged_sizes(k_pages, v_pages, cu_q)
    _rows(q, "q")
    dt = _dtype(q, k_pages, v_pages)
    T, Hq, d = q.shape
    P, page, Hkv, dk = k_pages.shape
    if dk != d:
        raise ValueError("the pages must be [pages, page, Hkv, d] with q's d")
    o = torch.empty((T, Hq, d), dtype=q.dtype, device=q.device)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    ws, nbytes, made = _workspace(workspace, d, q)
    tp, width, ts = _table(page_table, n)
    s = _stream_of(stream, o, lse, made)
    _call("blasst_paged_fwd", PagedArgs(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), o.data_ptr(), lse.data_ptr(), tp,
        _index(kv_lens, "kv_lens", n), _index(cu_q, "cu_q"), n, T, Hq, Hkv, d, P, page, width, ts,
        *_strides(q), *_page_strides(k_pages), *_page_strides(v_pages), int(bool(causal)), scale, dt,
        ws.data_ptr(), nbytes, s))
    return o, lse
