"""torch-facing calls of the serving operators of the CUDA library.

``rope_frequencies`` / ``rope`` / ``rope_backward`` (rotary positions on Q and
K), ``cache_write`` / ``cache_read`` (the paged K/V cache, 16-bit or e4m3 with
one scale per row) and ``forward_tree`` (attention of drafted tokens over the
cache; one token per sequence is ordinary decoding).  As in ``attention``:
properties of the tensors are checked here, outputs and the workspace are
allocated with torch, and the library runs on the current CUDA stream of the
tensors' device.  A decoding step makes these calls for a few microseconds of
GPU work each, so a good call is told by one cheap test per tensor, and what is
wrong with a bad one is looked for only then.

One decoding step::

    q, k = rope(q, k, inv_freq, positions=positions)
    cache_write(k, v, k_cache, v_cache, ctx_lens, block_table=table,
                k_scale=k_scale, v_scale=v_scale)
    o, lse = forward_tree(q, k_cache, v_cache, ctx_lens, tree_mask=mask,
                          block_table=table, k_scale=k_scale, v_scale=v_scale)
"""

import ctypes
import functools
import math

import torch

from . import _lib
from .attention import _DTYPES, _E4M3, _check_inputs, _on_device

_I64x3 = ctypes.c_int64 * 3
_INT32 = torch.iinfo(torch.int32)
_WIDE = (torch.int64, torch.uint32, torch.uint64)   # integers past int32
_functions = {}      # the library's functions by name


def rope_frequencies(rot, base=10000.0, scaling=None, factor=1.0, original_len=None,
                     ramp=(1.0, 32.0), device=None):
    """Rotary frequencies of the rot / 2 pairs, float64, and the factor that
    the rotated values are multiplied by: ``(inv_freq, out_factor)``.

    f_i = base^(-2 i / rot).  ``scaling`` stretches them for contexts
    ``factor`` times longer than those trained on:

    * ``"linear"``: f_i / factor (positions interpolated);
    * ``"base"``: base replaced by base * factor^(rot / (rot - 2)), which
      leaves the fastest pair as it is and divides the slowest by ``factor``;
    * ``"ramp"``: by parts (Peng, Quesnelle, Fan, Shippole, "YaRN", 2023):
      with r_i = original_len f_i / (2 pi) turns over the trained length and
      g_i = clamp((r_i - low) / (high - low), 0, 1) for ``ramp`` = (low, high),
      f_i (g_i + (1 - g_i) / factor); out_factor = 1 + 0.1 ln factor.

    Elsewhere out_factor is 1.
    """
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and >= 2")
    if not factor >= 1.0:
        raise ValueError("factor must be >= 1")
    if scaling not in (None, "linear", "base", "ramp"):
        raise ValueError(f"scaling {scaling!r} is not one of None, 'linear', 'base', 'ramp'")
    if scaling == "base":
        if rot < 4:
            raise ValueError("scaling 'base' needs rot >= 4")
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    out_factor = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "ramp":
        if original_len is None:
            raise ValueError("scaling 'ramp' needs original_len")
        low, high = ramp
        if not low < high:
            raise ValueError("ramp must be (low, high) with low < high")
        g = ((original_len * f / (2.0 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        f = f * (g + (1.0 - g) / factor)
        out_factor = 1.0 + 0.1 * math.log(factor)
    return (f if device is None else f.to(device)), out_factor


def _ptr(t):
    return None if t is None else t.data_ptr()


def _strides(t):
    """Strides for the library: None if contiguous.  Dimensions of one element
    have no stride (torch gives them any)."""
    if t.is_contiguous():
        return None
    return _I64x3(*(s if n > 1 else 0 for n, s in zip(t.shape[:3], t.stride()[:3])))


def _check_strided(name, t, shape, dtype, device):
    if (torch.is_tensor(t) and t.is_cuda and t.dtype == dtype and t.shape == shape
            and t.device == device and t.stride(-1) == 1):
        return
    if not torch.is_tensor(t) or not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous in its last dimension")


def _check(name, t, shape, dtype, device):
    if not (torch.is_tensor(t) and t.is_cuda and t.dtype == dtype and t.shape == shape
            and t.device == device and t.is_contiguous()):
        if t is not None and not torch.is_tensor(t):
            raise ValueError(f"{name} must be a tensor")
        _check_inputs({name: t}, shape, dtype, device)


def _int32_arg(name, x, shape, device, other=None):
    """Device int32 tensor of the shape (or the other one); lists and host
    tensors are copied, and refused where a value does not fit.  Device tensors of
    wider integers are converted without a look at them from the host: values that
    do not fit become the nearest that do."""
    if x is None:
        return None
    if not (torch.is_tensor(x) and x.is_cuda and x.dtype == torch.int32 and x.device == device
            and x.is_contiguous()):
        _on_device(name, x, device)
        x = torch.as_tensor(x)
        if x.numel() and (x.is_floating_point() or x.is_complex() or x.dtype == torch.bool):
            raise ValueError(f"{name} has dtype {x.dtype}, expected integers")
        if x.dtype in _WIDE:
            x = x.to(torch.int64)
            low, high = _INT32.min, _INT32.max
            if x.device.type != "cpu":
                x = x.clamp(low, high)
            elif x.numel() and not low <= int(x.min()) <= int(x.max()) <= high:
                raise ValueError(f"{name} has values outside int32")
        x = x.to(device, torch.int32).contiguous()
    if x.shape != shape and (other is None or x.shape != other):
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected {tuple(shape)}"
                         + ("" if other is None else f" or {tuple(other)}"))
    return x


def _launch(name, device, *args):
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(_lib.load(), name)
    index = device.index
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index) or None)
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index) or None)
    if status:
        _lib.check(name, status)


def _rope(name, q, k, inv_freq, positions, interleaved, factor, q_out, k_out):
    packed = q.dim() == 3
    if packed:                                   # [H, T, d]: one batch of T rows
        q, k, q_out, k_out = (None if t is None else t.unsqueeze(0) for t in (q, k, q_out, k_out))
    if q.dim() != 4:
        raise ValueError("q must be [B, H, N, d] or packed [H, T, d]")
    shape = q.shape
    B, Hq, N, d = shape
    dev, dt = q.device, q.dtype
    code = _DTYPES.get(dt)
    if code is None:
        raise ValueError("dtype must be bfloat16 or float16")
    q_contiguous = q.is_contiguous()
    if not (q.is_cuda and (q_contiguous or q.stride(-1) == 1)):
        _check_strided("q", q, shape, dt, dev)
    if q_out is None:
        q_out = torch.empty_like(q) if q_contiguous else torch.empty(shape, dtype=dt, device=dev)
        q_out_strides = None
    else:
        _check_strided("q_out", q_out, shape, dt, dev)
        q_out_strides = _strides(q_out)
    Hk = 0
    k_ptr = k_out_ptr = k_strides = k_out_strides = None
    if k is not None:
        if not torch.is_tensor(k) or k.dim() != 4:
            raise ValueError("k must have as many dimensions as q")
        Hk = k.shape[1]
        shape = (B, Hk, N, d)
        _check_strided("k", k, shape, dt, dev)
        k_contiguous = k.is_contiguous()
        if k_out is None:
            k_out = torch.empty_like(k) if k_contiguous else torch.empty(shape, dtype=dt, device=dev)
        else:
            _check_strided("k_out", k_out, shape, dt, dev)
            k_out_strides = _strides(k_out)
        if not k_contiguous:
            k_strides = _strides(k)
        k_ptr, k_out_ptr = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    f = inv_freq
    if not (torch.is_tensor(f) and f.is_cuda and f.dtype == torch.float64 and f.device == dev
            and f.is_contiguous()):
        _on_device("inv_freq", inv_freq, dev)
        f = torch.as_tensor(f, dtype=torch.float64).to(dev).contiguous()
    if len(f.shape) != 1:
        raise ValueError("inv_freq must be [rot / 2]")
    pos = _int32_arg("positions", positions, (N,), dev, (B, N))
    _launch(name, dev, q.data_ptr(), None if q_contiguous else _strides(q), q_out.data_ptr(),
            q_out_strides, Hq, k_ptr, k_strides, k_out_ptr, k_out_strides, Hk, _ptr(pos),
            N if pos is not None and pos.dim() == 2 else 0, f.data_ptr(), B, N, d, 2 * f.shape[0],
            1 if interleaved else 0, factor, code)
    if packed:
        q_out, k_out = q_out[0], None if k_out is None else k_out[0]
    return q_out, k_out


def rope(q, k, inv_freq, positions=None, interleaved=False, factor=1.0, q_out=None, k_out=None):
    """q and k rotated by their positions: ``(q_out, k_out)``.

    q [B, Hq, N, d] and k [B, Hk, N, d] (or None), bf16/fp16, any strides with
    d contiguous and 16-byte aligned rows, or packed [H, T, d].  The first
    2 len(inv_freq) columns (a multiple of 16) are rotated, pairs being
    (2 i, 2 i + 1) if interleaved, else (i, i + rot / 2).  positions: int32 [N]
    or [B, N] (packed: [T]); None: 0 .. N - 1.  q_out, k_out: where the result
    goes (any strides; q and k themselves rotate in place), else new tensors.

    Here and below, int32 arguments may be lists, host tensors or device tensors
    of other integer types too.  Values that do not fit are refused on the host
    and become the nearest that fit on the device (no call waits for the GPU).
    """
    return _rope("fa_rope", q, k, inv_freq, positions, interleaved, factor, q_out, k_out)


def rope_backward(dq, dk, inv_freq, positions=None, interleaved=False, factor=1.0, q_out=None,
                  k_out=None):
    """Gradients of ``rope``'s inputs from those of its outputs (same
    inv_freq, positions, interleaved and factor)."""
    return _rope("fa_rope_bwd", dq, dk, inv_freq, positions, interleaved, factor, q_out, k_out)


def _cache_args(k_cache, v_cache, k_scale, v_scale, block_table, B, device):
    """Checks a cache; returns (Hk, page, d, format, block_table, arguments)."""
    if not torch.is_tensor(k_cache) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, Hk, page_size, d]")
    shape = k_cache.shape
    P, Hk, page, d = shape
    dt = k_cache.dtype
    if dt not in _E4M3 and dt not in _DTYPES:
        raise ValueError("k_cache must be float8_e4m3fn (or uint8 codes), bfloat16 or float16")
    _check("k_cache", k_cache, shape, dt, device)
    _check("v_cache", v_cache, shape, dt, device)
    if dt in _E4M3:
        shape = (P, Hk, page)
        _check("k_scale", k_scale, shape, torch.float32, device)
        _check("v_scale", v_scale, shape, torch.float32, device)
        fmt = _lib.FA_CACHE_E4M3
    else:
        if k_scale is not None or v_scale is not None:
            raise ValueError("a 16-bit cache has no scales")
        fmt = _lib.FA_CACHE_16
    stride = 1
    if block_table is not None:
        if not torch.is_tensor(block_table) or block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError(f"block_table must be an int32 tensor [{B}, pages per sequence]")
        block_table = _int32_arg("block_table", block_table, block_table.shape, device)
        stride = block_table.shape[1]
    elif P < B:
        raise ValueError("without a block_table sequence b is page b: num_pages >= B")
    return Hk, page, d, fmt, block_table, stride


def cache_write(k, v, k_cache, v_cache, start=None, lens=None, block_table=None, k_scale=None,
                v_scale=None):
    """Write rows of k, v [B, Hk, N, d] (bf16/fp16, strides as in ``rope``)
    into the cache, row n of sequence b at position start[b] + n for
    n < lens[b] (start None: 0; lens None: N).

    The cache is a pool of pages [num_pages, Hk, page_size, d] for K and for V:
    16-bit (k's dtype), or float8_e4m3fn (or uint8 codes) with k_scale, v_scale
    [num_pages, Hk, page_size] float32, one scale per row, which is quantised
    as it is written.  block_table: int32 [B, pages per sequence]; None: page b
    is sequence b.  Returns nothing: the cache (and scales) are updated.
    """
    if k.dim() != 4:
        raise ValueError("k must be [B, Hk, N, d]")
    B, _, N, _ = k.shape
    dev = k.device
    if k.dtype not in _DTYPES:
        raise ValueError("dtype must be bfloat16 or float16")
    Hk, page, d, fmt, table, stride = _cache_args(k_cache, v_cache, k_scale, v_scale, block_table,
                                                  B, dev)
    _check_strided("k", k, (B, Hk, N, d), k.dtype, dev)
    _check_strided("v", v, (B, Hk, N, d), k.dtype, dev)
    if fmt == _lib.FA_CACHE_16 and k_cache.dtype != k.dtype:
        raise ValueError(f"k has dtype {k.dtype}, the cache {k_cache.dtype}")
    start = _int32_arg("start", start, (B,), dev)
    lens = _int32_arg("lens", lens, (B,), dev)
    _launch("fa_cache_write", dev, k.data_ptr(), _strides(k), v.data_ptr(), _strides(v),
            k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_scale), _ptr(v_scale), _ptr(table),
            stride, _ptr(start), _ptr(lens), B, Hk, N, d, k_cache.shape[0], page, fmt,
            _DTYPES[k.dtype])


def cache_read(k_cache, v_cache, start, n, lens=None, block_table=None, k_scale=None,
               v_scale=None, dtype=None, k_out=None, v_out=None):
    """Rows start[b] .. start[b] + lens[b] - 1 of every sequence of the cache
    (start a tensor or list [B]; lens None: n) as ``(k, v)`` [B, Hk, n, d] in
    ``dtype`` (default: the cache's, bfloat16 for e4m3).  Rows behind lens[b] and
    rows of bad positions are left as they were in k_out, v_out, and are zero in
    new tensors."""
    if not torch.is_tensor(k_cache):
        raise ValueError("k_cache must be a CUDA tensor")
    if start is None:
        raise ValueError("start must be a tensor or a list [B]")
    dev = k_cache.device
    B = len(start)
    Hk, page, d, fmt, table, stride = _cache_args(k_cache, v_cache, k_scale, v_scale, block_table,
                                                  B, dev)
    if dtype is None:
        dtype = (k_out.dtype if k_out is not None
                 else torch.bfloat16 if fmt == _lib.FA_CACHE_E4M3 else k_cache.dtype)
    if dtype not in _DTYPES:
        raise ValueError("dtype must be bfloat16 or float16")
    if fmt == _lib.FA_CACHE_16 and dtype != k_cache.dtype:
        raise ValueError(f"a {k_cache.dtype} cache is read back as {k_cache.dtype}")
    # new tensors are cleared by the kernel, beside one that is given by torch
    both = k_out is None and v_out is None
    new = torch.empty if both else torch.zeros
    k_out = new((B, Hk, n, d), dtype=dtype, device=dev) if k_out is None else k_out
    v_out = new((B, Hk, n, d), dtype=dtype, device=dev) if v_out is None else v_out
    _check("k_out", k_out, (B, Hk, n, d), dtype, dev)
    _check("v_out", v_out, (B, Hk, n, d), dtype, dev)
    start = _int32_arg("start", start, (B,), dev)
    lens = _int32_arg("lens", lens, (B,), dev)
    _launch("fa_cache_read", dev, k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_scale),
            _ptr(v_scale), k_out.data_ptr(), v_out.data_ptr(), _ptr(table), stride, _ptr(start),
            _ptr(lens), B, Hk, n, d, k_cache.shape[0], page, fmt | _lib.FA_CACHE_CLEAR if both else fmt,
            _DTYPES[dtype])
    return k_out, v_out


def tree_workspace_bytes(B, Hq, Hk, T, d):
    return _lib.fa_fwd_tree_workspace_size(B, Hq, Hk, T, d)


_tree_workspace_bytes = functools.lru_cache(maxsize=256)(tree_workspace_bytes)


def forward_tree(q, k_cache, v_cache, ctx_lens, draft_lens=None, tree_mask=None, block_table=None,
                 k_scale=None, v_scale=None, scale=None, out=None, lse=None, workspace=None):
    """O, LSE of the drafted tokens q [B, Hq, T, d] (bf16/fp16) over a cache.

    Sequence b has ctx_lens[b] positions of context, then the rows of its
    drafted tokens (both written by ``cache_write``).  Query t sees the whole
    context and the drafted tokens u with tree_mask[t, u] != 0 (uint8 or bool
    [T, T], or [B, T, T]; None: u <= t).  T = 1 is ordinary decoding.  Hq may be
    a multiple of the cache's Hk (shared K/V heads).  draft_lens [B]: how many
    of the T tokens a sequence has; rows behind them are left as they were in
    out and lse, and are O = 0, LSE = -inf in new tensors (as are tokens past the
    positions of the table, which are reported).  Cache and block_table as in
    ``cache_write``; a v_scale should be what its row's codes need, as there,
    since one far above it costs the other keys bits.
    """
    if q.dim() != 4:
        raise ValueError("q must be [B, Hq, T, d]")
    B, Hq, T, d = q.shape
    dev = q.device
    if q.dtype not in _DTYPES:
        raise ValueError("dtype must be bfloat16 or float16")
    shape, dt = q.shape, q.dtype
    _check("q", q, shape, dt, dev)
    Hk, page, dc, fmt, table, stride = _cache_args(k_cache, v_cache, k_scale, v_scale, block_table,
                                                   B, dev)
    if dc != d:
        raise ValueError(f"the cache has d = {dc}, q has d = {d}")
    if Hk == 0 or Hq % Hk:
        raise ValueError(f"{Hq} query heads do not share {Hk} K/V heads evenly")
    if fmt == _lib.FA_CACHE_16 and k_cache.dtype != q.dtype:
        raise ValueError(f"q has dtype {q.dtype}, the cache {k_cache.dtype}")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    full = draft_lens is None and T <= stride * page     # every row has a result
    if out is None:
        out = torch.empty_like(q) if full else torch.zeros_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, T), dtype=torch.float32, device=dev)
        if not full:
            lse.fill_(-math.inf)
    _check("out", out, shape, dt, dev)
    _check("lse", lse, (B, Hq, T), torch.float32, dev)
    ctx = _int32_arg("ctx_lens", ctx_lens, (B,), dev)
    if ctx is None:
        raise ValueError("ctx_lens is None")
    drafts = _int32_arg("draft_lens", draft_lens, (B,), dev)
    mask = None
    if tree_mask is not None:
        mask = tree_mask
        if not (torch.is_tensor(mask) and mask.is_cuda and mask.device == dev
                and mask.dtype in (torch.uint8, torch.bool) and mask.is_contiguous()):
            _on_device("tree_mask", tree_mask, dev)
            if torch.as_tensor(mask).is_floating_point():  # (0 and -inf would mean the opposite)
                raise ValueError("tree_mask must be uint8 or bool: nonzero where a query sees a key")
            mask = (torch.as_tensor(mask) != 0).to(dev).contiguous()
        if mask.shape != (T, T) and mask.shape != (B, T, T):
            raise ValueError(f"tree_mask must be [{T}, {T}] or [{B}, {T}, {T}]")
    if workspace is None:
        workspace = q.new_empty(_tree_workspace_bytes(B, Hq, Hk, T, d), dtype=torch.uint8)
    elif not (torch.is_tensor(workspace) and workspace.is_cuda and workspace.device == dev
              and workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous CUDA tensor on {dev}")
    _launch("fa_fwd_tree", dev, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
            _ptr(k_scale), _ptr(v_scale), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _ptr(table), stride, ctx.data_ptr(),
            _ptr(drafts), _ptr(mask), int(mask is not None and mask.dim() == 3), B, Hq, Hk, T, d,
            k_cache.shape[0], page, scale, fmt, _DTYPES[q.dtype])
    return out, lse
