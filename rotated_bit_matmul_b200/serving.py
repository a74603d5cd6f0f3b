"""Torch-facing binding of the serving operators of libharp.so (include/harp.h): residual RMS
norm with an optional 8-bit output, the 8-bit linear, rotary positions with the write into a
paged key-value cache, and attention of one new token over that cache.

As in the package's other wrappers only marshalling happens here. Calls run on the tensors'
device, on its current stream. Outputs and scratch come from torch's allocator, call by call,
so calls on several streams and captured graphs do not share any.
"""
from __future__ import annotations

import ctypes
import math

import torch

from ._lib import KVCache, call, check, load

BLOCK = 128  # columns that share one 8-bit scale
E4M3 = torch.float8_e4m3fn
_DT = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "ramp": 4}
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else None
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


def _device(*ts) -> int:
    """The index of the one CUDA device that the tensors share."""
    dev = ts[0].device
    for t in ts:
        if t is not None and (not t.is_cuda or t.device != dev):
            raise ValueError("rotated_bit_matmul_b200 works on CUDA tensors of one device only")
    return dev.index


def _launch(name, dev, *args):
    """Calls the entry point with the current stream of device `dev` as its last argument.
    (Callers return before it on empty inputs, which have no address.)"""
    fn = getattr(load(), name)
    if _current_device() == dev:
        st = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(dev))
    if st:
        check(st, name)


def _dtype(t, what) -> int:
    code = _DT.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be float32, bfloat16 or float16, not {t.dtype}")
    return code


def _rows(t):
    """t as rows of its last dimension, contiguous inside a row, on a 16-byte boundary."""
    if t.dim() != 2:
        t = t.reshape(-1, t.shape[-1])
    if (t.stride(1) != 1 and t.shape[1] > 1) or t.data_ptr() & 15 or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        t = t.clone(memory_format=torch.contiguous_format)
    return t


def _stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _target(t, shape, what):
    """An output the caller passed: rows of the given shape, contiguous inside a row, where it lies."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    v = t if t.dim() == 2 else t.view(-1, t.shape[-1])
    if (v.shape[1] > 1 and v.stride(1) != 1) or v.data_ptr() & 15 or (v.shape[0] > 1 and v.stride(0) < v.shape[1]):
        raise ValueError(f"{what} must hold its rows contiguously, on a 16-byte boundary")
    return v


def _norm_inputs(x, weight, residual, residual_out, eps):
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x needs a last dimension of at least one column")
    n = x.shape[-1]
    x2 = _rows(x)
    w = r = h = None
    if weight is not None:
        if weight.shape != (n,):
            raise ValueError(f"weight must have shape ({n},)")
        w = weight if weight.data_ptr() & 15 == 0 and (n == 1 or weight.stride(0) == 1) else weight.clone(
            memory_format=torch.contiguous_format)
    if residual is not None:
        if residual.shape != x.shape:
            raise ValueError("residual must have x's shape")
        r = _rows(residual)
        if residual_out is None:
            residual_out = torch.empty(x.shape, dtype=residual.dtype, device=x.device)
        elif residual_out.dtype != residual.dtype:
            raise ValueError("residual_out must have the residual's dtype")
        h = _target(residual_out, x.shape, "residual_out")
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    rt = _dtype(residual, "residual") if r is not None else 0
    args = (x2.shape[0], n, eps, x2.data_ptr(), _dtype(x, "x"), _stride(x2), r.data_ptr() if r is not None else None, rt,
            _stride(r) if r is not None else 0, w.data_ptr() if w is not None else None,
            _dtype(w, "weight") if w is not None else 0, h.data_ptr() if h is not None else None,
            _stride(h) if h is not None else 0)
    return args, (x2, w, r, h), residual_out


def harp_rmsnorm(x, weight=None, residual=None, eps=1e-5, out_dtype=None, out=None, residual_out=None):
    """y = h / sqrt(mean(h^2) + eps) * weight over the last dimension, h = x + residual.

    Returns y (out_dtype, default x's), and with a residual (y, h): h rounded to the residual's
    dtype, in residual_out when given (which may be the residual itself)."""
    dev = _device(x, weight, residual, out, residual_out)
    args, keep, h = _norm_inputs(x, weight, residual, residual_out, eps)
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
    o = _target(out, x.shape, "out")
    if args[0]:
        _launch("harp_rmsnorm", dev, *args, o.data_ptr(), _dtype(out, "out"), _stride(o))
    return out if residual is None else (out, h)


def _q8_outputs(rows, n, device):
    """e4m3 rows on 16-byte boundaries, and scales [rows, blocks] held block by block."""
    q = torch.empty_strided((rows, n), ((n + 15) & ~15, 1), dtype=E4M3, device=device)
    scale = torch.empty_strided((rows, -(-n // BLOCK)), (1, (rows + 3) & ~3), dtype=torch.float32, device=device)
    return q, scale


def _lead(t, shape):
    return t if len(shape) == 2 else t.unflatten(0, shape[:-1]) if len(shape) > 2 else t[0]


def harp_rmsnorm_q8(x, weight=None, residual=None, eps=1e-5, residual_out=None):
    """harp_rmsnorm with an 8-bit output: (q, scale), with a residual (q, scale, h).

    q: float8_e4m3fn of x's shape, rows padded to 16 bytes; scale: fp32 [..., ceil(n / 128)],
    max |y| / 448 of every row and 128 columns, held block by block as HarpLinear8 reads it."""
    dev = _device(x, weight, residual, residual_out)
    args, keep, h = _norm_inputs(x, weight, residual, residual_out, eps)
    rows, n = keep[0].shape
    q, scale = _q8_outputs(rows, n, x.device)
    if rows:
        _launch("harp_rmsnorm_q8", dev, *args, q.data_ptr(), q.stride(0), scale.data_ptr(), scale.stride(1))
    if x.dim() != 2:
        q, scale = _lead(q, x.shape), _lead(scale, x.shape)
    return (q, scale) if residual is None else (q, scale, h)


def harp_quantize_q8(x):
    """(q, scale) of x itself, as harp_rmsnorm_q8 lays them out."""
    dev = _device(x)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x needs a last dimension of at least one column")
    x2 = _rows(x)
    q, scale = _q8_outputs(*x2.shape, x.device)
    if x2.shape[0]:
        _launch("harp_quantize_q8", dev, *x2.shape, x2.data_ptr(), _dtype(x, "x"), _stride(x2), q.data_ptr(), q.stride(0),
                scale.data_ptr(), scale.stride(1))
    return (q, scale) if x.dim() == 2 else (_lead(q, x.shape), _lead(scale, x.shape))


def harp_quantize_weights_q8(W):
    """e4m3 codes [n_out, n_in] and fp32 scales [ceil(n_out / 128), ceil(n_in / 128)] of a weight
    matrix, a scale per 128 x 128 block, as HarpLinear8 takes them."""
    dev = _device(W)
    if W.dim() != 2 or not W.numel():
        raise ValueError("W must be a matrix")
    W = _rows(W)
    n_out, n_in = W.shape
    q = torch.empty_strided((n_out, n_in), ((n_in + 15) & ~15, 1), dtype=E4M3, device=W.device)
    scale = torch.empty((-(-n_out // BLOCK), -(-n_in // BLOCK)), dtype=torch.float32, device=W.device)
    _launch("harp_quantize_weights_q8", dev, n_out, n_in, W.data_ptr(), _dtype(W, "W"), _stride(W), q.data_ptr(),
            q.stride(0), scale.data_ptr())
    return q, scale


def _wide_rows(q):
    """e4m3 rows on 16-byte boundaries (a copy where they are not)."""
    if q.data_ptr() & 15 or (q.shape[1] > 1 and q.stride(1) != 1) or (
            q.shape[0] > 1 and (q.stride(0) & 15 or q.stride(0) < q.shape[1])):
        w = torch.empty_strided(q.shape, ((q.shape[1] + 15) & ~15, 1), dtype=E4M3, device=q.device)
        w.view(torch.uint8).copy_(q.view(torch.uint8))
        return w
    return q


def _wide_stride(q):
    return q.stride(0) if q.shape[0] > 1 else (q.shape[1] + 15) & ~15


class HarpLinear8:
    """An 8-bit linear on the device (wraps harp_create_layer8): codes float8_e4m3fn
    [n_out, n_in] and fp32 scale [ceil(n_out / 128), ceil(n_in / 128)], as
    harp_quantize_weights_q8 returns them. Both are kept, not copied, when they are laid out so."""

    def __init__(self, codes, scale):
        self.handle = None
        dev = _device(codes, scale)
        if codes.dim() != 2 or codes.dtype != E4M3 or not codes.numel():
            raise ValueError("codes must be a float8_e4m3fn matrix")
        self.n_out, self.n_in = codes.shape
        want = (-(-self.n_out // BLOCK), -(-self.n_in // BLOCK))
        if scale.dtype != torch.float32 or tuple(scale.shape) != want:
            raise ValueError(f"scale must be float32 {want}")
        self.codes, self.scale = _wide_rows(codes), scale.contiguous()
        if self.scale.data_ptr() & 15:
            self.scale = self.scale.clone()
        self.device = codes.device
        self._blocks = want[1]
        h = ctypes.c_void_p()
        _launch("harp_create_layer8", dev, ctypes.byref(h), self.n_in, self.n_out, self.codes.data_ptr(),
                _wide_stride(self.codes), self.scale.data_ptr())
        self.handle = h

    def __call__(self, x, scale, out_dtype=torch.bfloat16, out=None):
        """y = (x * scale) @ W.T for e4m3 rows x [..., n_in] with fp32 scales [..., blocks]."""
        dev = _device(x, scale, self.codes, out)
        if x.dtype != E4M3 or x.dim() < 1 or x.shape[-1] != self.n_in:
            raise ValueError(f"x must be float8_e4m3fn with rows of {self.n_in}")
        if scale.dtype != torch.float32 or scale.shape != (*x.shape[:-1], self._blocks):
            raise ValueError(f"scale must be float32 {(*x.shape[:-1], self._blocks)}")
        x2, s2 = x, scale
        if x.dim() != 2:
            x2, s2 = x.reshape(-1, self.n_in), scale.reshape(-1, self._blocks)
        x2 = _wide_rows(x2)
        rows = x2.shape[0]
        ld = s2.stride(1) if self._blocks > 1 else (rows + 3) & ~3
        if (rows > 1 and s2.stride(0) != 1) or ld & 3 or ld < rows or s2.data_ptr() & 15:
            t = torch.empty_strided(s2.shape, (1, (rows + 3) & ~3), dtype=torch.float32, device=x.device)
            t.copy_(s2)
            s2, ld = t, (rows + 3) & ~3
        if out is None:
            out = torch.empty((*x.shape[:-1], self.n_out), dtype=out_dtype, device=x.device)
            o = out if out.dim() == 2 else out.view(rows, self.n_out)
        else:
            o = _target(out, (*x.shape[:-1], self.n_out), "out")
        if rows:
            _launch("harp_linear8_fwd", dev, self.handle, rows, x2.data_ptr(), _wide_stride(x2), s2.data_ptr(), ld,
                    o.data_ptr(), _dtype(out, "out"), _stride(o))
        return out

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            call("harp_destroy_layer8", self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class HarpCache:
    """A paged key-value cache over two bf16 or f16 tensors of one layout, kept and not copied:
    k, v [n_pages, n_kv_heads, page_size, head_dim], or with the layers in front. Any strides in
    multiples of 8 with a contiguous head_dim, so a transposed view of [n_pages, page_size,
    n_kv_heads, head_dim] works too. page_size is a power of two."""

    def __init__(self, k, v):
        self._device = _device(k, v)
        if k.dim() not in (4, 5) or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride():
            raise ValueError("k and v must be 4- or 5-dimensional and agree in shape, dtype and strides")
        if k.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("the cache holds bfloat16 or float16")
        if k.stride(-1) != 1:
            raise ValueError("head_dim must be contiguous")
        self.k, self.v = k, v
        self.n_layers = k.shape[0] if k.dim() == 5 else 1
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape[-4:]
        self.dtype, self.device = k.dtype, k.device
        self.layer_stride = k.stride(0) if k.dim() == 5 else 0
        self._layers = [
            KVCache(k.data_ptr() + 2 * i * self.layer_stride, v.data_ptr() + 2 * i * self.layer_stride, _DT[k.dtype],
                    self.n_kv_heads, self.head_dim, self.page_size, self.n_pages, k.stride(-4), k.stride(-3), k.stride(-2))
            for i in range(self.n_layers)]
        self._refs = [ctypes.addressof(s) for s in self._layers]

    @classmethod
    def empty(cls, n_layers, n_pages, n_kv_heads, page_size, head_dim, dtype=torch.bfloat16, device="cuda"):
        """A cache of zeros for n_layers layers."""
        shape = (n_layers, n_pages, n_kv_heads, page_size, head_dim)
        return cls(torch.zeros(shape, dtype=dtype, device=device), torch.zeros(shape, dtype=dtype, device=device))

    def layer(self, i=0):
        """Address of layer i's harp_kv_cache."""
        return self._refs[i]


def _index(t, what, dim):
    if t.dtype != torch.int32 or t.dim() != dim:
        raise ValueError(f"{what} must be a {dim}-dimensional int32 tensor")
    return t if t.is_contiguous() else t.contiguous()


def _heads(t, what):
    if t.dim() != 3:
        raise ValueError(f"{what} must be [tokens, heads, head_dim]")
    return t if t.stride(2) == 1 or t.shape[2] == 1 else t.contiguous()


class HarpRope:
    """Rotary positions for heads of head_dim, the first rot_dim of them turned (default all).

    interleaved: pairs (2 i, 2 i + 1), else (i, i + rot_dim / 2). base, scaling ("none", "linear",
    "ntk", "bands", "ramp"), factor, original, low, high: harp_rope_frequencies; or frequencies,
    rot_dim / 2 radians per position. amplitude multiplies cos and sin."""

    def __init__(self, head_dim, rot_dim=None, interleaved=False, base=10000.0, scaling="none", factor=1.0, original=0.0,
                 low=1.0, high=32.0, amplitude=1.0, frequencies=None):
        self.handle = None
        rot_dim = head_dim if rot_dim is None else rot_dim
        self.head_dim, self.rot_dim = int(head_dim), int(rot_dim)
        f = (ctypes.c_double * max(1, self.rot_dim // 2))()
        if frequencies is not None:
            values = [float(x) for x in frequencies]
            if len(values) != self.rot_dim // 2:
                raise ValueError(f"{self.rot_dim // 2} frequencies are needed, not {len(values)}")
            f[:] = values
        else:
            if scaling not in _SCALINGS:
                raise ValueError(f"scaling must be one of {', '.join(_SCALINGS)}")
            call("harp_rope_frequencies", self.rot_dim, float(base), _SCALINGS[scaling], float(factor), float(original),
                 float(low), float(high), f)
        self.frequencies = list(f)
        h = ctypes.c_void_p()
        call("harp_rope_create", ctypes.byref(h), self.head_dim, self.rot_dim, int(bool(interleaved)), f, float(amplitude))
        self.handle = h

    def __call__(self, x, positions, inverse=False, out_dtype=None, out=None):
        """x [tokens, heads, head_dim] turned by int32 positions [tokens] (inverse: back, which is
        also the gradient). Rows of negative positions are left as they were in out."""
        dev = _device(x, positions, out)
        x = _heads(x, "x")
        positions = _index(positions, "positions", 1)
        if x.shape[0] != positions.shape[0] or x.shape[2] != self.head_dim:
            raise ValueError(f"x must be [{positions.shape[0]}, heads, {self.head_dim}]")
        if out is None:
            out = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
        elif out.shape != x.shape or out.stride(2) != 1:
            raise ValueError("out must have x's shape with a contiguous head_dim")
        if x.numel():
            _launch("harp_rope_apply", dev, self.handle, x.shape[0], x.shape[1], positions.data_ptr(), x.data_ptr(),
                    _dtype(x, "x"), x.stride(0), x.stride(1), out.data_ptr(), _dtype(out, "out"), out.stride(0),
                    out.stride(1), int(bool(inverse)))
        return out

    def append(self, cache, q, k, v, positions, page_table, seq_ids=None, layer=0, out=None, out_dtype=None):
        """Turned q (default: in the cache's dtype), with turned k and v written to the cache at every
        token's position (one launch; wraps harp_rope_append). Token t belongs to sequence
        seq_ids[t], or t; page_table int32 [sequences, pages]."""
        dev = _device(q, k, v, positions, page_table, seq_ids, cache.k, out)
        q, k, v = _heads(q, "q"), _heads(k, "k"), _heads(v, "v")
        positions, page_table = _index(positions, "positions", 1), _index(page_table, "page_table", 2)
        ids = None
        tokens = positions.shape[0]
        if seq_ids is not None:
            seq_ids = _index(seq_ids, "seq_ids", 1)
            if seq_ids.shape[0] != tokens:
                raise ValueError("seq_ids must have a sequence for every token")
            ids = seq_ids.data_ptr()
        kv = (tokens, cache.n_kv_heads, cache.head_dim)
        if q.shape[0] != tokens or q.shape[2] != self.head_dim or k.shape != kv or v.shape != kv:
            raise ValueError(f"q must be [{tokens}, heads, {self.head_dim}], k and v {list(kv)}")
        if k.dtype != q.dtype or v.dtype != q.dtype:
            raise ValueError("q, k and v must share a dtype")
        if out is None:
            out = torch.empty(q.shape, dtype=out_dtype or cache.dtype, device=q.device)
        elif out.shape != q.shape or out.stride(2) != 1:
            raise ValueError("out must have q's shape with a contiguous head_dim")
        if tokens:
            _launch("harp_rope_append", dev, self.handle, cache.layer(layer), tokens, q.shape[1], positions.data_ptr(), ids,
                    page_table.shape[0], page_table.data_ptr(), page_table.shape[1], q.data_ptr(), q.stride(0), q.stride(1),
                    k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), _dtype(q, "q"),
                    out.data_ptr(), _dtype(out, "out"), out.stride(0), out.stride(1))
        return out

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            call("harp_rope_destroy", self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_attention_ws = {}


def harp_paged_attention_workspace_bytes(head_dim: int) -> int:
    n = _attention_ws.get(head_dim)
    if n is None:
        b = ctypes.c_size_t()
        call("harp_paged_attention_workspace_size", int(head_dim), ctypes.byref(b))
        n = _attention_ws[head_dim] = b.value
    return n


def harp_paged_attention(q, cache, page_table, seq_lens, layer=0, scale=None, window=0, return_lse=False, out=None,
                         workspace=None):
    """Attention of one new token per sequence, q [sequences, heads, head_dim], over its first
    seq_lens[s] cached positions (window > 0: the last `window` of them), scaled by `scale`
    (default head_dim^-1/2). With return_lse also the fp32 log-sum-exp [sequences, heads]. A
    sequence of length 0 gives zeros; rows of negative length are left as they were in out."""
    dev = _device(q, page_table, seq_lens, cache.k, out, workspace)
    page_table, seq_lens = _index(page_table, "page_table", 2), _index(seq_lens, "seq_lens", 1)
    q = _heads(q, "q")
    n, heads, dim = q.shape
    if page_table.shape[0] != n or seq_lens.shape[0] != n or dim != cache.head_dim:
        raise ValueError(f"q [{n}, heads, {dim}] does not match page_table, seq_lens or the cache's head_dim")
    if q.dtype != cache.dtype:
        raise ValueError("q must have the cache's dtype")
    if q.data_ptr() & 3 or q.stride(0) & 1 or q.stride(1) & 1:
        q = q.clone(memory_format=torch.contiguous_format)
    if out is None:
        out = torch.empty((n, heads, dim), dtype=q.dtype, device=q.device)
    elif out.shape != q.shape or out.dtype != q.dtype or out.stride(2) != 1:
        raise ValueError("out must have q's shape and dtype with a contiguous head_dim")
    if workspace is None:
        workspace = torch.empty(harp_paged_attention_workspace_bytes(dim), dtype=torch.uint8, device=q.device)
    lse = torch.empty((n, heads), dtype=torch.float32, device=q.device) if return_lse else None
    if not n:
        return (out, lse) if return_lse else out
    _launch("harp_paged_attention", dev, cache.layer(layer), n, heads, q.data_ptr(), q.stride(0), q.stride(1),
            page_table.data_ptr(), page_table.shape[1], seq_lens.data_ptr(), dim ** -0.5 if scale is None else scale, window,
            out.data_ptr(), out.stride(0), out.stride(1), lse.data_ptr() if return_lse else None, workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    return (out, lse) if return_lse else out
