"""Binding of the core-attention entry points (``include/spin.h``): rotary
positions, the paged latent cache and the attention that reads it.

Argument marshalling only, as in the package itself: every function has the
name of the C entry point it calls.  Tensors may be strided where the C call
takes strides (queries, new tokens); everything else is contiguous.  A call
runs on the device of its :class:`SpinLatent` and on that device's current
stream, whichever device is current; all tensors must live there.
"""
from __future__ import annotations

import ctypes
import sys
from typing import Optional

import torch

__all__ = [
    "SpinLatentConfig", "SpinLatent", "make_latent_config", "spin_latent_bytes", "spin_rope", "spin_latent_append",
    "spin_latent_attention", "spin_latent_prefill", "spin_latent_error", "SPIN_ROPE_INTERLEAVED", "SPIN_ROPE_HALF",
    "SPIN_ROPE_PLAIN", "SPIN_ROPE_LINEAR", "SPIN_ROPE_YARN",
]

SPIN_ROPE_INTERLEAVED, SPIN_ROPE_HALF = 0, 1  # which elements form a pair
SPIN_ROPE_PLAIN, SPIN_ROPE_LINEAR, SPIN_ROPE_YARN = 0, 1, 2  # frequency scaling

_vp, _i32, _i64, _u32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32


class SpinLatentConfig(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("num_requests", "max_slots", "block_size", "num_heads", "latent_dim", "rope_dim",
                                    "nope_dim", "v_dim", "topk", "max_rows", "prefill_slots", "dtype", "rope_layout",
                                    "rope_scaling", "rope_original")] + \
               [(n, ctypes.c_float) for n in ("softmax_scale", "beta_fast", "beta_slow", "attn_factor")] + \
               [("reserved", _i32), ("rope_base", ctypes.c_double), ("rope_factor", ctypes.c_double)]


_CFG = ctypes.POINTER(SpinLatentConfig)
SIGNATURES = {
    "spin_latent_bytes": (ctypes.c_size_t, [_CFG]),
    "spin_latent_create": (ctypes.c_int, [_CFG, _vp, ctypes.c_size_t, _vp, ctypes.POINTER(_vp)]),
    "spin_latent_destroy": (ctypes.c_int, [_vp]),
    "spin_rope": (ctypes.c_int, [_vp, _i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp, _i64, _i64, _vp, _vp, _i64,
                                 _i64, _vp]),
    "spin_latent_append": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i64, _vp, _i64, _vp, _i32, _vp, _i32, _vp, _vp,
                                          _vp]),
    "spin_latent_attention": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i32, _vp, _i32, _vp, _i64, _i64, _vp, _i64,
                                             _i64, _vp, _vp, _vp, _vp, _vp]),
    "spin_latent_prefill": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i32, _vp, _i32, _vp, _i64, _i64, _vp, _vp, _vp,
                                           _vp, _vp]),
    "spin_latent_error": (ctypes.c_int, [_vp, _vp, ctypes.POINTER(_u32)]),
}


def _pkg():
    """The package itself (it imports this module, so not at the top)."""
    return sys.modules[__package__]


def make_latent_config(*, num_requests, max_slots, block_size=64, num_heads=128, latent_dim=512, rope_dim=64,
                       nope_dim=128, v_dim=128, topk=2048, max_rows=1, prefill_slots=0, bf16=True, softmax_scale=None,
                       rope_layout=SPIN_ROPE_INTERLEAVED, rope_base=10000.0, rope_scaling=SPIN_ROPE_PLAIN,
                       rope_factor=1.0, rope_original=4096, beta_fast=32.0, beta_slow=1.0,
                       attn_factor=0.0) -> SpinLatentConfig:
    """``softmax_scale`` None: (nope_dim + rope_dim) ** -0.5."""
    isa = _pkg()
    if softmax_scale is None:
        softmax_scale = (nope_dim + rope_dim) ** -0.5
    return SpinLatentConfig(num_requests, max_slots, block_size, num_heads, latent_dim, rope_dim, nope_dim, v_dim,
                            topk, max_rows, prefill_slots, isa.SPIN_BF16 if bf16 else isa.SPIN_F32, rope_layout,
                            rope_scaling, rope_original, softmax_scale, beta_fast, beta_slow, attn_factor, 0,
                            rope_base, rope_factor)


def spin_latent_bytes(cfg: SpinLatentConfig) -> int:
    return int(_pkg().load().spin_latent_bytes(ctypes.byref(cfg)))


class SpinLatent:
    """A handle of the latent-attention calls: the config, its rotary
    frequencies, the device error word and the scratch, in one device buffer
    allocated with PyTorch and handed to ``spin_latent_create``."""

    def __init__(self, cfg: SpinLatentConfig, device="cuda", stream=None):
        isa = _pkg()
        lib = isa.load()
        self.cfg = cfg
        nbytes = lib.spin_latent_bytes(ctypes.byref(cfg))
        if nbytes == 0:
            raise isa.SpinError(1, "spin_latent_bytes (invalid config)")
        self.nbytes = nbytes
        self.dtype = torch.bfloat16 if cfg.dtype == isa.SPIN_BF16 else torch.float32
        self.mem = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
        self.device = self.mem.device
        self._derive()
        off = (-self.mem.data_ptr()) % 256
        self.base = self.mem[off:off + nbytes]
        h = _vp()
        isa._check(lib.spin_latent_create(ctypes.byref(cfg), _vp(self.base.data_ptr()), nbytes,
                                          _stream(self, stream), ctypes.byref(h)), "spin_latent_create")
        self.handle = h

    def _derive(self):
        """What the calls' checks compare with, taken from the config once."""
        c = self.cfg
        self.index = -1 if self.device.type == "cpu" else self.device.index
        self.requests, self.heads, self.latent, self.rope = c.num_requests, c.num_heads, c.latent_dim, c.rope_dim
        self.page = (c.block_size, c.latent_dim + c.rope_dim)
        self.blocks = -(-c.max_slots // c.block_size)
        self.per_request = (c.num_requests,)

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            _pkg().load().spin_latent_destroy(self.handle)
            self.handle = _vp(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _stream(lt: SpinLatent, stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(lt.index)
    if stream.device != lt.device:
        raise ValueError(f"the stream is on {stream.device}, the handle on {lt.device}")
    return stream.cuda_stream


# Each check is one expression where everything is as it should be (these run
# in every call), and the reason is looked for only where it is not.
def _refuse(lt: SpinLatent, t: torch.Tensor, name: str, dtype, shape: tuple):
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != lt.index:
        raise ValueError(f"{name} must be on {lt.device}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _dense(lt: SpinLatent, t: Optional[torch.Tensor], name: str, dtype, shape: tuple) -> Optional[int]:
    """The address of a contiguous tensor of exactly this shape (None: a NULL pointer)."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == lt.index and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _refuse(lt, t, name, dtype, shape)


def _tokens(lt: SpinLatent, t: torch.Tensor, name: str, shape: tuple):
    """(address, token stride, head stride) of a tensor [Q, rows, (heads,) width] whose tokens lie at one stride."""
    st = t.stride()
    if t.dtype is not lt.dtype or t.get_device() != lt.index or t.shape != shape:
        _refuse(lt, t, name, lt.dtype, shape)
    if st[-1] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    Q, rows = shape[0], shape[1]
    if rows > 1:
        token = st[1]
        if Q > 1 and st[0] != rows * token:
            raise ValueError(f"the rows of all requests of {name} must lie at one stride")
    else:
        token = st[0] if Q > 1 else 0
    return t.data_ptr(), token, st[2] if len(shape) == 4 and shape[2] > 1 else 0


def _cache(lt: SpinLatent, cache: torch.Tensor, block_table: torch.Tensor):
    if cache.dim() != 3:
        raise ValueError("cache must have the shape (pages, block_size, latent_dim + rope_dim)")
    if block_table.dim() != 2:
        raise ValueError("block_table must have the shape (num_requests, blocks)")
    pages, columns = cache.shape[0], block_table.shape[1]
    if columns < lt.blocks:
        raise ValueError(f"block_table must have at least {lt.blocks} columns, got {columns}")
    return (_dense(lt, cache, "cache", lt.dtype, (pages, *lt.page)), pages,
            _dense(lt, block_table, "block_table", torch.int32, (lt.requests, columns)), columns)


def _steps(*dims):
    """(stride, size) of those of the dimensions that have more than one place, the smallest stride first."""
    return sorted(d for d in dims if d[1] > 1)


def _overlap(a: torch.Tensor, b: torch.Tensor, dims: Optional[tuple]) -> bool:
    """Whether two tensors [.., .., width] of one shape share an element.
    ``dims``: (stride, size) of the outer dimensions, where both tensors have
    these strides and their rows do not overlap; None: the answer is whether
    the byte ranges meet."""
    def span(t):
        last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
        return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()
    (a0, a1), (b0, b1) = span(a), span(b)
    if a.numel() == 0 or a0 >= b1 or b0 >= a1:
        return False
    if dims is None or (b0 - a0) % a.element_size():
        return True
    # a row of a against one of b, n places of a dimension apart: as all rows behind a dimension fit its stride, only
    # the two n whose rows are nearest can meet
    apart = [(b0 - a0) // a.element_size()]
    for step, size in reversed(_steps(*dims)):
        apart = [d - n * step for d in apart for n in (d // step, d // step + 1) if abs(n) < size]
    return any(abs(d) < a.shape[-1] for d in apart)


# --------------------------------------------------------------------------
# entry points (same names as the C ABI)
# --------------------------------------------------------------------------
def _call(name: str, *args) -> None:
    status = getattr(_pkg().load(), name)(*args)
    if status != 0:
        raise _pkg().SpinError(status, name)


def spin_rope(lt: SpinLatent, x: torch.Tensor, positions: torch.Tensor, offset: int = 0,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rotates elements offset .. offset + rope_dim - 1 of every head of x
    [tokens, heads, head_dim] by its token's position; ``out`` None: in place.
    Where the memory of out lies among that of x (parts of one packed tensor),
    they have the same strides.  Returns the tensor it wrote."""
    out = x if out is None else out
    shape = x.shape
    if len(shape) != 3 or out.shape != shape:
        raise ValueError("x and out must have one shape (tokens, heads, head_dim)")
    if x.dtype is not lt.dtype or x.get_device() != lt.index:
        _refuse(lt, x, "x", lt.dtype, shape)
    tokens, heads, width = shape
    sx = x.stride()
    xt, xh = sx[0] if tokens > 1 else 0, sx[1] if heads > 1 else 0
    if out is x:
        so, ot, oh = sx, xt, xh
    else:
        if out.dtype is not lt.dtype or out.get_device() != lt.index:
            _refuse(lt, out, "out", lt.dtype, shape)
        so = out.stride()
        ot, oh = so[0] if tokens > 1 else 0, so[1] if heads > 1 else 0
    if sx[2] != 1 or so[2] != 1:
        raise ValueError("the last dimension of x and out must be contiguous")
    # heads of out one behind the other, in either order of tokens and heads
    if not (oh >= width and ot >= oh * (heads - 1) + width):
        reach = width
        for step, n in _steps((ot, tokens), (oh, heads)):
            if step < reach:
                raise ValueError("the heads of out must not overlap")
            reach += step * (n - 1)
    if out is not x and (out.data_ptr() != x.data_ptr() or ot != xt or oh != xh) and _overlap(
            x, out, ((ot, tokens), (oh, heads)) if ot == xt and oh == xh else None):
        raise ValueError("out must be x or not overlap it")
    _call("spin_rope", lt.handle, tokens, heads, width, offset, x.data_ptr(), xt, xh,
          _dense(lt, positions, "positions", torch.int32, (tokens,)), out.data_ptr(), ot, oh, _stream(lt, stream))
    return out


def spin_latent_append(lt: SpinLatent, rows: int, c: torch.Tensor, k_rope: torch.Tensor, cache: torch.Tensor,
                       block_table: torch.Tensor, ctx_len: torch.Tensor, row_count: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    """Writes c [Q, rows, latent_dim] and the rotated k_rope [Q, rows,
    rope_dim] into slots ctx_len - 1 .. of each request."""
    cp, ct, _ = _tokens(lt, c, "c", (lt.requests, rows, lt.latent))
    kp, kt, _ = _tokens(lt, k_rope, "k_rope", (lt.requests, rows, lt.rope))
    _call("spin_latent_append", lt.handle, rows, cp, ct, kp, kt, *_cache(lt, cache, block_table),
          _dense(lt, ctx_len, "ctx_len", torch.int32, lt.per_request),
          _dense(lt, row_count, "row_count", torch.int32, lt.per_request),
          _stream(lt, stream))


def spin_latent_attention(lt: SpinLatent, rows: int, cache: torch.Tensor, block_table: torch.Tensor,
                          q_latent: torch.Tensor, q_rope: torch.Tensor, ctx_len: torch.Tensor,
                          topk: Optional[torch.Tensor], out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                          stream=None) -> None:
    """Absorbed attention of q_latent [Q, rows, H, latent_dim], q_rope [Q,
    rows, H, rope_dim] over the slots that topk [Q, rows, k] lists (None: all
    visible ones) into out [Q, rows, H, latent_dim] and lse [Q, rows, H]."""
    cfg = lt.cfg
    Q, H = lt.requests, lt.heads
    ql = _tokens(lt, q_latent, "q_latent", (Q, rows, H, lt.latent))
    qr = _tokens(lt, q_rope, "q_rope", (Q, rows, H, lt.rope))
    _call("spin_latent_attention", lt.handle, rows, *_cache(lt, cache, block_table), *ql, *qr,
          _dense(lt, ctx_len, "ctx_len", torch.int32, lt.per_request),
          _dense(lt, topk, "topk", torch.int32, (Q, rows, cfg.topk)),
          _dense(lt, out, "out", lt.dtype, (Q, rows, H, lt.latent)),
          _dense(lt, lse, "lse", torch.float32, (Q, rows, H)), _stream(lt, stream))


def spin_latent_prefill(lt: SpinLatent, rows: int, cache: torch.Tensor, block_table: torch.Tensor, q: torch.Tensor,
                        w_kv: torch.Tensor, ctx_len: torch.Tensor, row_count: Optional[torch.Tensor],
                        out: torch.Tensor, stream=None) -> None:
    """Expanded attention of a chunk q [Q, rows, H, nope_dim + rope_dim] over
    the context its tokens were appended to, into out [Q, rows, H, v_dim]."""
    cfg = lt.cfg
    Q, H = cfg.num_requests, cfg.num_heads
    if not cfg.prefill_slots:
        raise _pkg().SpinError(7, "spin_latent_prefill (the handle has no prefill_slots)")
    qp = _tokens(lt, q, "q", (Q, rows, H, cfg.nope_dim + cfg.rope_dim))
    _call("spin_latent_prefill", lt.handle, rows, *_cache(lt, cache, block_table), *qp,
          _dense(lt, w_kv, "w_kv", lt.dtype, (H, cfg.nope_dim + cfg.v_dim, cfg.latent_dim)),
          _dense(lt, ctx_len, "ctx_len", torch.int32, lt.per_request),
          _dense(lt, row_count, "row_count", torch.int32, lt.per_request),
          _dense(lt, out, "out", lt.dtype, (Q, rows, H, cfg.v_dim)), _stream(lt, stream))


def spin_latent_error(lt: SpinLatent, stream=None):
    """Returns (status, raw device error word) and clears it; synchronises the stream."""
    word = _u32()
    status = _pkg().load().spin_latent_error(lt.handle, _stream(lt, stream), ctypes.byref(word))
    return int(status), int(word.value)
