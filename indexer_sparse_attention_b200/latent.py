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
    import indexer_sparse_attention_b200 as isa
    return isa


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
        off = (-self.mem.data_ptr()) % 256
        self.base = self.mem[off:off + nbytes]
        h = _vp()
        isa._check(lib.spin_latent_create(ctypes.byref(cfg), _vp(self.base.data_ptr()), nbytes,
                                          _stream(self, stream), ctypes.byref(h)), "spin_latent_create")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            _pkg().load().spin_latent_destroy(self.handle)
            self.handle = _vp(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _stream(lt: SpinLatent, stream) -> _vp:
    if stream is None:
        stream = torch.cuda.current_stream(lt.device)
    elif stream.device != lt.device:
        raise ValueError(f"the stream is on {stream.device}, the handle on {lt.device}")
    return _vp(stream.cuda_stream)


def _place(lt: SpinLatent, t: torch.Tensor, name: str, dtype) -> None:
    if t.device != lt.device:
        raise ValueError(f"{name} must be on {lt.device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _dense(lt: SpinLatent, t: Optional[torch.Tensor], name: str, dtype, shape) -> _vp:
    """A contiguous tensor of exactly this shape (None: a NULL pointer)."""
    if t is None:
        return _vp(0)
    _place(lt, t, name, dtype)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _vp(t.data_ptr())


def _stride(t: torch.Tensor, dim: int) -> int:
    return t.stride(dim) if t.shape[dim] > 1 else 0


def _tokens(lt: SpinLatent, t: torch.Tensor, name: str, shape):
    """(pointer, token stride, head stride) of a tensor [Q, rows, (heads,) width] whose tokens lie at one stride."""
    _place(lt, t, name, lt.dtype)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.stride(-1) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    Q, rows = t.shape[:2]
    if Q > 1 and rows > 1 and t.stride(0) != rows * t.stride(1):
        raise ValueError(f"the rows of all requests of {name} must lie at one stride")
    token = _stride(t, 1) if rows > 1 else _stride(t, 0)
    return _vp(t.data_ptr()), token, _stride(t, 2) if t.dim() == 4 else 0


def _cache(lt: SpinLatent, cache: torch.Tensor, block_table: torch.Tensor):
    c = lt.cfg
    if cache.dim() != 3:
        raise ValueError("cache must have the shape (pages, block_size, latent_dim + rope_dim)")
    if block_table.dim() != 2:
        raise ValueError("block_table must have the shape (num_requests, blocks)")
    blocks = -(-c.max_slots // c.block_size)
    if block_table.shape[1] < blocks:
        raise ValueError(f"block_table must have at least {blocks} columns, got {block_table.shape[1]}")
    return (_dense(lt, cache, "cache", lt.dtype, (cache.shape[0], c.block_size, c.latent_dim + c.rope_dim)),
            cache.shape[0],
            _dense(lt, block_table, "block_table", torch.int32, (c.num_requests, block_table.shape[1])),
            block_table.shape[1])


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether the byte ranges of two tensors meet."""
    def span(t):
        last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
        return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()
    (a0, a1), (b0, b1) = span(a), span(b)
    return a.numel() > 0 and b.numel() > 0 and a0 < b1 and b0 < a1


# --------------------------------------------------------------------------
# entry points (same names as the C ABI)
# --------------------------------------------------------------------------
def spin_rope(lt: SpinLatent, x: torch.Tensor, positions: torch.Tensor, offset: int = 0,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rotates elements offset .. offset + rope_dim - 1 of every head of x
    [tokens, heads, head_dim] by its token's position; ``out`` None: in place.
    Returns the tensor it wrote."""
    isa = _pkg()
    out = x if out is None else out
    if x.dim() != 3 or out.shape != x.shape:
        raise ValueError("x and out must have one shape (tokens, heads, head_dim)")
    for t, name in ((x, "x"), (out, "out")):
        _place(lt, t, name, lt.dtype)
        if t.stride(-1) != 1:
            raise ValueError(f"the last dimension of {name} must be contiguous")
    if any(n > 1 and s < w for n, s, w in ((x.shape[0], out.stride(0), 1), (x.shape[1], out.stride(1), x.shape[2]))):
        raise ValueError("the heads of out must not overlap")
    same = out.data_ptr() == x.data_ptr() and all(_stride(out, d) == _stride(x, d) for d in (0, 1))
    if not same and _overlap(x, out):
        raise ValueError("out must be x or not overlap it")
    pos = _dense(lt, positions, "positions", torch.int32, x.shape[:1])
    isa._check(isa.load().spin_rope(lt.handle, x.shape[0], x.shape[1], x.shape[2], offset, _vp(x.data_ptr()),
                                    _stride(x, 0), _stride(x, 1), pos, _vp(out.data_ptr()), _stride(out, 0),
                                    _stride(out, 1), _stream(lt, stream)), "spin_rope")
    return out


def spin_latent_append(lt: SpinLatent, rows: int, c: torch.Tensor, k_rope: torch.Tensor, cache: torch.Tensor,
                       block_table: torch.Tensor, ctx_len: torch.Tensor, row_count: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    """Writes c [Q, rows, latent_dim] and the rotated k_rope [Q, rows,
    rope_dim] into slots ctx_len - 1 .. of each request."""
    isa = _pkg()
    cfg = lt.cfg
    Q = cfg.num_requests
    cp, ct, _ = _tokens(lt, c, "c", (Q, rows, cfg.latent_dim))
    kp, kt, _ = _tokens(lt, k_rope, "k_rope", (Q, rows, cfg.rope_dim))
    isa._check(isa.load().spin_latent_append(
        lt.handle, rows, cp, ct, kp, kt, *_cache(lt, cache, block_table),
        _dense(lt, ctx_len, "ctx_len", torch.int32, (Q,)), _dense(lt, row_count, "row_count", torch.int32, (Q,)),
        _stream(lt, stream)), "spin_latent_append")


def spin_latent_attention(lt: SpinLatent, rows: int, cache: torch.Tensor, block_table: torch.Tensor,
                          q_latent: torch.Tensor, q_rope: torch.Tensor, ctx_len: torch.Tensor,
                          topk: Optional[torch.Tensor], out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                          stream=None) -> None:
    """Absorbed attention of q_latent [Q, rows, H, latent_dim], q_rope [Q,
    rows, H, rope_dim] over the slots that topk [Q, rows, k] lists (None: all
    visible ones) into out [Q, rows, H, latent_dim] and lse [Q, rows, H]."""
    isa = _pkg()
    cfg = lt.cfg
    Q, H = cfg.num_requests, cfg.num_heads
    ql = _tokens(lt, q_latent, "q_latent", (Q, rows, H, cfg.latent_dim))
    qr = _tokens(lt, q_rope, "q_rope", (Q, rows, H, cfg.rope_dim))
    isa._check(isa.load().spin_latent_attention(
        lt.handle, rows, *_cache(lt, cache, block_table), *ql, *qr,
        _dense(lt, ctx_len, "ctx_len", torch.int32, (Q,)), _dense(lt, topk, "topk", torch.int32, (Q, rows, cfg.topk)),
        _dense(lt, out, "out", lt.dtype, (Q, rows, H, cfg.latent_dim)),
        _dense(lt, lse, "lse", torch.float32, (Q, rows, H)), _stream(lt, stream)), "spin_latent_attention")


def spin_latent_prefill(lt: SpinLatent, rows: int, cache: torch.Tensor, block_table: torch.Tensor, q: torch.Tensor,
                        w_kv: torch.Tensor, ctx_len: torch.Tensor, row_count: Optional[torch.Tensor],
                        out: torch.Tensor, stream=None) -> None:
    """Expanded attention of a chunk q [Q, rows, H, nope_dim + rope_dim] over
    the context its tokens were appended to, into out [Q, rows, H, v_dim]."""
    isa = _pkg()
    cfg = lt.cfg
    Q, H = cfg.num_requests, cfg.num_heads
    if not cfg.prefill_slots:
        raise isa.SpinError(7, "spin_latent_prefill (the handle has no prefill_slots)")
    qp = _tokens(lt, q, "q", (Q, rows, H, cfg.nope_dim + cfg.rope_dim))
    isa._check(isa.load().spin_latent_prefill(
        lt.handle, rows, *_cache(lt, cache, block_table), *qp,
        _dense(lt, w_kv, "w_kv", lt.dtype, (H, cfg.nope_dim + cfg.v_dim, cfg.latent_dim)),
        _dense(lt, ctx_len, "ctx_len", torch.int32, (Q,)), _dense(lt, row_count, "row_count", torch.int32, (Q,)),
        _dense(lt, out, "out", lt.dtype, (Q, rows, H, cfg.v_dim)), _stream(lt, stream)), "spin_latent_prefill")


def spin_latent_error(lt: SpinLatent, stream=None):
    """Returns (status, raw device error word) and clears it; synchronises the stream."""
    word = _u32()
    status = _pkg().load().spin_latent_error(lt.handle, _stream(lt, stream), ctypes.byref(word))
    return int(status), int(word.value)
