"""CPU-only checks of the latent-attention entry points: handle sizes against
the documented layout, refused configs and arguments (before anything is
launched), and the binding's shape, stride and overlap checks.  No call here
touches a GPU: where a handle is needed, the binding's checks run against one
that was never created, and they refuse before the library is reached."""
import ctypes
import itertools

import pytest
import torch

import indexer_sparse_attention_b200 as isa
from indexer_sparse_attention_b200 import build as isa_build
from indexer_sparse_attention_b200 import latent


@pytest.fixture(scope="module")
def lib():
    isa_build.build()
    return isa.load()


def _cfg(**over):
    base = dict(num_requests=3, max_slots=1000, num_heads=16, topk=256, max_rows=4, prefill_slots=1024)
    base.update(over)
    return isa.make_latent_config(**base)


def _expected_bytes(H, dc, dr, dn, dv, cap, el):
    a = lambda x: (x + 255) // 256 * 256
    heads = max(2 * 148 * min(64, -(-H // 16) * 16), 2 * 296 * 8)  # shares: two per block, of the larger kernel
    parts = 148 * 256 if cap else 0  # rows of the expanded form's parts, in the same place
    return a(16) + a(64 * 8) + a(max(heads, parts) * 8) + a(max(heads * dc, parts * dv) * 4) + a(cap * H * (dn + dv) * el) + a(cap * dr * el) \
        + a(cap // 128 * H * 4)


@pytest.mark.parametrize("over", [{}, {"num_heads": 128}, {"num_heads": 1}, {"bf16": False}, {"prefill_slots": 0},
                                  {"latent_dim": 64, "rope_dim": 32, "nope_dim": 8, "v_dim": 256}])
def test_bytes_match_the_documented_parts(lib, over):
    c = _cfg(**over)
    assert isa.spin_latent_bytes(c) == _expected_bytes(c.num_heads, c.latent_dim, c.rope_dim, c.nope_dim, c.v_dim,
                                                       c.prefill_slots, 2 if c.dtype == isa.SPIN_BF16 else 4)


@pytest.mark.parametrize("over", [
    {"num_requests": 0}, {"num_requests": 16384}, {"max_slots": 0}, {"block_size": 8}, {"block_size": 48},
    {"block_size": 512}, {"num_heads": 0}, {"num_heads": 257}, {"latent_dim": 520}, {"latent_dim": 500},
    {"latent_dim": 0}, {"rope_dim": 136}, {"rope_dim": 4}, {"topk": 0}, {"topk": 65537}, {"max_rows": 0},
    {"max_rows": 5}, {"prefill_slots": -128}, {"prefill_slots": 100}, {"nope_dim": 264}, {"v_dim": 0},
    {"softmax_scale": 0.0}, {"softmax_scale": float("nan")}, {"softmax_scale": float("inf")}, {"rope_layout": 2},
    {"rope_scaling": 3}, {"rope_base": 1.0}, {"rope_base": float("inf")},
    {"rope_scaling": 1, "rope_factor": 0.5}, {"rope_scaling": 2, "rope_original": 0},
    {"rope_scaling": 2, "beta_fast": 1.0}, {"rope_scaling": 2, "beta_slow": 0.0},
    {"rope_scaling": 2, "attn_factor": -1.0}, {"max_slots": 2**31 - 1, "num_requests": 16383},
    {"max_slots": 2**30 + 1, "num_requests": 1}])
def test_invalid_configs_are_refused(lib, over):
    c = _cfg(**over)
    assert isa.spin_latent_bytes(c) == 0
    h = ctypes.c_void_p(77)
    assert lib.spin_latent_create(ctypes.byref(c), ctypes.c_void_p(4096), 1 << 40, ctypes.c_void_p(0),
                                  ctypes.byref(h)) == 1 and not h.value


def test_a_softmax_scale_that_is_infinite_in_log2_units_is_refused(lib):
    assert isa.spin_latent_bytes(_cfg(softmax_scale=2.3e38)) > 0
    assert isa.spin_latent_bytes(_cfg(softmax_scale=2.4e38)) == 0


def test_a_handle_without_prefill_ignores_its_dims(lib):
    assert isa.spin_latent_bytes(_cfg(prefill_slots=0, nope_dim=0, v_dim=0, softmax_scale=0.1)) > 0


def test_create_refuses_bad_blocks_without_a_device(lib):
    c = _cfg()
    h = ctypes.c_void_p()
    create = lambda at, n: lib.spin_latent_create(ctypes.byref(c), ctypes.c_void_p(at), n, ctypes.c_void_p(0),
                                                  ctypes.byref(h))
    assert create(0, 1 << 40) == 1          # NULL
    assert create(4096 + 16, 1 << 40) == 1  # misaligned
    assert create(4096, isa.spin_latent_bytes(c) - 1) == 2
    assert lib.spin_latent_destroy(None) == 4


def test_every_call_answers_a_null_handle(lib):
    for name, (res, args) in latent.SIGNATURES.items():
        if name in ("spin_latent_bytes", "spin_latent_create"):
            continue
        pointer = lambda t: t is ctypes.c_void_p or issubclass(t, ctypes._Pointer)
        assert getattr(lib, name)(*[None if pointer(t) else 0 for t in args]) == 4, name


class _NoHandle:
    """What the binding's checks look at, on the CPU."""

    def __init__(self, cfg, dtype=torch.bfloat16):
        self.cfg, self.dtype, self.device, self.handle = cfg, dtype, torch.device("cpu"), None
        isa.SpinLatent._derive(self)


def _args(cfg, rows=2, dtype=torch.bfloat16):
    Q, H, W = cfg.num_requests, cfg.num_heads, cfg.latent_dim + cfg.rope_dim
    blocks = -(-cfg.max_slots // cfg.block_size)
    z = lambda *shape, t=dtype: torch.zeros(shape, dtype=t)
    return dict(cache=z(Q * blocks, cfg.block_size, W), block_table=z(Q, blocks, t=torch.int32),
                q_latent=z(Q, rows, H, cfg.latent_dim), q_rope=z(Q, rows, H, cfg.rope_dim),
                ctx_len=z(Q, t=torch.int32), topk=z(Q, rows, cfg.topk, t=torch.int32),
                out=z(Q, rows, H, cfg.latent_dim), lse=z(Q, rows, H, t=torch.float32))


def _bad(t, how):
    if how == "dtype":
        return t.to(torch.float16) if t.is_floating_point() else t.long()
    if how == "shape":
        return torch.zeros((*t.shape[:-1], t.shape[-1] + 1), dtype=t.dtype)
    return torch.zeros((*t.shape, 2), dtype=t.dtype)[..., 0]  # last dimension strided


@pytest.mark.parametrize("name", ["cache", "block_table", "q_latent", "q_rope", "ctx_len", "topk", "out", "lse"])
@pytest.mark.parametrize("how", ["dtype", "shape", "strided"])
def test_attention_refuses_wrong_tensors(lib, name, how):
    if (name, how) == ("block_table", "shape"):
        pytest.skip("a wider block table is fine")
    cfg = _cfg()
    a = _args(cfg)
    a[name] = _bad(a[name], how)
    with pytest.raises(ValueError, match=name):
        isa.spin_latent_attention(_NoHandle(cfg), 2, **a)


def test_attention_refuses_a_short_block_table_and_uneven_rows(lib):
    cfg = _cfg()
    a = _args(cfg)
    a["block_table"] = a["block_table"][:, :-1].contiguous()
    with pytest.raises(ValueError, match="block_table"):
        isa.spin_latent_attention(_NoHandle(cfg), 2, **a)
    a = _args(cfg)
    a["q_latent"] = torch.zeros((3, 3, 16, 512), dtype=torch.bfloat16)[:, :2]  # a gap after each request
    with pytest.raises(ValueError, match="stride"):
        isa.spin_latent_attention(_NoHandle(cfg), 2, **a)


def test_rope_refuses_wrong_tensors(lib):
    lt = _NoHandle(_cfg())
    x = torch.zeros((5, 4, 128), dtype=torch.bfloat16)
    pos = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError):
        isa.spin_rope(lt, x.float(), pos)
    with pytest.raises(ValueError):
        isa.spin_rope(lt, x, pos.long())
    with pytest.raises(ValueError):
        isa.spin_rope(lt, x, pos[:4])
    with pytest.raises(ValueError):
        isa.spin_rope(lt, x[0], pos)
    with pytest.raises(ValueError):
        isa.spin_rope(lt, x, pos, out=torch.zeros((5, 4, 120), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="overlap"):  # heads on top of one another
        isa.spin_rope(lt, torch.zeros((5, 1, 128), dtype=torch.bfloat16).expand(5, 4, 128), pos)
    big = torch.zeros(5 * 4 * 128 + 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="overlap"):
        isa.spin_rope(lt, big[:-64].view(5, 4, 128), pos, out=big[64:].view(5, 4, 128))


@pytest.mark.parametrize("shape,strides", [((5, 4, 8), (64, 16, 1)), ((5, 4, 8), (40, 8, 1)), ((3, 4, 8), (10, 50, 1)),
                                           ((1, 6, 8), (0, 19, 1)), ((6, 1, 8), (19, 0, 1)), ((1, 1, 8), (0, 0, 1)),
                                           ((4, 3, 8), (33, 11, 1))])
def test_overlap_of_views_with_the_same_strides(shape, strides):
    """Every distance of two views against the sets of their elements."""
    room = torch.zeros(2000, dtype=torch.bfloat16)
    at = lambda first: torch.as_strided(room, shape, strides, first)
    cells = lambda first: {first + sum(i * s for i, s in zip(place, strides))
                           for place in itertools.product(*map(range, shape))}
    dims = tuple(zip(strides[:2], shape[:2]))
    for distance in range(-500, 500):
        meet = bool(cells(700) & cells(700 + distance))
        assert latent._overlap(at(700), at(700 + distance), dims) == meet, distance
        assert latent._overlap(at(700), at(700 + distance), None) >= meet


def test_rope_takes_parts_of_one_packed_tensor(lib, monkeypatch):
    """Queries and their rotated copies side by side, per head and per token; the same a step closer overlap."""
    lt = _NoHandle(_cfg())
    monkeypatch.setattr(latent, "_stream", lambda lt, stream: None)
    pos = torch.zeros(5, dtype=torch.int32)
    room = torch.zeros((5, 4, 256), dtype=torch.bfloat16)
    by_token = torch.zeros((5, 8, 128), dtype=torch.bfloat16)
    for x, out in ((room[..., :128], room[..., 128:]), (room[..., 128:], room[..., :128]),
                   (by_token[:, :4], by_token[:, 4:]), (room[..., :64], room[..., 64:128])):
        with pytest.raises(isa.SpinError) as e:  # past the checks: the library has no handle
            isa.spin_rope(lt, x, pos, out=out)
        assert e.value.status == 4
    for x, out in ((room[..., :128], room[..., 120:248]), (by_token[:, :5], by_token[:, 3:]),
                   (room[..., :128], room.view(5, 8, 128)[:, 1:5])):
        with pytest.raises(ValueError, match="overlap"):
            isa.spin_rope(lt, x, pos, out=out)


def test_prefill_without_slots_is_refused(lib):
    cfg = _cfg(prefill_slots=0)
    with pytest.raises(isa.SpinError) as e:
        isa.spin_latent_prefill(_NoHandle(cfg), 1, None, None, None, None, None, None, None)
    assert e.value.status == 7
