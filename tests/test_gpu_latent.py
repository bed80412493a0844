"""Latent-attention operators on the GPU against their formulas in 64 bits:
rotary positions, the cache append, absorbed attention (top-k lists and whole
contexts) and expanded attention of a chunk, over dtypes, widths, head counts,
lengths, page sizes and strides, with masked places full of NaN, empty rows,
bad lengths and pages, other streams, captured graphs, and a whole layer run
with the indexer's own top-k."""
import decimal
import math

import pytest
import torch

import indexer_sparse_attention_b200 as isa
import latent_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from indexer_sparse_attention_b200 import build
    build.build()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=BF16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def handle(Q, max_slots, *, poison=True, **over):
    """A handle whose scratch holds NaN: nothing may be read before it is written."""
    over.setdefault("softmax_scale", 0.0722)
    lt = isa.SpinLatent(isa.make_latent_config(num_requests=Q, max_slots=max_slots, **over))
    if poison:
        lt.base[768:] = 255  # behind the error word and the rotary frequencies
    return lt


def pages(g, Q, max_slots, b, spare=3):
    blocks = -(-max_slots // b)
    return torch.randperm(Q * blocks + spare, generator=g, device="cuda")[:Q * blocks].to(torch.int32).view(Q, blocks)


def nan_cache(bt, b, width, dtype, spare=3):
    return torch.full((bt.numel() + spare, b, width), math.nan, dtype=dtype, device="cuda")


def put(cache, bt, q, slots, values):
    b = cache.shape[1]
    cache[bt[q].long()[slots // b], slots % b] = values


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
ROPE = [
    # tokens, heads, head_dim, offset, rope_dim, half, dtype, scaling
    (1, 1, 64, 0, 64, False, BF16, {}),
    (96, 64, 128, 64, 64, False, BF16, {}),
    (7, 3, 192, 128, 64, True, BF16, {"rope_scaling": 2, "rope_factor": 32.0}),
    (33, 5, 136, 8, 128, True, F32, {"rope_scaling": 1, "rope_factor": 4.0}),
    (301, 2, 40, 0, 8, False, F32, {"rope_scaling": 2, "rope_factor": 40.0, "rope_base": 500000.0}),
    (130, 9, 72, 40, 32, True, BF16, {"rope_base": 1e6}),
    (5, 2, 24, 0, 24, True, BF16, {}),
    (1000, 17, 56, 16, 40, False, F32, {}),
]


def rope_want(x, pos, offset, d, half, over):
    freq, mul = ref.frequencies(d, over.get("rope_base", 10000.0),
                                {0: "plain", 1: "linear", 2: "yarn"}[over.get("rope_scaling", 0)],
                                over.get("rope_factor", 1.0))
    y = x.double()
    bound = torch.zeros_like(y)
    u = ref.half_step(x.dtype)
    for h in range(x.shape[1]):
        part = x[:, h, offset:offset + d]
        y[:, h, offset:offset + d] = ref.rotate(part, pos, half, freq, mul)
        # each of cos and sin: the angle to 2^-31 turns and half a step of its 24 bits (pi 2^-24), sincospi and the
        # factor a few steps, the products' and the sum's roundings: below 2^-20 of |a| + |b| together
        ab = part.double().abs()
        i = torch.arange(d // 2, device=x.device)
        e0, e1 = (i, i + d // 2) if half else (2 * i, 2 * i + 1)
        both = torch.empty_like(ab)
        both[:, e0] = both[:, e1] = ab[:, e0] + ab[:, e1]
        bound[:, h, offset:offset + d] = both * mul * 2.0 ** -20 + u * y[:, h, offset:offset + d].abs()
    return y, bound


@pytest.mark.parametrize("tokens,heads,head_dim,offset,d,half,dtype,over", ROPE)
def test_rope(tokens, heads, head_dim, offset, d, half, dtype, over):
    g = gen(tokens)
    lt = handle(1, 64, rope_dim=d, bf16=dtype == BF16, rope_layout=int(half), **over)
    x = randn(g, tokens, heads, head_dim, dtype=dtype)
    pos = torch.randint(-2**31, 2**31 - 1, (tokens,), generator=g, device="cuda").to(torch.int32)
    pos[0] = 0
    want, bound = rope_want(x, pos.double().cpu().cuda(), offset, d, half, over)
    # the reference's own angle (64-bit product, below 2^31): its fraction is good to 2^31 * 2^-53
    bound += 2.0 ** -18 * x.double().abs().amax()
    if tokens < 100:  # moderate positions: the derived bound alone
        pos = pos % 1000000
        want, bound = rope_want(x, pos, offset, d, half, over)
    out = torch.full_like(x, math.nan)
    assert isa.spin_rope(lt, x, pos, offset=offset, out=out) is out
    ref.check(out, want, bound, what="out of place")
    same = x.clone()
    isa.spin_rope(lt, same, pos, offset=offset)
    assert torch.equal(same, out)
    # token and head strides, heads outermost, at an odd element offset
    room = torch.full((heads * (tokens + 1) * (head_dim + 3) + 1,), math.nan, dtype=dtype, device="cuda")
    view = room[1:].view(heads, tokens + 1, head_dim + 3)[:, :tokens, :head_dim].transpose(0, 1)
    view.copy_(x)
    kept = torch.isnan(room)
    isa.spin_rope(lt, view, pos, offset=offset)
    assert torch.equal(view, out) and torch.equal(torch.isnan(room), kept)
    # the negative position undoes the rotation up to its roundings
    if not over.get("rope_scaling") == 2:
        back = isa.spin_rope(lt, out.clone(), -pos.clamp(min=-2**31 + 1), offset=offset)
        assert (back.double() - x.double()).abs().max() <= (4 * ref.half_step(dtype) + 2.0 ** -18) * x.abs().max()
    assert isa.spin_latent_error(lt) == (0, 0)


@pytest.mark.parametrize("base,scaling,factor", [(10000.0, 0, 1.0), (500000.0, 0, 1.0), (10000.0, 1, 40.0)])
def test_rope_angles_at_any_position(base, scaling, factor):
    """fp32 at positions over the whole range of int32, against angles from 60
    decimal digits, to the bound that the header states."""
    d, tokens = 64, 130
    g = gen(5)
    lt = handle(1, 64, rope_dim=d, bf16=False, rope_base=base, rope_scaling=scaling, rope_factor=factor)
    x = randn(g, tokens, 2, d, dtype=F32)
    pos = torch.randint(-2**31, 2**31 - 1, (tokens,), generator=g, device="cuda").to(torch.int32)
    pos[:8] = ints([0, 1, -1, 2**20, 2**24 + 1, 2**30, 2**31 - 1, -2**31])
    out = isa.spin_rope(lt, x, pos, out=torch.full_like(x, math.nan))
    with decimal.localcontext(prec=60):
        two_pi = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494")
        f = [decimal.Decimal(base) ** (decimal.Decimal(-2 * i) / d) / decimal.Decimal(factor) for i in range(d // 2)]
        angle = torch.tensor([[float(p * fi % two_pi) for fi in f] for p in pos.tolist()], dtype=torch.float64,
                             device="cuda")[:, None]
    a, b = x[..., 0::2].double(), x[..., 1::2].double()
    want = torch.stack([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], dim=-1).flatten(-2)
    # radians: the fraction's cut (2^-32 of a turn) and float, f's rounding (a double's half step from each of pow and
    # the division); of cos and sin: sincospif's step, 2^-24; each product and the sum half a step of |a| + |b|
    err = 2 * math.pi * (2.0 ** -26 + 2.0 ** -32) + pos.double().abs()[:, None, None] * torch.tensor(
        [float(fi) for fi in f], dtype=torch.float64, device="cuda") * 2.0 ** -52 + 3 * 2.0 ** -24
    bound = ((a.abs() + b.abs()) * err).repeat_interleave(2, dim=-1)
    ref.check(out, want, bound)


@pytest.mark.parametrize("dtype,half", [(BF16, False), (F32, True)])
def test_rope_into_the_other_part_of_a_packed_tensor(dtype, half):
    lt = handle(1, 64, bf16=dtype == BF16, rope_layout=int(half))
    g = gen(8)
    x = randn(g, 70, 3, 192, dtype=dtype)
    pos = torch.randint(0, 100000, (70,), generator=g, device="cuda").to(torch.int32)
    want = isa.spin_rope(lt, x, pos, offset=128, out=torch.empty_like(x))
    for pad in (0, 1):  # in 16-byte pieces, and not
        room = torch.full((70, 3, 384 + pad), math.nan, dtype=dtype, device="cuda")
        for a, b in ((0, 192), (192 + pad, 0)):
            room[..., a:a + 192] = x
            isa.spin_rope(lt, room[..., a:a + 192], pos, offset=128, out=room[..., b:b + 192])
            assert torch.equal(room[..., b:b + 192], want) and torch.equal(room[..., a:a + 192], x)


def test_rope_of_no_tokens():
    lt = handle(1, 64)
    x = torch.empty((0, 4, 64), dtype=BF16, device="cuda")
    assert isa.spin_rope(lt, x, ints([])).shape == (0, 4, 64)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("Q,rows,b,dc,d,half,dtype,ragged", [
    (1, 1, 16, 512, 64, False, BF16, False), (96, 1, 64, 512, 64, False, BF16, False),
    (5, 37, 32, 512, 64, True, BF16, True), (3, 130, 64, 64, 8, False, F32, True),
    (2, 300, 256, 256, 128, True, F32, True), (4, 3, 128, 72, 40, True, BF16, False)])
def test_append(Q, rows, b, dc, d, half, dtype, ragged):
    g = gen(Q * rows)
    max_slots = rows + 200
    lt = handle(Q, max_slots, block_size=b, latent_dim=dc, rope_dim=d, bf16=dtype == BF16, rope_layout=int(half))
    bt = pages(g, Q, max_slots, b)
    cache = randn(g, bt.numel() + 3, b, dc + d, dtype=dtype)
    before = cache.clone()
    both = randn(g, Q, rows, dc + d, dtype=dtype)
    ctx = torch.randint(1, max_slots - rows + 2, (Q,), generator=g, device="cuda").to(torch.int32)
    ctx[0] = max_slots - rows + 1
    count = torch.randint(0, rows + 1, (Q,), generator=g, device="cuda").to(torch.int32) if ragged else None
    isa.spin_latent_append(lt, rows, both[..., :dc], both[..., dc:], cache, bt, ctx, count)
    freq, _ = ref.frequencies(d)
    want, bound = before.double(), torch.zeros(before.shape, dtype=torch.float64, device="cuda")
    for q in range(Q):
        n = rows if count is None else int(count[q])
        slot = torch.arange(int(ctx[q]) - 1, int(ctx[q]) - 1 + n, device="cuda")
        at = bt[q].long()[slot // b], slot % b
        kr = ref.rotate(both[q, :n, dc:], slot, half, freq)
        want[at] = torch.cat([both[q, :n, :dc].double(), kr], dim=-1)
        big = both[q, :n, dc:].double().abs().amax(-1, keepdim=True) if n else kr
        bound[at] = torch.cat([torch.zeros_like(both[q, :n, :dc]).double(),
                               kr.abs() * ref.half_step(dtype) + 2.0 ** -19 * big], dim=-1)
    ref.check(cache, want, bound)
    # unaligned, separate parts: the same bits
    again = before.clone()
    odd = [torch.full((Q * rows * (w + 3) + 1,), math.nan, dtype=dtype, device="cuda")[1:].view(Q, rows, w + 3)[..., :w]
           for w in (dc, d)]
    odd[0].copy_(both[..., :dc])
    odd[1].copy_(both[..., dc:])
    isa.spin_latent_append(lt, rows, odd[0], odd[1], again, bt, ctx, count)
    assert torch.equal(again, cache)
    assert isa.spin_latent_error(lt) == (0, 0)


def test_append_refuses_bad_lengths_and_pages_on_the_device():
    Q, rows, b = 6, 4, 16
    lt = handle(Q, 64, block_size=b)
    g = gen(0)
    bt = pages(g, Q, 64, b)
    cache = randn(g, bt.numel() + 3, b, 576)
    before = cache.clone()
    c, kr = randn(g, Q, rows, 512), randn(g, Q, rows, 64)
    ctx, count = ints([0, 62, 1, 1, -7, 61]), ints([4, 4, 5, -1, 0, 4])
    isa.spin_latent_append(lt, rows, c, kr, cache, bt, ctx, count)
    changed = (cache != before).any(-1).nonzero()
    assert sorted(map(tuple, changed.tolist())) == sorted((int(bt[5, 3]), i) for i in range(12, 16))
    status, word = isa.spin_latent_error(lt)
    assert status == 6 and word == 1 | 4
    cache.copy_(before)
    bt[0, 0], bt[1, 0] = -1, bt.numel() + 3
    isa.spin_latent_append(lt, rows, c, kr, cache, bt, ints([1, 1, 1, 1, 1, 15]), None)
    assert (cache != before).any(-1).sum() == 4 * rows
    assert isa.spin_latent_error(lt) == (6, 2)
    assert isa.spin_latent_error(lt) == (0, 0)


# ---------------------------------------------------------------------------
# absorbed attention
# ---------------------------------------------------------------------------
def lists_for(g, ctx, rows, k, mess=False):
    """Ascending lists padded with -1; `mess`: shuffled, with repeats, entries that are not visible and gaps."""
    out = torch.full((len(ctx), rows, k), -1, dtype=torch.int32)
    cg = torch.Generator().manual_seed(int(torch.randint(1 << 30, (1,), generator=g, device="cuda")))
    for q, c in enumerate(ctx):
        for r in range(rows):
            n = min(k, c + r)
            s = torch.randperm(c + r, generator=cg)[:n].sort().values.to(torch.int32)
            out[q, r, :n] = s
            if mess and k > 4:
                row = out[q, r]
                row[::5] = -1
                row[1::7] = c + r + torch.arange(row[1::7].numel(), dtype=torch.int32)  # past the row's slots
                row[2::9] = int(s[0])
                row[3] = -2**31
                out[q, r] = row[torch.randperm(k, generator=cg)]
    return out.cuda()


def run_attention(lt, rows, cache, bt, ql, qr, ctx, topk, stream=None):
    Q, H, dc = lt.cfg.num_requests, lt.cfg.num_heads, lt.cfg.latent_dim
    out = torch.full((Q, rows, H, dc), math.nan, dtype=lt.dtype, device="cuda")
    lse = torch.full((Q, rows, H), math.nan, device="cuda")
    isa.spin_latent_attention(lt, rows, cache, bt, ql, qr, ctx, topk, out, lse, stream=stream)
    return out, lse


def attended(topk, q, r, end):
    if topk is None:
        return torch.arange(end, device="cuda")
    s = topk[q, r].long()
    return s[(s >= 0) & (s < end)]


def check_attention(lt, rows, cache, bt, ql, qr, ctx, topk, out, lse, skip=()):
    """Every (request, row) against 64 bits."""
    cfg = lt.cfg
    scale = cfg.softmax_scale
    for q in range(cfg.num_requests):
        for r in range(rows):
            end = int(ctx[q]) + r
            slots = attended(topk, q, r, end)
            slots = slots[[int(s) // cfg.block_size not in skip for s in slots]] if skip else slots
            kv = ref.slots_of(cache, bt, q, slots)
            qv = torch.cat([ql[q, r], qr[q, r]], dim=-1).double()
            o, z, a, rr, zz = ref.attend(qv, kv, kv[:, :cfg.latent_dim], scale)
            elem, lse_tol, norm = ref.attention_bounds(o, z, a, rr, zz, lt.dtype, cfg.latent_dim + cfg.rope_dim)
            ref.check(out[q, r], o, elem, norm, (q, r))
            if slots.numel() == 0:
                assert (out[q, r] == 0).all() and (lse[q, r] == -math.inf).all()
            else:
                ref.check(lse[q, r], z, lse_tol, what=("lse", q, r))


ATTN = [
    # Q, rows, H, topk (0: all), contexts, block, dtype, dc, dr
    (1, 1, 1, 0, [1], 64, BF16, 512, 64),
    (1, 1, 16, 256, [300], 64, BF16, 512, 64),
    (1, 1, 128, 2048, [5000], 64, BF16, 512, 64),
    (2, 1, 64, 64, [64, 65], 16, BF16, 512, 64),
    (3, 4, 20, 1000, [1, 999, 2500], 32, BF16, 512, 64),
    (5, 2, 40, 100, [63, 64, 65, 127, 129], 128, BF16, 512, 64),
    (2, 3, 100, 300, [700, 40], 256, BF16, 512, 64),
    (7, 1, 32, 0, [1, 63, 64, 65, 1000, 4097, 2], 64, BF16, 512, 64),
    (3, 4, 16, 0, [61, 62, 3000], 16, BF16, 512, 64),
    (1, 1, 13, 0, [20001], 64, BF16, 512, 64),
    (40, 1, 128, 512, None, 64, BF16, 512, 64),
    (150, 1, 8, 64, None, 64, BF16, 512, 64),
    (1, 2, 256, 128, [400], 64, BF16, 512, 64),
    (2, 1, 16, 128, [400, 10], 64, BF16, 256, 64),
    (2, 1, 16, 0, [400, 10], 64, BF16, 512, 32),
    (1, 1, 8, 256, [4096], 64, F32, 256, 64),
    (3, 2, 13, 100, [50, 333, 1], 16, F32, 512, 64),
    (4, 4, 3, 0, [1, 31, 33, 500], 32, F32, 64, 8),
    (2, 1, 9, 0, [100, 7], 64, BF16, 8, 128),
    (140, 2, 16, 0, None, 64, BF16, 512, 64),
    (300, 1, 3, 0, None, 16, F32, 64, 32),
    (155, 1, 40, 700, None, 64, BF16, 512, 64),
    (120, 1, 16, 2048, None, 64, BF16, 512, 64),
    (60, 1, 16, 1500, None, 64, BF16, 512, 64),
]


def attention_case(Q, rows, H, topk, ctxs, b, dtype, dc, dr, mess=False, **over):
    g = gen(Q * 1000 + H)
    if ctxs is None:
        ctxs = torch.randint(1, 3000, (Q,), generator=torch.Generator().manual_seed(Q)).tolist()
    max_slots = max(ctxs) + rows - 1
    lt = handle(Q, max_slots, block_size=b, num_heads=H, latent_dim=dc, rope_dim=dr, topk=max(topk, 1), max_rows=rows,
                bf16=dtype == BF16, **over)
    bt = pages(g, Q, max_slots, b)
    topk = lists_for(g, ctxs, rows, topk, mess) if topk else None
    # only what some row attends to holds numbers: everything else is NaN
    cache = nan_cache(bt, b, dc + dr, dtype)
    for q in range(Q):
        s = torch.unique(torch.cat([attended(topk, q, r, ctxs[q] + r) for r in range(rows)]))
        put(cache, bt, q, s, randn(g, s.numel(), dc + dr, dtype=dtype))
    ql, qr = randn(g, Q, rows, H, dc, dtype=dtype), randn(g, Q, rows, H, dr, dtype=dtype)
    return lt, cache, bt, ql, qr, ints(ctxs), topk


@pytest.mark.parametrize("Q,rows,H,topk,ctxs,b,dtype,dc,dr", ATTN)
def test_attention(Q, rows, H, topk, ctxs, b, dtype, dc, dr):
    lt, *a = attention_case(Q, rows, H, topk, ctxs, b, dtype, dc, dr)
    out, lse = run_attention(lt, rows, *a)
    check_attention(lt, rows, *a, out, lse)
    again, lse2 = run_attention(lt, rows, *a)  # the scratch now holds the first call's shares
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    assert isa.spin_latent_error(lt) == (0, 0)


@pytest.mark.parametrize("Q,rows,H,topk,ctxs,dtype", [(3, 2, 16, 300, [1, 200, 900], BF16),
                                                     (2, 1, 128, 700, [800, 5], BF16),
                                                     (2, 2, 5, 77, [90, 20], F32)])
def test_attention_lists_in_any_order_with_gaps_and_repeats(Q, rows, H, topk, ctxs, dtype):
    lt, *a = attention_case(Q, rows, H, topk, ctxs, 64, dtype, 512, 64, mess=True)
    out, lse = run_attention(lt, rows, *a)
    check_attention(lt, rows, *a, out, lse)
    assert isa.spin_latent_error(lt) == (0, 0)


@pytest.mark.parametrize("dtype,H", [(BF16, 16), (BF16, 128), (F32, 8)])
def test_attention_rows_that_see_nothing_and_bad_lengths(dtype, H):
    lt, cache, bt, ql, qr, ctx, topk = attention_case(4, 2, H, 200, [500, 300, 200, 100], 64, dtype, 512, 64)
    topk[0] = -1              # both rows empty
    topk[1, 0] = -1           # one row empty
    topk[2, 1, 64:] = -1      # a list that ends with its first tile
    out, lse = run_attention(lt, 2, cache, bt, ql, qr, ctx, topk)
    check_attention(lt, 2, cache, bt, ql, qr, ctx, topk, out, lse)
    assert isa.spin_latent_error(lt) == (0, 0)
    for bad in (0, -5, lt.cfg.max_slots, 2**31 - 1):
        c = ctx.clone()
        c[3] = bad
        for t in (topk, None):
            cache2 = cache if t is not None else cache.nan_to_num(nan=0.5)
            out2, lse2 = run_attention(lt, 2, cache2, bt, ql, qr, c, t)
            assert (out2[3] == 0).all() and (lse2[3] == -math.inf).all()
            if t is not None:
                assert torch.equal(out2[:3], out[:3])
            assert isa.spin_latent_error(lt) == (6, 1)


@pytest.mark.parametrize("dtype,H", [(BF16, 32), (F32, 4)])
def test_attention_skips_pages_outside_the_cache(dtype, H):
    lt, cache, bt, ql, qr, ctx, topk = attention_case(2, 1, H, 0, [300, 200], 32, dtype, 512, 64)
    bt[:, 2], bt[:, 5] = -1, cache.shape[0]
    out, lse = run_attention(lt, 1, cache, bt, ql, qr, ctx, None)
    check_attention(lt, 1, cache, bt.clamp(0, cache.shape[0] - 1), ql, qr, ctx, None, out, lse, skip=(2, 5))
    assert isa.spin_latent_error(lt) == (6, 2)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_takes_strided_and_unaligned_queries(dtype):
    Q, rows, H = 3, 2, 20
    lt, cache, bt, ql, qr, ctx, topk = attention_case(Q, rows, H, 100, [150, 90, 400], 64, dtype, 512, 64)
    out, lse = run_attention(lt, rows, cache, bt, ql, qr, ctx, topk)
    for lead, pad in ((0, 0), (8, 8), (1, 3)):  # a row of [q_latent | q_rope], aligned and not
        w = 576 + pad
        room = torch.full((Q * rows * H * w + lead,), math.nan, dtype=dtype, device="cuda")[lead:].view(Q, rows, H, w)
        room[..., :512], room[..., 512:576] = ql, qr
        got = run_attention(lt, rows, cache, bt, room[..., :512], room[..., 512:576], ctx, topk)
        assert torch.equal(got[0], out) and torch.equal(got[1], lse), (lead, pad)
    # heads outermost, and one query for all tokens and heads
    got = run_attention(lt, rows, cache, bt, ql.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3),
                        qr.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3), ctx, topk)
    assert torch.equal(got[0], out)
    one = ql[:1, :1, :1].expand(Q, rows, H, 512), qr[:1, :1, :1].expand(Q, rows, H, 64)
    got = run_attention(lt, rows, cache, bt, *one, ctx, topk)
    full = run_attention(lt, rows, cache, bt, one[0].contiguous(), one[1].contiguous(), ctx, topk)
    assert torch.equal(got[0], full[0])


@pytest.mark.parametrize("Q,rows,H,topk", [(1, 1, 16, 64), (200, 2, 16, 130), (160, 1, 128, 64), (9, 4, 40, 0)])
def test_attention_unaligned_queries_of_many_items_a_block(Q, rows, H, topk):
    """The first item of a block and those behind it, over and over."""
    lt, cache, bt, ql, qr, ctx, topk = attention_case(Q, rows, H, topk, [150 + 7 * q % 400 for q in range(Q)], 64, BF16,
                                                      512, 64)
    out, lse = run_attention(lt, rows, cache, bt, ql, qr, ctx, topk)
    room = torch.full((Q * rows * H * 579 + 1,), math.nan, dtype=BF16, device="cuda")[1:].view(Q, rows, H, 579)
    room[..., :512], room[..., 512:576] = ql, qr
    for _ in range(20):
        got = run_attention(lt, rows, cache, bt, room[..., :512], room[..., 512:576], ctx, topk)
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)
    assert isa.spin_latent_error(lt) == (0, 0)


def test_attention_large_logits_and_one_sided_weights():
    """Weights that all sit on one token, and maxima that rise tile by tile."""
    lt, cache, bt, ql, qr, ctx, _ = attention_case(1, 1, 16, 0, [500], 64, BF16, 512, 64)
    ql *= 40  # logits of some hundreds
    out, lse = run_attention(lt, 1, cache, bt, ql, qr, ctx, None)
    check_attention(lt, 1, cache, bt, ql, qr, ctx, None, out, lse)
    rise = torch.linspace(0.01, 8, 500, device="cuda").to(BF16)[:, None] * ql[0, 0, 0, :].sign() * 0.05
    s = torch.arange(500, device="cuda")
    kv = ref.slots_of(cache, bt, 0, s).to(BF16)
    kv[:, :512] = kv[:, :512] * 0.05 + rise
    put(cache, bt, 0, s, kv)
    ql = ql / 40
    out, lse = run_attention(lt, 1, cache, bt, ql, qr, ctx, None)
    check_attention(lt, 1, cache, bt, ql, qr, ctx, None, out, lse)


def ranked_keys(kr, order, power, sign):
    """Rotary parts of tokens whose logits are (rank - 0 or n) 2^power (exact in fp32): the query's first two elements
    are 2^(power + 4) and 2^power."""
    rank = order - (order.numel() if sign < 0 else 0)
    kr.zero_()
    kr[:, 0], kr[:, 1] = torch.div(rank, 16, rounding_mode="floor"), rank % 16


@pytest.mark.parametrize("dtype,H", [(BF16, 16), (BF16, 128), (F32, 8)])
@pytest.mark.parametrize("power", [20, 24, 31, 40, 60, 110])
@pytest.mark.parametrize("sign", [1, -1])
def test_attention_logits_of_any_size(power, sign, dtype, H):
    """All weight on the token of the largest logit, wherever it lies: the output is its latent up to roundings."""
    lt, cache, bt, ql, qr, ctx, topk = attention_case(3, 2, H, 300, [900, 65, 400], 64, dtype, 512, 64)
    ql.zero_()
    qr.zero_()
    qr[..., 0], qr[..., 1] = 2.0 ** (power + 4), 2.0 ** power
    g = gen(power)
    for t in (topk, None):
        for _ in range(4):
            want, want_lse = torch.empty((3, 2, H, 512), dtype=dtype, device="cuda"), torch.empty((3, 2, H), device="cuda")
            for q, c in enumerate(ctx.tolist()):
                order = torch.randperm(c + 1, generator=g, device="cuda")
                kv = randn(g, c + 1, 576, dtype=dtype)
                ranked_keys(kv[:, 512:], order, power, sign)
                put(cache, bt, q, torch.arange(c + 1, device="cuda"), kv)
                for r in range(2):
                    s = attended(t, q, r, c + r)
                    best = s[order[s].argmax()]
                    want[q, r] = kv[best, :512]
                    want_lse[q, r] = float(order[best] - (c + 1 if sign < 0 else 0)) * 2.0 ** power * lt.cfg.softmax_scale
            out, lse = run_attention(lt, 2, cache, bt, ql, qr, ctx, t)
            # the weight, near 1, in bf16 and the output: half a step each
            ref.check(out, want.double(), 2.1 * ref.half_step(dtype) * want.double().abs())
            # the scale by log2 e and back: three roundings of 2^-24
            assert ((lse.double() - want_lse.double()).abs() <= 4 * 2.0 ** -24 * want_lse.double().abs()).all()


def test_attention_passes_nan_of_an_attended_token_to_its_row_alone():
    lt, cache, bt, ql, qr, ctx, topk = attention_case(2, 2, 16, 64, [300, 300], 64, BF16, 512, 64)
    out, lse = run_attention(lt, 2, cache, bt, ql, qr, ctx, topk)
    mine = [s for s in topk[0, 1].tolist() if s >= 0 and s not in topk[0, 0].tolist()]
    put(cache, bt, 0, ints(mine[:1]).long(), math.nan)
    out2, lse2 = run_attention(lt, 2, cache, bt, ql, qr, ctx, topk)
    assert torch.isnan(out2[0, 1]).all() and torch.isnan(lse2[0, 1]).all()
    out2[0, 1], lse2[0, 1] = out[0, 1], lse[0, 1]
    assert torch.equal(out2, out) and torch.equal(lse2, lse)


def test_attention_cache_beyond_31_bits():
    """Elements past 2^31 and bytes past 2^32."""
    b, n = 64, 60000
    lt = handle(1, 1000, num_heads=16, topk=100)
    cache = torch.empty((n, b, 576), dtype=BF16, device="cuda")
    g = gen(3)
    bt = (n - 1 - torch.arange(16, device="cuda") * 3).to(torch.int32)[None]
    bt[0, 3] = 1
    for p in bt[0].tolist():
        cache[p] = randn(g, b, 576)
    ctx, topk = ints([1000]), lists_for(g, [1000], 1, 100)
    ql, qr = randn(g, 1, 1, 16, 512), randn(g, 1, 1, 16, 64)
    for t in (topk, None):
        out, lse = run_attention(lt, 1, cache, bt, ql, qr, ctx, t)
        check_attention(lt, 1, cache, bt, ql, qr, ctx, t, out, lse)
    c, kr = randn(g, 1, 1, 512), randn(g, 1, 1, 64)
    isa.spin_latent_append(lt, 1, c, kr, cache, bt, ints([1000]))
    assert torch.equal(cache[int(bt[0, 15]), 999 % 64, :512], c[0, 0])
    assert isa.spin_latent_error(lt) == (0, 0)


@pytest.mark.parametrize("dtype,H", [(BF16, 128), (F32, 8)])
def test_attention_without_lse_on_another_stream_and_in_a_graph(dtype, H):
    lt, cache, bt, ql, qr, ctx, topk = attention_case(3, 1, H, 300, [900, 100, 400], 64, dtype, 512, 64)
    out, lse = run_attention(lt, 1, cache, bt, ql, qr, ctx, topk)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run_attention(lt, 1, cache, bt, ql, qr, ctx, topk)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)
    only = torch.full_like(out, math.nan)
    isa.spin_latent_attention(lt, 1, cache, bt, ql, qr, ctx, topk, only)
    assert torch.equal(only, out)
    graph = torch.cuda.CUDAGraph()
    cap = torch.full_like(out, math.nan)
    with torch.cuda.graph(graph):
        isa.spin_latent_attention(lt, 1, cache, bt, ql, qr, ctx, topk, cap)
    graph.replay()
    assert torch.equal(cap, out)
    ql.mul_(0.5)
    ctx.copy_(ints([800, 101, 2]))
    topk.copy_(lists_for(gen(9), [800, 101, 2], 1, 300))
    cache.copy_(randn(gen(10), *cache.shape, dtype=dtype))
    lt.base[768:] = 255
    graph.replay()
    want, _ = run_attention(lt, 1, cache, bt, ql, qr, ctx, topk)
    assert torch.equal(cap, want)
    del graph


def test_two_handles_on_two_streams_at_once():
    cases = [attention_case(4, 1, 64, 0, [3000, 20, 900, 2000], 64, BF16, 512, 64) for _ in range(2)]
    cases[1][3].mul_(0.7)
    alone = [run_attention(c[0], 1, *c[1:]) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.full_like(a[0], math.nan) for _ in range(5)] for a in alone]
    torch.cuda.synchronize()
    for i in range(5):
        for c, s, o in zip(cases, streams, outs):
            isa.spin_latent_attention(c[0], 1, *c[1:], o[i], stream=s)
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert all(torch.equal(x, a[0]) for x in o)


# ---------------------------------------------------------------------------
# expanded attention
# ---------------------------------------------------------------------------
PREFILL = [
    # Q, rows, H, contexts, counts (None: all rows), block, dtype, dc, dr, dn, dv
    (1, 1, 1, [1], None, 64, BF16, 512, 64, 128, 128),
    (1, 101, 16, [1], None, 64, BF16, 512, 64, 128, 128),
    (1, 128, 2, [1], None, 64, BF16, 512, 64, 128, 128),
    (2, 129, 3, [128, 1], [129, 127], 16, BF16, 512, 64, 128, 128),
    (4, 300, 4, [1, 500, 77, 1000], [300, 1, 0, 257], 32, BF16, 512, 64, 128, 128),
    (3, 7, 5, [2000, 127, 129], [7, 3, 6], 128, BF16, 512, 64, 128, 128),
    (1, 1000, 8, [300], None, 256, BF16, 512, 64, 128, 128),
    (2, 260, 4, [200, 1], [260, 256], 64, BF16, 256, 64, 128, 128),
    (2, 40, 3, [30, 1], [40, 11], 16, BF16, 512, 32, 64, 128),
    (3, 50, 2, [1, 100, 33], [50, 0, 20], 16, F32, 128, 32, 64, 32),
    (1, 90, 3, [200], None, 64, F32, 512, 64, 128, 128),
    (2, 9, 2, [5, 60], [9, 8], 64, F32, 8, 8, 8, 256),
    (1, 700, 50, [900], None, 64, BF16, 512, 64, 128, 128),
    (2, 520, 60, [600, 1], [520, 300], 64, BF16, 512, 64, 128, 128),
    (300, 2, 1, None, None, 16, BF16, 512, 64, 128, 128),
    (2, 30, 3, [4000, 3000], [30, 29], 64, BF16, 512, 64, 128, 128),
    (1, 257, 2, [2500], None, 64, BF16, 512, 64, 128, 128),
    (1, 130, 1, [40000], None, 128, BF16, 512, 64, 128, 128),  # blocks that change slot tiles with every unit
]


def prefill_case(Q, rows, H, ctxs, counts, b, dtype, dc, dr, dn, dv, **over):
    g = gen(Q * 100 + rows)
    if ctxs is None:
        ctxs = torch.randint(1, 300, (Q,), generator=torch.Generator().manual_seed(Q)).tolist()
    max_slots = max(c - 1 + rows for c in ctxs)
    ends = [c - 1 + n if n else 0 for c, n in zip(ctxs, counts or [rows] * Q)]
    over.setdefault("prefill_slots", sum(-(-e // 128) * 128 for e in ends))
    lt = handle(Q, max_slots, block_size=b, num_heads=H, latent_dim=dc, rope_dim=dr, nope_dim=dn, v_dim=dv,
                bf16=dtype == BF16, **over)
    bt = pages(g, Q, max_slots, b)
    cache = nan_cache(bt, b, dc + dr, dtype)
    for q in range(Q):
        put(cache, bt, q, torch.arange(ends[q], device="cuda"), randn(g, ends[q], dc + dr, dtype=dtype))
    qv = randn(g, Q, rows, H, dn + dr, dtype=dtype)
    w = (torch.randn((H, dn + dv, dc), generator=g, device="cuda") * dc ** -0.5).to(dtype)
    return lt, cache, bt, qv, w, ints(ctxs), ints(counts) if counts else None


def run_prefill(lt, rows, cache, bt, qv, w, ctx, count, stream=None):
    out = torch.full((lt.cfg.num_requests, rows, lt.cfg.num_heads, lt.cfg.v_dim), 7.0, dtype=lt.dtype, device="cuda")
    isa.spin_latent_prefill(lt, rows, cache, bt, qv, w, ctx, count, out, stream=stream)
    return out


def check_prefill(lt, rows, cache, bt, qv, w, ctx, count, out):
    """Against 64 bits.  Keys and values are rounded to dtype once expanded:
    the reference rounds them too.  Where the kernel's fp32 sum of an expanded
    element lands on the other side of a rounding border, the element differs
    by one step; that happens to a share of about dc 2^-24 / u of them, and
    the weights' bound below leaves room for it (2-norm: sqrt of that share).
    Values and weights that a kernel keeps finer than dtype differ by the
    reference's own rounding of the values, within the same bounds."""
    cfg = lt.cfg
    dn, dc = cfg.nope_dim, cfg.latent_dim
    for q in range(cfg.num_requests):
        n = rows if count is None else int(count[q])
        assert (out[q, n:] == 7).all()
        if not n:
            continue
        end = int(ctx[q]) - 1 + n
        token = ref.slots_of(cache, bt, q, torch.arange(end, device="cuda"))
        hidden = torch.arange(end, device="cuda")[None, :] > (torch.arange(n, device="cuda") + int(ctx[q]) - 1)[:, None]
        for h in range(cfg.num_heads):
            kv = (token[:, :dc] @ w[h].double().T).to(lt.dtype).double()
            k, v = torch.cat([kv[:, :dn], token[:, dc:]], dim=1), kv[:, dn:]
            qh = qv[q, :n, h].double()
            s = (qh @ k.T * cfg.softmax_scale).masked_fill(hidden, -math.inf)
            p = torch.softmax(s, dim=-1)
            o, a, r = p @ v, p @ v.abs(), (p.square() @ v.square()).sqrt()
            z = (qh.abs() @ k.abs().T * cfg.softmax_scale).amax(-1)
            elem, _, norm = ref.attention_bounds(o, z * 0, a, r, z, lt.dtype, dn + cfg.rope_dim)
            if lt.dtype == BF16:
                # flipped expanded elements: a step of the largest value each
                elem = elem + 2 * ref.half_step(lt.dtype) * a
            else:
                # fp32: the expanded elements' sums over dc, a logit's and a value's
                e = dc * 2.0 ** -24
                elem = elem + 2.1 * e * z[:, None] * a + e * a * math.sqrt(dc)
                norm = norm + (2.1 * e * z[:, None] * a + e * a * math.sqrt(dc)).norm()
            ref.check(out[q, :n, h], o, elem, norm, (q, h))


@pytest.mark.parametrize("Q,rows,H,ctxs,counts,b,dtype,dc,dr,dn,dv", PREFILL)
def test_prefill(Q, rows, H, ctxs, counts, b, dtype, dc, dr, dn, dv):
    lt, *a = prefill_case(Q, rows, H, ctxs, counts, b, dtype, dc, dr, dn, dv)
    out = run_prefill(lt, rows, *a)
    check_prefill(lt, rows, *a, out)
    assert torch.equal(run_prefill(lt, rows, *a), out)
    assert isa.spin_latent_error(lt) == (0, 0)


def test_prefill_takes_strided_and_unaligned_queries_and_graphs():
    lt, cache, bt, qv, w, ctx, count = prefill_case(2, 140, 4, [50, 1], [140, 60], 64, BF16, 512, 64, 128, 128)
    out = run_prefill(lt, 140, cache, bt, qv, w, ctx, count)
    for lead, pad in ((8, 8), (1, 3)):
        room = torch.full((qv.numel() // 192 * (192 + pad) + lead,), math.nan, dtype=BF16, device="cuda")
        view = room[lead:].view(2, 140, 4, 192 + pad)[..., :192]
        view.copy_(qv)
        assert torch.equal(run_prefill(lt, 140, cache, bt, view, w, ctx, count), out), (lead, pad)
    heads_first = qv.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    assert torch.equal(run_prefill(lt, 140, cache, bt, heads_first, w, ctx, count), out)
    graph, cap = torch.cuda.CUDAGraph(), torch.full_like(out, 7)
    with torch.cuda.graph(graph):
        isa.spin_latent_prefill(lt, 140, cache, bt, qv, w, ctx, count, cap)
    lt.base[768:] = 255
    graph.replay()
    assert torch.equal(cap, out)
    ctx.copy_(ints([30, 1]))
    count.copy_(ints([3, 140]))
    cache.copy_(randn(gen(5), *cache.shape))
    cap.fill_(7)
    graph.replay()
    check_prefill(lt, 140, cache, bt, qv, w, ctx, count, cap)
    del graph


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_rows_before_a_token_that_is_not_finite_stay_clean(dtype, value):
    """Slots 150 and 260 of the first request, of a chunk at slots 99..298:
    their rows and those behind are NaN, the rows before and the other request
    have the bits that they had.  All latents of a head's keys meet an
    infinity as inf or -inf, so a logit sums both signs."""
    lt, cache, bt, qv, w, ctx, count = prefill_case(2, 200, 2, [100, 40], [200, 130], 64, dtype, 512, 64, 128, 128)
    out = run_prefill(lt, 200, cache, bt, qv, w, ctx, count)
    for slot, where in ((150, slice(0, 512)), (260, slice(0, 512)), (150, slice(512, 576)), (198, slice(17, 18))):
        broken = cache.clone()
        kv = ref.slots_of(cache, bt, 0, ints([slot]).long()).to(dtype)
        kv[:, where] = value
        put(broken, bt, 0, ints([slot]).long(), kv)
        got = run_prefill(lt, 200, broken, bt, qv, w, ctx, count)
        row = slot - 99
        assert torch.equal(got[0, :row], out[0, :row]) and torch.equal(got[1], out[1])
        assert torch.isnan(got[0, row:]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_refuses_bad_lengths_pages_and_a_full_workspace(dtype):
    lt, cache, bt, qv, w, ctx, count = prefill_case(4, 20, 2, [200, 100, 50, 1], [20, 10, 20, 5], 32, dtype, 512, 64,
                                                    128, 128)
    out = run_prefill(lt, 20, cache, bt, qv, w, ctx, count)
    whole = lambda x, q: torch.equal(x[q], out[q])
    untouched = lambda x, q: bool((x[q] == 7).all())
    for c, n, word in ((ctx, ints([20, 21, 20, 5]), 4), (ctx, ints([20, -1, 20, 5]), 4),
                       (ints([200, 0, 50, 1]), count, 1), (ints([200, 211, 50, 1]), count, 1),
                       (ints([200, 0, 50, 1]), ints([20, 0, 20, 5]), 0)):
        got = run_prefill(lt, 20, cache, bt, qv, w, c, n)
        assert untouched(got, 1) and all(whole(got, q) for q in (0, 2, 3))
        assert isa.spin_latent_error(lt) == (6 if word else 0, word)
    bt2 = bt.clone()
    bt2[1, 2] = -1              # slots 64..95 of request 1
    bt2[2, 3] = cache.shape[0]  # past request 2's slots: not looked at
    got = run_prefill(lt, 20, cache, bt2, qv, w, ctx, count)
    assert untouched(got, 1) and all(whole(got, q) for q in (0, 2, 3))
    assert isa.spin_latent_error(lt) == (6, 2)
    small, *_ = prefill_case(4, 20, 2, [200, 100, 50, 1], [20, 10, 20, 5], 32, dtype, 512, 64, 128, 128,
                             prefill_slots=384)
    got = run_prefill(small, 20, cache, bt, qv, w, ctx, count)
    assert whole(got, 0) and whole(got, 1) and untouched(got, 2) and untouched(got, 3)
    assert isa.spin_latent_error(small) == (6, 16)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("steps", [[40, 40, 40, 40], [-60, -60, -60, -60], [0, 20, 0, -20], [-30, 0, 30, 10], [90, 90, 90, 90]])
def test_prefill_values_of_any_magnitude(steps, dtype):
    """Latents times a power of two for each 128 slots, keys' weights divided by
    the largest, so that logits stay moderate while values leave the range of
    16-bit formats of few exponent bits."""
    lt, cache, bt, qv, w, ctx, count = prefill_case(1, 200, 2, [300], None, 64, dtype, 512, 64, 128, 128)
    s = torch.arange(499, device="cuda")
    kv = ref.slots_of(cache, bt, 0, s)
    factor = torch.tensor([2.0 ** e for e in steps], device="cuda", dtype=torch.float64)[s // 128]
    kv[:, :512] *= factor[:, None]
    put(cache, bt, 0, s, kv.to(dtype))
    w[:, :128] *= 2.0 ** -max(steps)
    out = run_prefill(lt, 200, cache, bt, qv, w, ctx, count)
    check_prefill(lt, 200, cache, bt, qv, w, ctx, count, out)


def check_first_rows(lt, cache, bt, qv, w, ctx, out, n):
    """The first n[q] rows of each request against 64 bits."""
    head = out.clone()
    for q, k in enumerate(n):
        head[q, k:] = 7
    check_prefill(lt, qv.shape[1], cache, bt, qv, w, ctx, ints(n), head)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("ctx0", [100, 3000])
@pytest.mark.parametrize("power", [8, 14, 18, 24, 30, 40, 60, 100])
def test_prefill_rows_before_a_large_token(power, ctx0, dtype):
    """One token of the chunk 2^power times as large as the others: the rows
    before it, those of its own 128 slots too, are as near to 64 bits as
    without it."""
    lt, cache, bt, qv, w, ctx, count = prefill_case(2, 200, 2, [ctx0, 40], [200, 130], 64, dtype, 512, 64, 128, 128)
    for row in (60, 199):
        slot = ints([ctx0 - 1 + row]).long()
        kept = ref.slots_of(cache, bt, 0, slot)
        large = kept.clone()
        large[:, :512] *= 2.0 ** power
        put(cache, bt, 0, slot, large.to(dtype))
        out = run_prefill(lt, 200, cache, bt, qv, w, ctx, count)
        check_first_rows(lt, cache, bt, qv, w, ctx, out, [row, 130])
        put(cache, bt, 0, slot, kept.to(dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("ctx0", [300, 3000])
@pytest.mark.parametrize("power", [12, 16, 20, 24, 28, 40])
def test_prefill_a_large_value_of_hardly_any_weight(power, ctx0, dtype):
    """A token of the context whose values are 2^power times the others' and
    whose weight is e^-46 of theirs (2^-66): at most 2^-26 of an output comes
    from it, and the other tokens keep their precision.  Keys are the rotary
    parts alone: q . k is 64 of the first token's -10 and about 0 of the others."""
    lt, cache, bt, qv, w, ctx, count = prefill_case(1, 150, 2, [ctx0], None, 64, dtype, 512, 64, 128, 128)
    w[:, :128] = 0
    qv[..., 128:] = 1
    slot = ints([17]).long()
    kv = ref.slots_of(cache, bt, 0, slot)
    kv[:, :512] *= 2.0 ** power
    kv[:, 512:] = -10
    put(cache, bt, 0, slot, kv.to(dtype))
    out = run_prefill(lt, 150, cache, bt, qv, w, ctx, count)
    check_prefill(lt, 150, cache, bt, qv, w, ctx, count, out)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,ctx0", [(2, 100), (1, 3000), (60, 300)])
def test_prefill_rows_before_finite_latents_whose_values_are_not(H, ctx0, dtype):
    """Latents of 2^127 (finite), value weights that sum them past the dtype's
    range in one element of every head (all 512 of one sign) and on the way, by
    signs in turn, in another, and keys of 0: the rows before have the bits that
    they had, those that see the slot are not finite in the first element."""
    lt, cache, bt, qv, w, ctx, count = prefill_case(2, 200, H, [ctx0, 40], [200, 130], 64, dtype, 512, 64, 128, 128)
    w[:, :128] = 0
    out = run_prefill(lt, 200, cache, bt, qv, w, ctx, count)
    check_prefill(lt, 200, cache, bt, qv, w, ctx, count, out)
    slots = [ctx0 - 1 + row for row in (70, 131, 199)]
    for column in (128, 200, 255):
        w2 = w.clone()
        w2[:, column] = 1
        w2[:, column ^ 1, ::2], w2[:, column ^ 1, 1::2] = 1, -1
        base = run_prefill(lt, 200, cache, bt, qv, w2, ctx, count)
        for slot in slots:
            broken = cache.clone()
            kv = ref.slots_of(cache, bt, 0, ints([slot]).long())
            kv[:, :512] = 2.0 ** 127
            put(broken, bt, 0, ints([slot]).long(), kv.to(dtype))
            got = run_prefill(lt, 200, broken, bt, qv, w2, ctx, count)
            row = slot - (ctx0 - 1)
            assert torch.equal(got[0, :row], base[0, :row]) and torch.equal(got[1], base[1])
            assert not torch.isfinite(got[0, row:, :, column - 128]).any()
    assert isa.spin_latent_error(lt) == (0, 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("ctx0", [100, 3000])
@pytest.mark.parametrize("power", [3, 8, 20, 100])
def test_prefill_rows_have_the_same_bits_whatever_comes_behind_them(power, ctx0, dtype):
    """A token of other latents, 2^power times as large, and another query of a
    later row: logits of the rows behind rise, those before keep their bits."""
    lt, cache, bt, qv, w, ctx, count = prefill_case(2, 200, 2, [ctx0, 40], [200, 130], 64, dtype, 512, 64, 128, 128)
    out = run_prefill(lt, 200, cache, bt, qv, w, ctx, count)
    for row in (5, 50, 113, 199):
        slot, broken, q2 = ints([ctx0 - 1 + row]).long(), cache.clone(), qv.clone()
        put(broken, bt, 0, slot, (randn(gen(row), 1, 576, dtype=F32) * 2.0 ** power).to(dtype))
        got = run_prefill(lt, 200, broken, bt, qv, w, ctx, count)
        assert torch.equal(got[0, :row], out[0, :row]) and torch.equal(got[1], out[1]), row
        q2[0, row] *= 2.0 ** power
        got = run_prefill(lt, 200, cache, bt, q2, w, ctx, count)
        assert torch.equal(got[0, :row], out[0, :row]) and torch.equal(got[0, row + 1:], out[0, row + 1:]), row


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("power", [20, 24, 31, 40, 60, 110])
@pytest.mark.parametrize("sign", [1, -1])
def test_prefill_logits_of_any_size(power, sign, dtype):
    """All weight on the visible slot of the largest logit, which changes from row to row (every slot of the chunk is a
    new largest with a chance that falls with its position): the output is its value."""
    lt, cache, bt, qv, w, ctx, count = prefill_case(2, 200, 3, [2200, 40], [200, 130], 64, dtype, 512, 64, 128, 128)
    w[:, :128] = 0
    qv.zero_()
    qv[..., 128], qv[..., 129] = 2.0 ** (power + 4), 2.0 ** power
    g = gen(power)
    for rising in (False, True):  # (the last rows' slots the largest, in order: the reference moves all the way)
        want = torch.full((2, 200, 3, 128), 7.0, dtype=torch.float64, device="cuda")
        for q, (c, n) in enumerate(zip(ctx.tolist(), count.tolist())):
            end = c - 1 + n
            slots = torch.arange(end, device="cuda")
            order = slots if rising else torch.randperm(end, generator=g, device="cuda")
            kv = randn(g, end, 576, dtype=dtype)
            ranked_keys(kv[:, 512:], order, power, sign)
            put(cache, bt, q, slots, kv)
            best = order.cummax(0).indices[c - 1:]
            want[q, :n] = torch.einsum("rc,hvc->rhv", kv[best, :512].double(), w[:, 128:].double())
        out = run_prefill(lt, 200, cache, bt, qv, w, ctx, count)
        # half a step each of the value, the weight (near 1) and the output, and the value's sum over 512 products, each
        # a step of 2^-24 of the sum of |c| |w|, below 40 (512 x 0.8 x 0.8 x 512^-1/2 = 14.5 on average)
        ref.check(out, want, 3.1 * ref.half_step(dtype) * want.abs() + 512 * 2.0 ** -24 * 40)


@pytest.mark.parametrize("Q,fit", [(30, 17), (40, 17), (400, 341)])
def test_prefill_of_many_requests_in_a_workspace_for_some(Q, fit):
    """Requests of two slot tiles each, in order: those behind the first that does not fit stay unwritten."""
    lt, cache, bt, qv, w, ctx, count = prefill_case(Q, 5, 2, [150] * Q, None, 16, BF16, 512, 64, 128, 128)
    out = run_prefill(lt, 5, cache, bt, qv, w, ctx, count)
    check_prefill(lt, 5, cache, bt, qv, w, ctx, count, out)
    assert isa.spin_latent_error(lt) == (0, 0)
    small, *_ = prefill_case(Q, 5, 2, [150] * Q, None, 16, BF16, 512, 64, 128, 128, prefill_slots=256 * fit + 128)
    got = run_prefill(small, 5, cache, bt, qv, w, ctx, count)
    assert torch.equal(got[:fit], out[:fit]) and bool((got[fit:] == 7).all())
    assert isa.spin_latent_error(small) == (6, 16)


def test_a_token_that_is_not_finite_in_a_context_of_many_slot_tiles():
    """One head, so that a block's units are slot tiles that follow one another, each with its own flags."""
    lt, cache, bt, qv, w, ctx, count = prefill_case(1, 300, 1, [40000], None, 128, BF16, 512, 64, 128, 128)
    out = run_prefill(lt, 300, cache, bt, qv, w, ctx, count)
    for slot, where in ((40100, slice(0, 1)), (40100, slice(511, 512)), (40298, slice(0, 512))):
        kv = ref.slots_of(cache, bt, 0, ints([slot]).long()).to(BF16)
        kept = kv.clone()
        kv[:, where] = math.nan
        put(cache, bt, 0, ints([slot]).long(), kv)
        got = run_prefill(lt, 300, cache, bt, qv, w, ctx, count)
        put(cache, bt, 0, ints([slot]).long(), kept)
        row = slot - 39999
        assert torch.equal(got[0, :row], out[0, :row]) and torch.isnan(got[0, row:]).all()


def test_sizes_beyond_the_counters_are_refused():
    lt, cache, bt, qv, w, ctx, count = prefill_case(1, 8, 2, [5], None, 64, BF16, 512, 64, 128, 128)
    lib, p, s = isa.load(), cache.data_ptr(), torch.cuda.current_stream().cuda_stream
    for rows in (2**30 + 1, 2**31 - 1):
        assert lib.spin_latent_prefill(lt.handle, rows, p, cache.shape[0], bt.data_ptr(), bt.shape[1], p, 0, 0, p,
                                       ctx.data_ptr(), None, p, s) == 7
    for heads, width in ((2**20 + 1, 1024), (1, 2**30 + 8), (2**31 - 1, 64)):
        assert lib.spin_rope(lt.handle, 1, heads, width, 0, p, 0, width, bt.data_ptr(), p, 0, width, s) == 1
    assert isa.spin_latent_error(lt) == (0, 0)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_a_layer_with_the_indexers_topk():
    """Prompt chunk (append, expanded attention), then a decode step: rotary
    positions, append, the indexer's top-k, absorbed attention over it.  The
    absorbed form of the whole context equals the expanded form of one row."""
    Q, P, H, dc, dr, dn, dv, k = 3, 700, 16, 512, 64, 128, 128, 256
    g = gen(11)
    lens = [700, 300, 513]
    lt = handle(Q, P + 8, num_heads=H, topk=k, prefill_slots=2560, softmax_scale=192 ** -0.5)
    bt = pages(g, Q, P + 8, 64)
    cache = nan_cache(bt, 64, dc + dr, BF16)
    count = ints(lens)
    one = ints([1] * Q)
    c, kr = randn(g, Q, P, dc), randn(g, Q, P, dr)
    w = (torch.randn((H, dn + dv, dc), generator=g, device="cuda") * dc ** -0.5).to(BF16)
    isa.spin_latent_append(lt, P, c, kr, cache, bt, one, count)
    pos = torch.arange(P, device="cuda", dtype=torch.int32).repeat(Q)
    q = randn(g, Q, P, H, dn + dr)
    isa.spin_rope(lt, q.view(Q * P, H, dn + dr), pos, offset=dn)
    out = run_prefill(lt, P, cache, bt, q, w, one, count)
    check_prefill(lt, P, cache, bt, q, w, one, count, out)

    # one decode step behind each prompt
    ctx = count + 1
    c1, kr1, q1 = randn(g, Q, 1, dc), randn(g, Q, 1, dr), randn(g, Q, 1, H, dn + dr)
    isa.spin_latent_append(lt, 1, c1, kr1, cache, bt, ctx)
    isa.spin_rope(lt, q1.view(Q, H, dn + dr), ctx - 1, offset=dn)
    st = isa.SpinState(isa.make_config(num_layers=1, num_requests=Q, max_slots=P + 8, topk=k, target_sparsity=0.0))
    keys = (torch.randn((bt.numel() + 3, 64, 128), generator=g, device="cuda")).to(torch.float8_e4m3fn)
    scale = torch.ones((bt.numel() + 3, 64), device="cuda")
    iq, iw = randn(g, Q, 1, 64, 128), torch.rand((Q, 1, 64), generator=g, device="cuda")
    mask, topk = st.new_mask(), torch.empty((Q, 1, k), dtype=torch.int32, device="cuda")
    isa.spin_decode_step(st, 0, 1, 0, keys.view(torch.uint8), scale, bt, iq, iw, ctx, False, mask, topk)
    assert (topk >= 0).all() and (topk[..., 1:] > topk[..., :-1]).all()
    ql = torch.einsum("qrhn,hnc->qrhc", q1[..., :dn].float(), w[:, :dn].float()).to(BF16)
    o, lse = run_attention(lt, 1, cache, bt, ql, q1[..., dn:], ctx, topk)
    check_attention(lt, 1, cache, bt, ql, q1[..., dn:], ctx, topk, o, lse)

    # absorbed over everything against expanded, both from the same cache
    o, lse = run_attention(lt, 1, cache, bt, ql, q1[..., dn:], ctx, None)
    absorbed = torch.einsum("qrhc,hvc->qrhv", o.double(), w[:, dn:].double())
    expanded = run_prefill(lt, 1, cache, bt, q1, w, ctx, None).double()
    # roundings to bf16 on the way: q_latent, o (absorbed), k, v, weights, out (expanded), half a step 2^-8 each,
    # independent; with logits of spread 1 each moves the result by at most 2^-8 of its 2-norm
    assert (absorbed - expanded).norm() <= 8 * 2.0 ** -8 * expanded.norm()
    assert isa.spin_latent_error(lt) == (0, 0) and isa.spin_get_error(st) == (0, 0)


def test_tensor_core_kernels_of_all_calls_one_behind_the_other():
    """The indexer's scores, the absorbed and the expanded attention back to
    back on one stream, each let in before the one before has ended."""
    Q, H, k = 8, 64, 512
    g = gen(21)
    lt, cache, bt, qv, w, ctx, count = prefill_case(Q, 40, H, [900 - 50 * q for q in range(Q)], None, 64, BF16, 512, 64,
                                                    128, 128, topk=k)
    st = isa.SpinState(isa.make_config(num_layers=1, num_requests=Q, max_slots=lt.cfg.max_slots, topk=k,
                                       target_sparsity=0.0))
    keys = torch.randn((cache.shape[0], 64, 128), generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    scale = torch.ones((cache.shape[0], 64), device="cuda")
    iq, iw = randn(g, Q, 1, 64, 128), torch.rand((Q, 1, 64), generator=g, device="cuda")
    mask, topk = st.new_mask(), torch.empty((Q, 1, k), dtype=torch.int32, device="cuda")
    ql, qr = randn(g, Q, 1, H, 512), randn(g, Q, 1, H, 64)
    out, pre = torch.empty_like(ql), torch.empty((Q, 40, H, 128), dtype=BF16, device="cuda")
    cache.nan_to_num_(nan=0.25)
    results = []
    for step in range(12):
        for x in (out, pre):
            x.fill_(math.nan)
        isa.spin_decode_step(st, 0, 1, step, keys, scale, bt, iq, iw, ctx, False, mask, topk)
        if step % 3 != 1:
            isa.spin_latent_attention(lt, 1, cache, bt, ql, qr, ctx, topk, out)
        isa.spin_latent_prefill(lt, 40, cache, bt, qv, w, ctx, count, pre)
        if step % 3 == 1:
            isa.spin_latent_attention(lt, 1, cache, bt, ql, qr, ctx, topk, out)
        results.append((topk.clone(), out.clone(), pre.clone()))
    assert all(torch.equal(a, b) for r in results[1:] for a, b in zip(r, results[0]))
    check_attention(lt, 1, cache, bt, ql, qr, ctx, topk, out, run_attention(lt, 1, cache, bt, ql, qr, ctx, topk)[1])
    assert isa.spin_latent_error(lt) == (0, 0) and isa.spin_get_error(st) == (0, 0)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second device")
def test_a_handle_of_another_device_than_the_current_one():
    lt = isa.SpinLatent(isa.make_latent_config(num_requests=1, max_slots=64), device="cuda:1")
    x = torch.randn((3, 2, 64), device="cuda:1").to(BF16)
    want = isa.spin_rope(isa.SpinLatent(lt.cfg, device="cuda:0"), x.to("cuda:0"), ints([1, 2, 3]))
    got = isa.spin_rope(lt, x, ints([1, 2, 3]).to("cuda:1"))
    assert torch.equal(got.cpu(), want.cpu()) and torch.cuda.current_device() == 0
