"""Measured cases of the operators around the latent cache: rotary positions, the cache's append, the absorbed
attention that decode steps run over a top-k list (or the whole context), and the expanded attention of a chunk of
new tokens.

Positions follow include/spin.h: row r of request q sits at p_r = ctx_len[q] - 1 + r and sees slots 0..p_r."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _rope(tokens, heads, head_dim, offset, rope_dim=64, layout="interleaved", scaling="plain", base=10000.0,
          factor=1.0, top=524288, dtype="bf16"):
    return {"op": "rope", "tokens": tokens, "heads": heads, "head_dim": head_dim, "offset": offset,
            "rope_dim": rope_dim, "layout": layout, "scaling": scaling, "base": base, "factor": factor, "top": top,
            "dtype": dtype}


def _append(requests, rows, ragged, max_slots, block, latent=512, rope_dim=64, layout="interleaved", dtype="bf16"):
    return {"op": "append", "requests": requests, "rows": rows, "ragged": ragged, "max_slots": max_slots,
            "block": block, "latent": latent, "rope_dim": rope_dim, "layout": layout, "dtype": dtype}


def _attention(requests, rows, heads, topk, ctx_lo, ctx_hi, block, latent=512, rope_dim=64, dtype="bf16"):
    """topk 0: every visible slot."""
    return {"op": "attention", "requests": requests, "rows": rows, "heads": heads, "topk": topk, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "block": block, "latent": latent, "rope_dim": rope_dim, "dtype": dtype}


def _prefill(requests, rows, ragged, ctx_lo, ctx_hi, heads, block, latent=512, rope_dim=64, nope=128, v=128,
             dtype="bf16"):
    return {"op": "prefill", "requests": requests, "rows": rows, "ragged": ragged, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "heads": heads, "block": block, "latent": latent, "rope_dim": rope_dim, "nope": nope,
            "v": v, "dtype": dtype}


def listed():
    return [
        # the indexer's queries of one decode step of the serving batch: 96 requests near 512K, half of each head
        {"name": "rope-decode-96", **_rope(96, 64, 128, 64)},
        # a long chunk's attention queries, half layout, positions scaled for a long context
        {"name": "rope-chunk-8192", **_rope(8192, 32, 192, 128, layout="half", scaling="yarn", factor=32.0,
                                            top=131072)},
        # the serving batch's step: one new token for each of 96 requests
        {"name": "append-decode-96", **_append(96, 1, False, 640, 64)},
        # prompts' chunks of different lengths, padded to the longest
        {"name": "append-chunk-8", **_append(8, 1024, True, 4096, 64)},
        # the smallest call: one request, one row, a short list (latency)
        {"name": "attention-one", **_attention(1, 1, 16, 256, 300, 300, 64)},
        # the serving batch: 96 requests, 128 heads, the indexer's 2048 slots
        {"name": "attention-serve-96", **_attention(96, 1, 128, 2048, 6000, 8192, 64)},
        # four speculative rows of 32 requests, an eighth of the heads, each row with its own list
        {"name": "attention-mtp-32", **_attention(32, 4, 16, 2048, 9000, 16384, 64)},
        # a layer without selection: ragged contexts, every visible slot
        {"name": "attention-dense-8", **_attention(8, 1, 32, 0, 1000, 32768, 64)},
        # the small fp32 workload: a 4K context, 256 of its slots
        {"name": "attention-f32", **_attention(1, 1, 8, 256, 4096, 4096, 64, latent=256, dtype="f32")},
        # a short prompt, odd length, from an empty cache
        {"name": "prefill-short", **_prefill(1, 101, False, 1, 1, 16, 64)},
        # four requests' chunks of different lengths on contexts of different lengths
        {"name": "prefill-chunk-4", **_prefill(4, 2048, True, 1, 6144, 16, 64)},
        # a long chunk at the end of a 16K context
        {"name": "prefill-long", **_prefill(1, 4096, False, 12289, 12289, 32, 64)},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention", "prefill"])
    block = rng.choice([16, 32, 64, 128])
    layout = rng.choice(["interleaved", "half"])
    if op == "rope":
        rope_dim = rng.choice([32, 64, 128])
        offset = rng.choice([0, 64, 128])
        scaling = rng.choice(["plain", "linear", "yarn"])
        return _rope(_log(rng, 1, 6000), rng.choice([1, 3, 8, 16, 32]), offset + rope_dim + rng.choice([0, 8, 64]),
                     offset, rope_dim, layout, scaling, rng.choice([10000.0, 500000.0]),
                     1.0 if scaling == "plain" else rng.choice([4.0, 40.0]), _log(rng, 2000, 1048576),
                     rng.choice(["bf16", "bf16", "f32"]))
    if op == "append":
        requests = _log(rng, 1, 128)
        rows = _log(rng, 1, max(1, 8192 // requests))
        return _append(requests, rows, rng.choice([True, False]), rows + _log(rng, 1, 400), block, layout=layout,
                       dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "attention":
        if rng.random() < 0.2:
            ctx = _log(rng, 1, 4096)
            return _attention(rng.randint(1, 4), rng.randint(1, 4), rng.choice([1, 8, 13]), rng.choice([0, 64, 300]),
                              max(1, ctx // 2), ctx, block, rng.choice([64, 128, 256]), rng.choice([32, 64]), "f32")
        rows = rng.choice([1, 1, 1, 2, 4])
        heads = rng.choice([8, 16, 20, 32, 64, 128])
        if rng.random() < 0.6:
            topk = rng.choice([256, 512, 1000, 2048])
            requests = _log(rng, 1, max(1, min(96, 96 * 128 // (rows * heads))))
            ctx = _log(rng, topk // 2, 12000)
            return _attention(requests, rows, heads, topk, max(1, ctx // 2), ctx, block)
        requests = _log(rng, 1, 24)
        ctx = _log(rng, 1, max(2, min(40000, 200000 * 128 // (requests * rows * heads))))
        return _attention(requests, rows, heads, 0, max(1, ctx // 3), ctx, block)
    if rng.random() < 0.2:
        return _prefill(rng.randint(1, 3), _log(rng, 1, 200), True, 1, _log(rng, 1, 500), rng.choice([2, 5]), block,
                        128, 32, rng.choice([32, 64]), rng.choice([32, 64]), "f32")
    requests = rng.choice([1, 2, 4])
    heads = rng.choice([4, 8, 16])
    return _prefill(requests, _log(rng, 2, 2048), rng.choice([True, False]), 1, _log(rng, 1, 6000), heads, block)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(gen, n, lo, hi):
    """n whole numbers in lo..hi, hi among them."""
    x = torch.randint(lo, hi + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
    x[0] = hi
    return x


def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(DTYPES[dtype])


def _paged(gen, requests, max_slots, block):
    """Every request's pages, in an order that is not theirs."""
    blocks = -(-max_slots // block)
    perm = torch.randperm(requests * blocks, generator=gen, device="cuda").to(torch.int32)
    return perm.view(requests, blocks).contiguous()


def _lists(gen, ctx_len, rows, topk):
    """A top-k list of each row as spin_topk writes it: ascending slots among the visible ones, padded with -1."""
    top = int(ctx_len.max()) + rows - 1
    pos = ctx_len[:, None].long() - 1 + torch.arange(rows, device="cuda")
    key = torch.rand((ctx_len.numel(), rows, top), generator=gen, device="cuda")
    key.masked_fill_(torch.arange(top, device="cuda") > pos[..., None], -1.0)
    n = min(topk, top)
    val, slot = key.topk(n, dim=-1)
    slot = torch.where(val < 0, torch.full_like(slot, 1 << 40), slot).sort(dim=-1).values
    out = torch.full((ctx_len.numel(), rows, topk), -1, dtype=torch.int32, device="cuda")
    out[..., :n] = torch.where(slot == 1 << 40, -1, slot).to(torch.int32)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s, op, dt = {"case": case}, case["op"], case["dtype"]
    if op == "rope":
        s["x"] = _randn(gen, (case["tokens"], case["heads"], case["head_dim"]), dt)
        s["positions"] = torch.randint(0, case["top"], (case["tokens"],), generator=gen, device="cuda",
                                       dtype=torch.int32)
        s["out"] = torch.zeros_like(s["x"])
        conf = dict(num_requests=1, max_slots=64, rope_scaling=case["scaling"], rope_base=case["base"],
                    rope_factor=case["factor"], rope_original=4096)
    else:
        Q, rows, block = case["requests"], case["rows"], case["block"]
        width = case["latent"] + case["rope_dim"]
        if op == "append":
            max_slots = case["max_slots"]
            s["row_count"] = _lengths(gen, Q, 0, rows) if case["ragged"] else torch.full_like(
                _lengths(gen, Q, 1, 1), rows)
            s["ctx_len"] = _lengths(gen, Q, 1, max_slots - rows + 1)
            both = _randn(gen, (Q, rows, width), dt)  # one projection gives both parts of a token
            s["c"], s["k_rope"] = both[..., :case["latent"]], both[..., case["latent"]:]
        elif op == "attention":
            s["ctx_len"] = _lengths(gen, Q, case["ctx_lo"], case["ctx_hi"])
            max_slots = case["ctx_hi"] + rows - 1
            s["q_latent"] = _randn(gen, (Q, rows, case["heads"], case["latent"]), dt)
            s["q_rope"] = _randn(gen, (Q, rows, case["heads"], case["rope_dim"]), dt)
            s["topk"] = _lists(gen, s["ctx_len"], rows, case["topk"]) if case["topk"] else None
            s["out"] = torch.zeros((Q, rows, case["heads"], case["latent"]), dtype=DTYPES[dt], device="cuda")
            s["lse"] = torch.zeros((Q, rows, case["heads"]), dtype=torch.float32, device="cuda")
        else:
            s["row_count"] = _lengths(gen, Q, 1, rows) if case["ragged"] else torch.full_like(
                _lengths(gen, Q, 1, 1), rows)
            s["ctx_len"] = _lengths(gen, Q, case["ctx_lo"], case["ctx_hi"])
            max_slots = case["ctx_hi"] + rows - 1
            s["q"] = _randn(gen, (Q, rows, case["heads"], case["nope"] + case["rope_dim"]), dt)
            s["w_kv"] = _randn(gen, (case["heads"], case["nope"] + case["v"], case["latent"]), "f32")
            s["w_kv"] = s["w_kv"].mul_(case["latent"] ** -0.5).to(DTYPES[dt])
            s["out"] = torch.zeros((Q, rows, case["heads"], case["v"]), dtype=DTYPES[dt], device="cuda")
        s["block_table"] = _paged(gen, Q, max_slots, block)
        s["cache"] = _randn(gen, (s["block_table"].numel(), block, width), dt)
        conf = dict(num_requests=Q, max_slots=max_slots, block_size=block, num_heads=case.get("heads", 1),
                    latent_dim=case["latent"], topk=max(1, case.get("topk", 1)),
                    max_rows=rows if op == "attention" else 1)
        if op == "prefill":
            conf |= dict(nope_dim=case["nope"], v_dim=case["v"], prefill_slots=Q * (-(-max_slots // 128) * 128))
    s["scale"] = (case.get("nope", 128) + case["rope_dim"]) ** -0.5
    if own:
        import indexer_sparse_attention_b200 as isa
        conf["rope_layout"] = {"interleaved": isa.SPIN_ROPE_INTERLEAVED, "half": isa.SPIN_ROPE_HALF}[
            case.get("layout", "interleaved")]
        conf["rope_scaling"] = {"plain": isa.SPIN_ROPE_PLAIN, "linear": isa.SPIN_ROPE_LINEAR,
                                "yarn": isa.SPIN_ROPE_YARN}[conf.get("rope_scaling", "plain")]
        s["latent"] = isa.SpinLatent(isa.make_latent_config(rope_dim=case["rope_dim"], bf16=dt == "bf16",
                                                            softmax_scale=s["scale"], **conf))
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _frequencies(case):
    """Angle per position of each rotated pair, in 64 bits, and the factor on cos and sin."""
    d, base, factor = case["rope_dim"], case.get("base", 10000.0), case.get("factor", 1.0)
    i = torch.arange(d // 2, device="cuda", dtype=torch.float64)
    f = base ** (-2.0 * i / d)
    scaling = case.get("scaling", "plain")
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        at = [d * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _rotate(x, positions, case):
    """x [..., rope_dim] in 32 bits, positions [...]."""
    f, m = _frequencies(case)
    angle = positions.double()[..., None] * f
    cos, sin = (angle.cos() * m).float(), (angle.sin() * m).float()
    y = torch.empty_like(x)
    if case.get("layout", "interleaved") == "half":
        a, b = x.chunk(2, dim=-1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    a, b = x[..., 0::2], x[..., 1::2]
    y[..., 0::2] = a * cos - b * sin
    y[..., 1::2] = a * sin + b * cos
    return y


def _gather(cache, block_table, block, slots):
    """Cache rows of slots [Q, n] (in 32 bits); a negative slot gives a zero row."""
    at = slots.clamp(min=0)
    page = block_table.long().gather(1, at // block)
    return torch.where((slots >= 0)[..., None], cache.view(-1, cache.shape[-1])[page * block + at % block].float(), 0.0)


def _softmax(logits, seen):
    """Weights and log-sum-exp over the last dimension of what is seen; rows that see nothing get 0 and -inf."""
    logits = logits.masked_fill(~seen, -math.inf)
    top = logits.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = (logits - top).exp()
    total = e.sum(dim=-1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total), (total.log() + top).squeeze(-1)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "rope":
        lo, hi = case["offset"], case["offset"] + case["rope_dim"]
        y = s["x"].clone()
        y[..., lo:hi] = _rotate(s["x"][..., lo:hi].float(), s["positions"][:, None].expand(
            -1, case["heads"]), case).to(y.dtype)
        return {"out": y}
    rows, block, dc = case["rows"], case["block"], case["latent"]
    pos = s["ctx_len"][:, None].long() - 1 + torch.arange(rows, device="cuda")
    if op == "append":
        live = torch.arange(rows, device="cuda") < s["row_count"][:, None]
        token = torch.cat([s["c"], _rotate(s["k_rope"].float(), pos, case).to(s["c"].dtype)], dim=-1)
        page = s["block_table"].long().gather(1, pos // block)
        s["cache"].view(-1, token.shape[-1])[(page * block + pos % block)[live]] = token[live]
        return {"cache": s["cache"]}
    Q, H = case["requests"], case["heads"]
    if op == "attention":
        q = torch.cat([s["q_latent"], s["q_rope"]], dim=-1).float()
        if s["topk"] is not None:
            slots = s["topk"].long()
            kv = _gather(s["cache"], s["block_table"], block, slots.view(Q, -1)).view(Q, rows, -1, q.shape[-1])
            seen = (slots >= 0) & (slots <= pos[..., None])
        else:
            slots = torch.arange(int(case["ctx_hi"]) + rows - 1, device="cuda").expand(Q, -1)
            slots = torch.where(slots <= pos[:, -1:], slots, -1)
            kv = _gather(s["cache"], s["block_table"], block, slots)[:, None].expand(-1, rows, -1, -1)
            seen = (slots >= 0)[:, None] & (slots[:, None] <= pos[..., None])
        p, lse = _softmax(q @ kv.transpose(-1, -2) * s["scale"], seen[:, :, None])
        return {"out": (p @ kv[..., :dc]).to(s["out"].dtype), "lse": lse}
    dn, dr = case["nope"], case["rope_dim"]
    slots = torch.arange(int(case["ctx_hi"]) + rows - 1, device="cuda").expand(Q, -1)
    last = s["ctx_len"][:, None].long() - 2 + s["row_count"][:, None]
    token = _gather(s["cache"], s["block_table"], block, torch.where(slots <= last, slots, -1))
    kv = torch.einsum("qsc,hnc->qhsn", token[..., :dc], s["w_kv"].float())
    q = s["q"].float().transpose(1, 2)
    logits = q[..., :dn] @ kv[..., :dn].transpose(-1, -2) + q[..., dn:] @ token[:, None, :, dc:].transpose(-1, -2)
    p, _ = _softmax(logits.mul_(s["scale"]), (slots[:, None] <= pos[..., None])[:, None])
    out = (p @ kv[..., dn:]).transpose(1, 2).to(s["out"].dtype)
    live = torch.arange(rows, device="cuda") < s["row_count"][:, None]
    return {"out": out.masked_fill(~live[..., None, None], 0)}


def run(state):
    if not own:
        return _plain(state)
    import indexer_sparse_attention_b200 as isa
    case, lt = state["case"], state["latent"]
    if case["op"] == "rope":
        isa.spin_rope(lt, state["x"], state["positions"], offset=case["offset"], out=state["out"])
        return {"out": state["out"]}
    if case["op"] == "append":
        isa.spin_latent_append(lt, case["rows"], state["c"], state["k_rope"], state["cache"], state["block_table"],
                               state["ctx_len"], state["row_count"])
        return {"cache": state["cache"]}
    if case["op"] == "attention":
        isa.spin_latent_attention(lt, case["rows"], state["cache"], state["block_table"], state["q_latent"],
                                  state["q_rope"], state["ctx_len"], state["topk"], state["out"], state["lse"])
        return {"out": state["out"], "lse": state["lse"]}
    isa.spin_latent_prefill(lt, case["rows"], state["cache"], state["block_table"], state["q"], state["w_kv"],
                            state["ctx_len"], state["row_count"], state["out"])
    return {"out": state["out"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    """Each input read once and each output written once; ragged lengths at their mean."""
    size, op = SIZES[case["dtype"]], case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["head_dim"] * size + 4 * case["tokens"], "flops": 3 * n * case["rope_dim"]}
    Q, rows, width = case["requests"], case["rows"], case["latent"] + case["rope_dim"]
    mean_rows = (1 + rows) / 2 if case.get("ragged") else rows
    if op == "append":
        n = Q * mean_rows
        return {"bytes": 2 * n * width * size + 8 * n, "flops": 3 * n * case["rope_dim"]}
    H, mean_ctx = case["heads"], (case["ctx_lo"] + case["ctx_hi"]) / 2
    if op == "attention":
        seen = min(case["topk"], mean_ctx) if case["topk"] else mean_ctx + (rows - 1) / 2
        read = Q * rows * seen if case["topk"] else Q * (mean_ctx + rows - 1)
        if case["topk"]:  # rows of a request may share slots: no more than its context is read
            read = min(read, Q * (mean_ctx + rows - 1))
        return {"bytes": size * (read * width + Q * rows * H * (width + case["latent"])) + 4 * Q * rows * H,
                "flops": 2 * Q * rows * H * seen * (width + case["latent"])}
    dn, dv, dr = case["nope"], case["v"], case["rope_dim"]
    slots = Q * (mean_ctx - 1 + mean_rows)
    pairs = Q * mean_rows * (mean_ctx - 1 + (mean_rows + 1) / 2)
    return {"bytes": size * (slots * width + Q * mean_rows * H * (dn + dr + dv) + H * (dn + dv) * case["latent"]),
            "flops": 2 * H * slots * case["latent"] * (dn + dv) + 2 * H * pairs * (dn + dr + dv)}


# ---------------------------------------------------------------------------
# the definition in 64 bits, row by row
# ---------------------------------------------------------------------------
def _turn(x, position, case):
    """One token's rotated elements x [n, rope_dim] in 64 bits, as products of complex numbers."""
    d, base, factor, scaling = case["rope_dim"], case.get("base", 10000.0), case.get("factor", 1.0), case.get(
        "scaling", "plain")
    freq, size = [], 1.0
    if scaling == "yarn":
        size = 1.0 + math.log(factor) / 10.0
        edge = [d / 2 * math.log(4096 / (2 * math.pi * turns), base) for turns in (32, 1)]
        edge = max(0, math.floor(edge[0])), min(d - 1, math.ceil(edge[1]))
    for i in range(d // 2):
        f = math.pow(base, -2.0 * i / d)
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            share = min(1.0, max(0.0, (i - edge[0]) / max(edge[1] - edge[0], 0.001)))
            f = f * ((1.0 - share) + share / factor)
        freq.append(f)
    w = torch.polar(torch.full((d // 2,), size, dtype=torch.float64, device=x.device).expand(position.numel(), -1),
                    position.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device=x.device))
    half = case.get("layout", "interleaved") == "half"
    pair = x.double().unflatten(-1, (2, d // 2) if half else (d // 2, 2))
    z = torch.complex(pair.select(-2 if half else -1, 0), pair.select(-2 if half else -1, 1))
    z = torch.view_as_real(z * w)
    return (z.transpose(-1, -2) if half else z).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        y = s["x"].double()
        part = slice(case["offset"], case["offset"] + case["rope_dim"])
        for h in range(case["heads"]):
            y[:, h, part] = _turn(s["x"][:, h, part], s["positions"], case)
        return {"out": y}
    Q, rows, block, dc = case["requests"], case["rows"], case["block"], case["latent"]
    ctx = s["ctx_len"].tolist()
    if case["op"] == "append":
        y, count = s["cache"].double(), s["row_count"].tolist()
        for q in range(Q):
            slot = torch.arange(ctx[q] - 1, ctx[q] - 1 + count[q], device="cuda")
            page = s["block_table"][q][slot // block].long()
            y[page, slot % block, :dc] = s["c"][q, :count[q]].double()
            y[page, slot % block, dc:] = _turn(s["k_rope"][q, :count[q]], slot, case)
        return {"cache": y}
    y = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "attention":
        lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
        for q in range(Q):
            own_pages = s["block_table"][q].long()
            for r in range(rows):
                if s["topk"] is None:
                    slot = torch.arange(ctx[q] + r, device="cuda")
                else:
                    slot = s["topk"][q, r].long()
                    slot = slot[(slot >= 0) & (slot < ctx[q] + r)]
                token = s["cache"][own_pages[slot // block], slot % block].double()
                a = (s["q_latent"][q, r].double() @ token[:, :dc].T + s["q_rope"][q, r].double() @ token[:, dc:].T)
                a = a * s["scale"]
                lse[q, r] = torch.logsumexp(a, dim=-1)
                y[q, r] = torch.softmax(a, dim=-1) @ token[:, :dc]
        return {"out": y, "lse": lse}
    dn, count = case["nope"], s["row_count"].tolist()
    for q in range(Q):
        end = ctx[q] - 1 + count[q]
        slot = torch.arange(end, device="cuda")
        token = s["cache"][s["block_table"][q].long()[slot // block], slot % block].double()
        hidden = slot[None, :] > (torch.arange(count[q], device="cuda") + ctx[q] - 1)[:, None]
        for h in range(case["heads"]):
            k = torch.cat([token[:, :dc] @ s["w_kv"][h, :dn].double().T, token[:, dc:]], dim=1)
            a = s["q"][q, :count[q], h].double() @ k.T * s["scale"]
            a = torch.softmax(a.masked_fill_(hidden, -math.inf), dim=-1)
            y[q, :count[q], h] = a @ (token[:, :dc] @ s["w_kv"][h, dn:].double().T)
    return {"out": y}
