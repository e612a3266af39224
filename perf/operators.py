"""The serving operators of the INT4 KV cache: cases, inputs, plain forms and work.

Four operators, in the order a decoder layer uses them:

- slots: block tables, slot maps and positions from request lengths;
- norm_rope: RMS norms of queries and keys per head with the rotary positions;
- append: the same for new tokens, with the per-head Hadamard rotation, the
  INT4 quantization of keys and values and the store into the cache's pages;
- attention: attention over the pages of the INT4 cache.

The cache holds, for each page, KV head and slot, the D codes of a row in
the library's stored form (D / 2 bytes) and one fp32 scale.
"""
import math

import torch

own = False

DEV = "cuda"
F32, BF16 = "float32", "bfloat16"
MASK_A, MASK_C = 0xE79E79E7, 0x9E79E79E


def _i32(u):
    """The int32 with the bits of the 32-bit word u."""
    return u - (1 << 32) if u >= 1 << 31 else u


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _attention(name, **kw):
    case = {"name": name, "op": "attention", "batch": 1, "q_min": 1, "q_max": 1, "kv_min": 1, "kv_max": 4096,
            "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "dtype": BF16, "causal": True, "window": 0,
            "lse": False}
    case.update(kw)
    return case


def listed():
    return [
        # one decode step of a running batch: every request adds one token
        {"name": "slots_step", "op": "slots", "batch": 48, "new_max": 1, "ctx_max": 4000, "page": 16, "finished": 3,
         "tokens": 64},
        # prompts arriving while others finish, a padded token budget
        {"name": "slots_prompts", "op": "slots", "batch": 700, "new_max": 160, "ctx_max": 9000, "page": 32,
         "finished": 90, "tokens": 65536},
        # a decode step of a few requests, q and k as views of the qkv product
        {"name": "norm_rope_step", "op": "norm_rope", "tokens": 7, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "rotate": False, "dtype": BF16},
        # a packed batch of prompts
        {"name": "norm_rope_prompt", "op": "norm_rope", "tokens": 12001, "heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "rotate": False, "dtype": BF16},
        # one decode step of a running batch into the cache
        {"name": "append_step", "op": "append", "tokens": 96, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "page": 16, "dtype": BF16},
        # a packed batch of prompts into the cache
        {"name": "append_prompt", "op": "append", "tokens": 8191, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "page": 64, "dtype": BF16},
        # fp32 activations, small heads, a part of each head rotated, pairs side by side
        {"name": "append_f32", "op": "append", "tokens": 1333, "heads": 16, "kv_heads": 4, "dim": 64, "rot": 32,
         "interleaved": True, "page": 32, "dtype": F32},
        # one request's decode step: latency
        _attention("decode_one", kv_min=4321, kv_max=4321),
        # a running batch of ragged lengths: the cache's bytes
        _attention("decode_batch", batch=64, kv_min=1, kv_max=16384, page=64),
        # whole prompts over their own keys: matrix products
        _attention("prompt", batch=4, q_min=1500, q_max=2048, kv_min=0, kv_max=0, page=64),
        # prompt chunks over longer contexts, small heads
        _attention("chunk", batch=6, q_min=129, q_max=256, kv_min=1000, kv_max=12000, heads=16, kv_heads=4, dim=64,
                   page=32, lse=True),
        # a few draft tokens for each request, fp32, wide heads, a sliding window
        _attention("draft_f32", batch=12, q_min=1, q_max=3, kv_min=0, kv_max=3500, heads=16, kv_heads=4, dim=256,
                   page=16, dtype=F32, window=1024, lse=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["slots", "norm_rope", "append", "attention", "attention", "attention"])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice([BF16, BF16, F32])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8] if kv_heads < 8 else [1, 2, 4])
    if op == "slots":
        batch = _spread(rng, 1, 700)
        new_max = 1 if rng.random() < 0.4 else _spread(rng, 2, 160)
        return {"op": op, "batch": batch, "new_max": new_max, "ctx_max": _spread(rng, 1, 9000), "page": page,
                "finished": rng.randint(0, batch // 4), "tokens": min(65536, batch * new_max + rng.randint(0, 64))}
    if op in ("norm_rope", "append"):
        rows = 8191 * 48 * 128 if dtype == BF16 else 8191 * 24 * 128
        tokens = _spread(rng, 1, max(1, min(8191, rows // ((heads + 2 * kv_heads) * dim))))
        case = {"op": op, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rot": rng.choice([dim, dim, dim // 2]), "interleaved": rng.random() < 0.4, "dtype": dtype}
        case.update({"rotate": rng.random() < 0.5} if op == "norm_rope" else {"page": page})
        return case
    kind = rng.choice(["decode", "decode", "chunk", "prompt"])
    causal = rng.random() < 0.8
    window = _spread(rng, 16, 4096) if causal and rng.random() < 0.25 else 0
    lse = rng.random() < 0.4
    if kind == "decode":
        batch = _spread(rng, 1, 64)
        kv_max = _spread(rng, 1, min(65536, 4000000 // (batch * kv_heads)))
        q_max = rng.choice([1, 1, 1, 2, 4])
        kv_min = rng.choice([0, kv_max // 2, kv_max])
    elif kind == "chunk":
        batch, q_max = _spread(rng, 1, 6), _spread(rng, 16, 300)
        kv_max = _spread(rng, 64, max(64, min(12000, 40000 // batch)))
        kv_min = kv_max // 3
    else:
        batch, q_max, kv_min, kv_max = _spread(rng, 1, 4), _spread(rng, 100, 1000), 0, 0
    return {"op": "attention", "batch": batch, "q_min": max(1, (2 * q_max) // 3), "q_max": q_max, "kv_min": kv_min,
            "kv_max": kv_max, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype,
            "causal": causal, "window": window, "lse": lse}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _gen(seed, device=DEV):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) % (1 << 62))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _randint(g, lo, hi, n):
    """n whole numbers of [lo, hi]."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int64)


def _lengths(case, seed):
    """The (query, key) lengths of an attention case's requests, as lists; the sum of the first goes by the case."""
    g = _gen(seed, "cpu")
    n, most = case["batch"], case["q_max"]
    q = most - (torch.arange(n) * 7919) % (most - case["q_min"] + 1)
    q = q[torch.randperm(n, generator=g)]
    ctx = torch.randint(case["kv_min"], case["kv_max"] + 1, (n,), generator=g)
    return q.tolist(), (q + ctx).tolist()


def _stored(codes):
    """The stored form (uint8 [rows, D / 2]) of codes in [-7, 7] (int64 [rows, D])."""
    f = (codes.abs() | ((codes < 0).long() << 5)).reshape(codes.shape[0], -1, 4, 8)
    a = torch.stack([f[:, :, 0], f[:, :, 1]], 2)  # the first words of the two pairs of a chunk
    b = torch.stack([f[:, :, 3], f[:, :, 2]], 2)  # their partners
    k = torch.arange(8, device=codes.device) * 6
    lo, hi = (a << k).sum(-1), (b << k).sum(-1)  # 48 bits each: X = lo | hi << 48
    x0, x1, x2 = lo & 0xFFFFFFFF, (lo >> 32) | ((hi & 0xFFFF) << 16), hi >> 16
    not_a, not_c = 0xFFFFFFFF ^ MASK_A, 0xFFFFFFFF ^ MASK_C
    wa = (x0 & MASK_A) | (x1 & not_a)
    wb = (x2 & MASK_C) | (x1 & not_c)
    w = torch.stack([wa[:, :, 0], wa[:, :, 1], wb[:, :, 1], wb[:, :, 0]], -1)
    w = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
    return w.reshape(codes.shape[0], -1).view(torch.uint8)


def _pool(g, pages, heads, page, dim, spread):
    """A cache half with earlier tokens in it: stored rows and their scales, [pages, heads, page, ...]."""
    n = pages * heads * page
    bank = _randn(g, min(n, 16384), dim)
    top = bank.abs().amax(1, keepdim=True)
    codes = _stored(torch.round(bank * 7 / top).long())
    pick = torch.randint(0, bank.shape[0], (n,), generator=g, device=DEV)
    scale = (top[:, 0] / 7)[pick] * torch.exp(spread * _randn(g, n))
    return (codes[pick].reshape(pages, heads, page, dim // 2), scale.reshape(pages, heads, page))


def _hadamard(dim):
    i = torch.arange(dim, device=DEV)
    p = i[:, None] & i[None, :]
    p = p ^ (p >> 4)
    p = p ^ (p >> 2)
    p = p ^ (p >> 1)
    return (1 - 2 * (p & 1)).double()  # dim <= 256: the parity of 8 bits


def _rope(rows, rot):
    """cos then sin of the rotary angles, [rows, rot]."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    a = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _prepare_slots(case, g):
    n, page = case["batch"], case["page"]
    ctx = _randint(g, 0, case["ctx_max"], n)
    new = _randint(g, 1, case["new_max"], n)
    done = torch.randperm(n, generator=g, device=DEV)[: case["finished"]]
    new[done] = -1
    width = -(-(case["ctx_max"] + case["new_max"]) // page) + 1
    have = (ctx + page - 1) // page
    capacity = n * (-(-case["ctx_max"] // page) + case["new_max"] // page + 2)
    order = torch.randperm(capacity, generator=g, device=DEV)
    table = torch.full((n, width), -1, device=DEV, dtype=torch.int64)
    cell = torch.arange(width, device=DEV)[None, :] < have[:, None]
    table[cell] = order[: int(have.sum())]
    free = torch.full((capacity,), -1, device=DEV, dtype=torch.int64)
    spare = order[int(have.sum()):]
    head = int(_randint(g, 0, capacity - 1, 1))
    free[(head + torch.arange(spare.numel(), device=DEV)) % capacity] = spare
    # in every third batch the pool is short: the last request or two that need a page find none
    need = torch.where(new >= 0, (ctx + new + page - 1) // page - have, torch.zeros_like(have))
    count = max(0, int(need.sum()) - 2) if n % 3 == 0 else spare.numel()
    return {"ctx": ctx.int(), "new": new.int(), "table": table.int(), "free": free.int(),
            "free_state": torch.tensor([head, count], device=DEV, dtype=torch.int32), "page": page,
            "tokens": case["tokens"]}


def _prepare_rows(case, g):
    t, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    dt = getattr(torch, case["dtype"])
    x = _randn(g, t, hq + 2 * hk, d)
    x = x * torch.exp(0.3 * _randn(g, t, 1, 1)) * torch.exp(0.5 * _randn(g, 1, hq + 2 * hk, d))
    x = x.to(dt)
    reach = 32768 if t < 32768 else t
    state = {"q": x[:, :hq], "k": x[:, hq:hq + hk], "v": x[:, hq + hk:],
             "wq": (1 + 0.2 * _randn(g, d)), "wk": (1 + 0.2 * _randn(g, d)), "eps": 1e-6,
             "rope": _rope(reach, case["rot"]), "pos": _randint(g, 0, reach - 1, t).int(),
             "interleaved": case["interleaved"], "rot": case["rot"], "had": _hadamard(d)}
    if case["op"] == "norm_rope":
        state["rotate"] = case["rotate"]
        return state
    page = case["page"]
    pages = -(-t // page) + 2
    state["kc"], state["ks"] = _pool(g, pages, hk, page, d, 0.2)
    state["vc"], state["vs"] = _pool(g, pages, hk, page, d, 0.2)
    state["slots"] = torch.randperm(pages * page, generator=g, device=DEV)[:t]
    return state


def _prepare_attention(case, g, seed):
    q_len, kv_len = _lengths(case, seed)
    page, n, d = case["page"], case["batch"], case["dim"]
    width = -(-max(kv_len) // page) + 1
    kv = torch.tensor(kv_len, device=DEV)
    have = (kv + page - 1) // page
    pages = int(have.sum()) + 3
    table = torch.zeros(n, width, device=DEV, dtype=torch.int64)
    table[torch.arange(width, device=DEV)[None, :] < have[:, None]] = torch.randperm(pages, generator=g, device=DEV)[
        : pages - 3]
    cu = torch.tensor([0] + q_len, device=DEV).cumsum(0)
    state = {"q": (1.8 * _randn(g, sum(q_len), case["heads"], d)).to(getattr(torch, case["dtype"])),
             "table": table.int(), "kv_len": kv.int(), "cu": cu.int(), "q_max": case["q_max"], "page": page,
             "kv_max": max(kv_len), "causal": case["causal"], "window": case["window"], "lse": case["lse"],
             "had": _hadamard(d)}
    state["kc"], state["ks"] = _pool(g, pages, case["kv_heads"], page, d, 0.1)
    state["vc"], state["vs"] = _pool(g, pages, case["kv_heads"], page, d, 0.3)
    return state


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "slots":
        state = _prepare_slots(case, g)
    elif case["op"] == "attention":
        state = _prepare_attention(case, g, seed)
    else:
        state = _prepare_rows(case, g)
    state["op"] = case["op"]
    return state


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------
def _opened(stored):
    """The codes, as float32, of stored rows [..., D / 2]."""
    w = stored.contiguous().view(torch.int32)
    w = w.reshape(*w.shape[:-1], -1, 4)
    a, b = w[..., 0:2], torch.stack([w[..., 3], w[..., 2]], -1)
    ma, mc = _i32(MASK_A), _i32(MASK_C)
    x0, x1, x2 = a & ma, (a & ~ma) | (b & ~mc), b & mc
    f = torch.stack([x0, x0 >> 6, x0 >> 12, x0 >> 18, x0 >> 24, ((x0 >> 30) & 3) | (x1 << 2), x1 >> 4, x1 >> 10,
                     x1 >> 16, x1 >> 22, ((x1 >> 28) & 15) | (x2 << 4), x2 >> 2, x2 >> 8, x2 >> 14, x2 >> 20,
                     x2 >> 26], -1)
    size = (f & 7).float()
    c = torch.where((f & 32) != 0, -size, size)  # [..., chunks, pair, 16]
    c = torch.cat([c[..., 0, 0:8], c[..., 1, :], c[..., 0, 8:16]], -1)
    return c.reshape(*stored.shape[:-1], -1)


def _plain_slots(s):
    page, tokens = s["page"], s["tokens"]
    ctx, new, table, free = s["ctx"].long(), s["new"].long(), s["table"], s["free"]
    n, width = table.shape
    size = free.numel()
    head, count = s["free_state"][0].long(), s["free_state"][1].long()
    have = (ctx + page - 1) // page
    grown = new >= 0
    want = (ctx + new + page - 1) // page
    fits = want <= width
    need = torch.where(grown & fits, want - have, torch.zeros_like(have))
    upto = need.cumsum(0)
    served = ~grown | (fits & ((need == 0) | (upto <= count)))
    taken = torch.where(upto <= count, upto, torch.zeros_like(upto)).max()
    col = torch.arange(width, device=DEV)
    nth = col[None, :] - have[:, None]  # which of the request's new pages
    fresh = (nth >= 0) & (nth < need[:, None]) & (served & grown)[:, None]
    at = (head + (upto - need)[:, None] + nth) % size
    table.copy_(torch.where(fresh, free[at.clamp(0, size - 1)], table))
    back = torch.where(grown, torch.zeros_like(have), have)
    before = back.cumsum(0) - back
    given = (col[None, :] < back[:, None])
    to = (head + count + before[:, None] + col[None, :]) % size
    ring = torch.cat([free, free[:1]])
    ring.scatter_(0, torch.where(given, to, torch.full_like(to, size)).reshape(-1), table.reshape(-1))
    free.copy_(ring[:size])
    kv_len = torch.where(grown, torch.where(served, ctx + new, ctx), torch.zeros_like(ctx))
    cu = torch.cat([torch.zeros_like(ctx[:1]), new.clamp(min=0).cumsum(0)])
    t = torch.arange(tokens, device=DEV)
    who = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    real = who < n
    who = who.clamp(max=n - 1)
    pos = ctx[who] + t - cu[who]
    ok = real & served[who]
    cell = table[who, (pos // page).clamp(0, width - 1)].long()
    none = torch.full_like(pos, -1)
    slot = torch.where(ok & (cell >= 0), cell * page + pos % page, none)
    state = torch.stack([(head + taken) % size, count - taken + back.sum()])
    return [kv_len.int(), cu.int(), served.int(), slot, torch.where(ok, pos, none).int(), table, free, state.int()]


def _normed(x, w, s, wide):
    """RMS norm and rotary positions of rows [T, heads, D], in 32 bits or (wide) 64."""
    t = torch.float64 if wide else torch.float32
    x = x.to(t)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.to(t)
    rot = s["rot"]
    cs = s["rope"][s["pos"].long()].to(t)[:, None, :]
    c, n = cs[..., : rot // 2], cs[..., rot // 2:]
    if s["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = y[..., : rot // 2], y[..., rot // 2: rot]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _plain_norm_rope(s):
    q, k = _normed(s["q"], s["wq"], s, False), _normed(s["k"], s["wk"], s, False)
    if s["rotate"]:
        h = s["had"].float()
        q, k = (q @ h) * h.shape[0] ** -0.5, (k @ h) * h.shape[0] ** -0.5
    return [q.to(s["q"].dtype), k.to(s["k"].dtype)]


def _quantized(u, dim):
    """Codes and scales of rotated rows, u the sums before the 1 / sqrt(D), in 64 bits: codes lie next to borders."""
    top = u.abs().amax(-1, keepdim=True)
    code = torch.where(top > 0, torch.round(7 * u / top), torch.zeros_like(u))
    return code, (top / (7 * math.sqrt(dim))).float()


def _plain_append(s):
    h = s["had"]
    d = h.shape[0]
    q = (_normed(s["q"], s["wq"], s, False) @ h.float()) * d ** -0.5
    k = _normed(s["k"], s["wk"], s, True) @ h
    v = s["v"].double() @ h
    pages, heads, page = s["ks"].shape
    dt = s["q"].dtype

    def stored(u, codes, scales):
        rows = (_opened(codes) * scales[..., None]).transpose(1, 2).reshape(pages * page, heads, d)
        code, scale = _quantized(u, d)
        rows[s["slots"]] = (code * scale).float()
        return rows.reshape(pages, page, heads, d).transpose(1, 2).to(dt)

    return [q.to(dt), stored(k, s["kc"], s["ks"]), stored(v, s["vc"], s["vs"])]


def _visible(s, rows, keys):
    """Which keys [batch, rows, keys] a row sees, and which rows exist."""
    cu, kv = s["cu"].long(), s["kv_len"].long()
    q_len = (cu[1:] - cu[:-1])[:, None]
    i, j = torch.arange(rows, device=DEV)[None, :], torch.arange(keys, device=DEV)
    real = i < q_len
    last = kv[:, None] - q_len + i
    end = last + 1 if s["causal"] else kv[:, None].expand(-1, rows)
    see = j < end[..., None]
    if s["window"]:
        see = see & (j > last[..., None] - s["window"])
    return see, real


def _plain_attention(s):
    n, rows, keys = s["kv_len"].numel(), s["q_max"], s["kv_max"]
    total, hq, d = s["q"].shape
    hk, page = s["ks"].shape[1:]
    group = hq // hk
    j = torch.arange(keys, device=DEV)
    cell = s["table"].long()[:, j // page]  # [n, keys]
    at = (cell[:, None, :] * hk + torch.arange(hk, device=DEV)[None, :, None]) * page + j % page
    kc = _opened(s["kc"].reshape(-1, d // 2)[at]) * s["ks"].reshape(-1)[at][..., None]
    see, real = _visible(s, rows, keys)
    cu = s["cu"].long()
    row = (cu[:-1, None] + torch.arange(rows, device=DEV)).clamp(max=total - 1)
    q = s["q"][row].float().reshape(n, rows, hk, group, d).permute(0, 2, 3, 1, 4).reshape(n, hk, group * rows, d)
    x = torch.matmul(q, kc.transpose(-1, -2)) * d ** -0.5
    del kc
    x = x.reshape(n, hk, group, rows, keys).masked_fill(~see[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - top)
    del x
    mass = p.sum(-1, keepdim=True)
    vc = _opened(s["vc"].reshape(-1, d // 2)[at]) * s["vs"].reshape(-1)[at][..., None]
    o = torch.matmul(p.reshape(n, hk, group * rows, keys), vc).reshape(n, hk, group, rows, d)
    o = (o / mass.clamp(min=1e-30)) @ s["had"].float() * d ** -0.5
    o = o.permute(0, 3, 1, 2, 4).reshape(n, rows, hq, d)[real].to(s["q"].dtype)
    if not s["lse"]:
        return [o]
    lse = (top + torch.log(mass)).permute(0, 3, 1, 2, 4).reshape(n, rows, hq)[real]
    return [o, lse]


# --------------------------------------------------------------------------
# The framework's operators
# --------------------------------------------------------------------------
def _own(s):
    import rotated_w4a4_amd as rw4
    if s["op"] == "slots":
        r = rw4.kv_slots(s["ctx"], s["new"], s["table"], s["free"], s["free_state"], s["page"], s["tokens"])
        return [r.kv_len, r.cu_new, r.served, r.slot_map, r.positions, s["table"], s["free"], r.free_state]
    if s["op"] == "norm_rope":
        return list(rw4.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["rope"], s["pos"], eps=s["eps"],
                                     interleaved=s["interleaved"], rotate=s["rotate"]))
    cache = rw4.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
    if s["op"] == "append":
        q = rw4.kv_append(cache, s["k"], s["v"], s["slots"], s["q"], s["wq"], s["wk"], s["rope"], s["pos"],
                          eps=s["eps"], interleaved=s["interleaved"])
        # the pages as the values they stand for, through the read-back call, a page a row
        pages, group = s["ks"].shape[0], s["q"].shape[-1]
        back = [rw4.dequantize(c.view(pages, -1), x.view(pages, -1), s["q"].dtype).view(*x.shape, group)
                for c, x in ((s["kc"], s["ks"]), (s["vc"], s["vs"]))]
        return [q, *back]
    r = rw4.kv_attention(s["q"], cache, s["table"], s["kv_len"], s["cu"], max_q_len=s["q_max"], causal=s["causal"],
                         window=s["window"], return_lse=s["lse"])
    return list(r) if s["lse"] else [r]


def run(state):
    if own:
        return _own(state)
    return {"slots": _plain_slots, "norm_rope": _plain_norm_rope, "append": _plain_append,
            "attention": _plain_attention}[state["op"]](state)


# --------------------------------------------------------------------------
# Work
# --------------------------------------------------------------------------
def work(case):
    if case["op"] == "slots":
        n, t = case["batch"], case["tokens"]
        pages = n * (1 + case["new_max"] // case["page"]) + case["finished"] * case["ctx_max"] // (2 * case["page"])
        # lengths in, length, start and served out; a slot (8 bytes) and a position (4) for each token;
        # a page id read and written for each new or returned page
        return {"bytes": 8 * n + 12 * n + 12 * t + 8 * pages, "flops": 10 * (n + t)}
    if case["op"] in ("norm_rope", "append"):
        t, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        size = 2 if case["dtype"] == BF16 else 4
        if case["op"] == "norm_rope":
            n = t * (hq + hk) * d
            return {"bytes": 2 * size * n + t * (4 + 4 * case["rot"]),
                    "flops": n * (10 + (math.log2(d) if case["rotate"] else 0))}
        n = t * (hq + 2 * hk) * d
        slots = (-(-t // case["page"]) + 2) * case["page"]
        row = d // 2 + 4
        # rows in, queries out, stored rows out; the cache read back as values
        return {"bytes": size * n + size * t * hq * d + 2 * t * hk * row + t * (12 + 4 * case["rot"])
                + 2 * slots * hk * (row + size * d), "flops": n * (10 + math.log2(d))}
    size = 2 if case["dtype"] == BF16 else 4
    d, hq, hk = case["dim"], case["heads"], case["kv_heads"]
    q = (case["q_min"] + case["q_max"]) / 2
    kv = q + (case["kv_min"] + case["kv_max"]) / 2
    if case["window"]:
        read = min(kv, case["window"] + q)
        seen = min(kv, case["window"])
    else:
        read = kv
        seen = kv - (q - 1) / 2 if case["causal"] else kv
    n = case["batch"]
    return {"bytes": n * (read * hk * (d + 8) + q * hq * (2 * size * d + (4 if case["lse"] else 0))),
            "flops": n * hq * q * seen * 4 * d}


# --------------------------------------------------------------------------
# The definitions in 64 bits, apart from the plain forms
# --------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "slots":
        return None  # whole numbers

    def _sylvester(dim):
        h = torch.ones(1, 1, dtype=torch.float64, device=DEV)
        two = torch.tensor([[1.0, 1.0], [1.0, -1.0]], dtype=torch.float64, device=DEV)
        while h.shape[0] < dim:
            h = torch.kron(two, h)
        return h

    def _exact_codes(stored):
        """Codes bit by bit from the table of the stored form: bit t (0-2 size, 3 sign) of code k of a pair."""
        d = 2 * stored.shape[-1]
        bits = (stored.reshape(-1, d // 32, 4, 4, 1) >> torch.arange(8, device=DEV, dtype=torch.uint8)) & 1
        bits = bits.reshape(-1, d // 32, 4, 32).bool()
        special = {5: "a30 a31 b0 a3", 6: "a4 b5 b6 a9", 7: "a10 b11 b12 a15", 8: "a16 b17 b18 a21",
                   9: "a22 b23 b24 a27", 10: "a28 b29 b30 b1"}
        out = torch.zeros(bits.shape[0], d // 32, 32, dtype=torch.float64, device=DEV)
        for first, partner in ((0, 3), (1, 2)):
            word = {"a": bits[:, :, first], "b": bits[:, :, partner]}
            for k in range(16):
                if k in special:
                    at = [(x[0], int(x[1:])) for x in special[k].split()]
                elif k < 5:
                    at = [("a", 6 * k + t) for t in (0, 1, 2, 5)]
                else:
                    at = [("b", 6 * k - 64 + t) for t in (0, 1, 2, 5)]
                v = [word[w][..., p].double() for w, p in at]
                channel = 8 * (first if k < 8 else partner) + k % 8
                out[:, :, channel] = (v[0] + 2 * v[1] + 4 * v[2]) * (1 - 2 * v[3])
        return out.reshape(*stored.shape[:-1], d)

    def _exact_normed(x, w, s):
        x = x.double()
        y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * w.double()
        rot = s["rot"]
        z = y.clone()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + rot // 2)
            c = s["rope"][s["pos"].long(), i].double()[:, None]
            n = s["rope"][s["pos"].long(), rot // 2 + i].double()[:, None]
            z[..., a] = y[..., a] * c - y[..., b] * n
            z[..., b] = y[..., b] * c + y[..., a] * n
        return z

    def _exact_attention(case, s):
        d = case["dim"]
        h = _sylvester(d)
        hk = case["kv_heads"]
        group = case["heads"] // hk
        page = case["page"]
        cu, kv_len = s["cu"].tolist(), s["kv_len"].tolist()
        outs, masses = [], []
        for b in range(case["batch"]):
            q_len, kv = cu[b + 1] - cu[b], kv_len[b]
            pages = s["table"][b, : -(-kv // page)].long()
            keys, values = [], []
            for c, x, to in ((s["kc"], s["ks"], keys), (s["vc"], s["vs"], values)):
                rows = c[pages].transpose(0, 1).reshape(hk, -1, d // 2)[:, :kv]
                scales = x[pages].transpose(0, 1).reshape(hk, -1)[:, :kv].double()
                to.append(_exact_codes(rows.contiguous()) * scales[..., None])
            k, v = keys[0], values[0]
            q = s["q"][cu[b]:cu[b + 1]].double()
            place = kv - q_len + torch.arange(q_len, device=DEV)[:, None]
            j = torch.arange(kv, device=DEV)[None, :]
            hidden = torch.zeros(q_len, kv, dtype=torch.bool, device=DEV)
            if case["causal"]:
                hidden |= j > place
            if case["window"]:
                hidden |= j <= place - case["window"]
            o = torch.zeros(q_len, case["heads"], d, dtype=torch.float64, device=DEV)
            m = torch.zeros(q_len, case["heads"], dtype=torch.float64, device=DEV)
            for head in range(case["heads"]):
                x = (q[:, head] @ k[head // group].t().contiguous()) / math.sqrt(d)
                x = x.masked_fill(hidden, -math.inf)
                m[:, head] = torch.logsumexp(x, -1)
                o[:, head] = torch.nan_to_num(torch.softmax(x, -1)) @ v[head // group]
            outs.append(o @ h / math.sqrt(d))
            masses.append(m)
        return [torch.cat(outs)] + ([torch.cat(masses)] if case["lse"] else [])

    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(case, s)
    h = _sylvester(case["dim"])
    root = math.sqrt(case["dim"])
    q = _exact_normed(s["q"], s["wq"], s)
    k = _exact_normed(s["k"], s["wk"], s)
    if case["op"] == "norm_rope":
        return [q @ h / root, k @ h / root] if case["rotate"] else [q, k]
    got = [q @ h / root]
    page = case["page"]
    for u, c, x in ((k @ h, s["kc"], s["ks"]), (s["v"].double() @ h, s["vc"], s["vs"])):
        values = _exact_codes(c) * x.double()[..., None]
        top = u.abs().max(-1, keepdim=True).values
        code = torch.round(u * 7 / top)
        values[s["slots"] // page, :, s["slots"] % page] = code * (top / 7 / root)
        got.append(values)
    return got
