"""Serving operators in the card's own 4-bit format, and windows with sinks: cases, inputs, plain forms and work.

Three operators of a long-running decode:

- quantize: activations or weights through the block Hadamard into MXFP4 (FP4 E2M1 codes, one power-of-two scale for
  32 channels), read back as the values they stand for;
- gemm: the product of two MXFP4 operands;
- sink_attention: attention over the INT4 KV cache with a sliding window, whose first tokens (sinks) stay visible.

Stored MXFP4: codes uint8 [rows, K / 2], the low four bits the even channel (sign, then the index into 0, 0.5, 1, 1.5,
2, 3, 4, 6); scales uint8 [K / 128, rows, 4], byte i of entry (g, r) the exponent plus 127 of channels 128 g + 32 i ..
of row r.  The INT4 cache is described in operators.py.
"""
import math

import torch

own = False

DEV = "cuda"
F32, BF16 = "float32", "bfloat16"
MASK_A, MASK_C = 0xE79E79E7, 0x9E79E79E
SIZES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _sinks(name, **kw):
    case = {"name": name, "op": "sink_attention", "batch": 1, "q_min": 1, "q_max": 1, "kv_min": 1, "kv_max": 4096,
            "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "dtype": BF16, "window": 1024, "sinks": 4, "lse": False}
    case.update(kw)
    return case


def listed():
    return [
        # activations of a few requests' decode step: latency
        {"name": "quantize_step", "op": "quantize", "rows": 7, "K": 4096, "block": 128, "signed": False, "dtype": BF16,
         "layout": "rows"},
        # a batch of prompts in front of the down projection
        {"name": "quantize_down", "op": "quantize", "rows": 4096, "K": 14336, "block": 128, "signed": False,
         "dtype": BF16, "layout": "rows"},
        # fp32 activations, an odd number of tokens, wider blocks with random signs
        {"name": "quantize_f32", "op": "quantize", "rows": 1333, "K": 8192, "block": 256, "signed": True, "dtype": F32,
         "layout": "rows"},
        # a layer's weights [K, N] packed
        {"name": "pack_weight", "op": "quantize", "rows": 4096, "K": 4096, "block": 128, "signed": False, "dtype": F32,
         "layout": "kn"},
        # one token through a projection: the weights' bytes
        {"name": "gemm_step", "op": "gemm", "M": 1, "N": 4096, "K": 4096, "dtype": BF16},
        # a running batch of odd size through the up projection
        {"name": "gemm_batch", "op": "gemm", "M": 61, "N": 11008, "K": 4096, "dtype": BF16},
        # a prompt through a projection
        {"name": "gemm_prompt", "op": "gemm", "M": 2048, "N": 4096, "K": 4096, "dtype": BF16},
        # a batch of prompts through the down projection
        {"name": "gemm_down", "op": "gemm", "M": 4096, "N": 4096, "K": 14336, "dtype": BF16},
        # one request's step far into a conversation: latency
        _sinks("sinks_one", kv_min=54321, kv_max=54321),
        # a running batch of ragged lengths, most beyond the window
        _sinks("sinks_batch", batch=64, kv_max=16384, window=2048),
        # whole prompts longer than the window
        _sinks("sinks_prompt", batch=4, q_min=1500, q_max=2048, kv_min=0, kv_max=0, window=512, sinks=16),
        # a few draft tokens for each request, fp32, wide heads, more sinks than a tile
        _sinks("sinks_draft_f32", batch=12, q_max=3, kv_min=0, kv_max=6000, heads=16, kv_heads=4, dim=256, page=16,
               dtype=F32, window=1000, sinks=100, lse=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "quantize", "gemm", "gemm", "gemm", "sink_attention", "sink_attention"])
    dtype = rng.choice([BF16, BF16, F32])
    if op == "quantize":
        block = rng.choice([1, 128, 128, 256, 512])
        K = rng.choice([512, 1024, 2048, 4096, 8192]) if block > 128 else 128 * _spread(rng, 1, 112)
        return {"op": op, "rows": _spread(rng, 1, max(1, min(16384, 4096 * 14336 // K))), "K": K, "block": block,
                "signed": block > 1 and rng.random() < 0.3, "dtype": dtype,
                "layout": rng.choice(["rows", "rows", "rows", "kn", "nk"])}
    if op == "gemm":
        M, K = _spread(rng, 1, 4096), 128 * _spread(rng, 1, 112)
        return {"op": op, "M": M, "N": _spread(rng, 1, min(14336, 4096 * 4096 * 14336 // (M * K))), "K": K,
                "dtype": dtype}
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8] if kv_heads < 8 else [1, 2, 4])
    kind = rng.choice(["decode", "decode", "chunk", "prompt"])
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
    return {"op": op, "batch": batch, "q_min": max(1, (2 * q_max) // 3), "q_max": q_max, "kv_min": kv_min,
            "kv_max": kv_max, "heads": heads, "kv_heads": kv_heads, "dim": rng.choice([64, 128, 128, 256]),
            "page": rng.choice([16, 32, 64, 128]), "dtype": dtype, "window": _spread(rng, 16, 4096),
            "sinks": _spread(rng, 1, 300), "lse": rng.random() < 0.4}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _gen(seed, device=DEV):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) % (1 << 62))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _hadamard(dim):
    i = torch.arange(dim, device=DEV)
    p = i[:, None] & i[None, :]
    p = p ^ (p >> 8)
    p = p ^ (p >> 4)
    p = p ^ (p >> 2)
    p = p ^ (p >> 1)
    return (1 - 2 * (p & 1)).double()  # dim <= 512: the parity of 9 bits


def _two(E):
    """2^E exactly, in 64 bits, from the number's own bits."""
    return ((E.long() + 1023) << 52).view(torch.float64)


def _index(y, E):
    """Indexes into SIZES of y 2^-E, ties to the even index (values: fp32 or fp64, E whole numbers of their blocks)."""
    a = y.abs() * _two(-E).to(y.dtype)
    i = (a > 0.25).to(torch.uint8)
    for tie, odd in ((0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False), (5.0, True)):
        i += (a > tie) if odd else (a >= tie)  # a tie between indexes i and i + 1 goes to the even one
    return i


def _exponent(y):
    """E of rows y [..., 32]; a block of zeros has -127."""
    top = y.abs().amax(-1, keepdim=True)
    e = torch.frexp(top).exponent - 3  # frexp's mantissa lies in [0.5, 1)
    return torch.where(top > 0, e.clamp(-127, 127), torch.full_like(e, -127))


def _encoded(g, rows, K, spread):
    """MXFP4 codes and scales of Gaussian rows: [rows, K / 2], [K / 128, rows, 4]."""
    y = _randn(g, rows, K // 32, 32)
    y *= torch.exp(spread * _randn(g, rows, 1, 1)) * torch.exp(spread * _randn(g, 1, K // 32, 1))
    E = _exponent(y)
    n = _index(y, E) | ((y < 0).to(torch.uint8) << 3)
    n = n.reshape(rows, K)
    q = n[:, 0::2] | (n[:, 1::2] << 4)
    s = (E[..., 0] + 127).to(torch.uint8).reshape(rows, K // 128, 4).transpose(0, 1).contiguous()
    return q.contiguous(), s


def _prepare_quantize(case, g):
    rows, K = case["rows"], case["K"]
    dt = getattr(torch, case["dtype"])
    signs = None
    if case["layout"] == "rows":
        # activations: a few channels far above the rest, single values far above those
        x = _randn(g, rows, K) * torch.exp(0.3 * _randn(g, rows, 1))
        few = torch.randperm(K, generator=g, device=DEV)[: max(1, K // 512)]
        x[:, few] *= 30
        spikes = torch.randint(0, rows * K, (1 + rows * K // 100000,), generator=g, device=DEV)
        x.view(-1)[spikes] *= 100
    else:
        x = 0.02 * _randn(g, rows, K)
    x = x.to(dt)
    if case["layout"] == "kn":
        x = x.t().contiguous()
    if case["signed"]:
        signs = torch.randint(0, 2, (K,), generator=g, device=DEV) * 2 - 1
    state = {"x": x, "layout": case["layout"], "block": case["block"], "signs": signs, "t": None,
             "had": _hadamard(case["block"])}
    if own and case["block"] > 1:
        import rotated_w4a4_amd as rw4
        state["t"] = rw4.Transform.hadamard(K, case["block"], None if signs is None else signs.cpu().numpy())
    return state


def _lengths(case, seed):
    """The (query, key) lengths of a case's requests, as lists; the sum of the first goes by the case."""
    g = _gen(seed, "cpu")
    n, most = case["batch"], case["q_max"]
    q = most - (torch.arange(n) * 7919) % (most - case["q_min"] + 1)
    q = q[torch.randperm(n, generator=g)]
    ctx = torch.randint(case["kv_min"], case["kv_max"] + 1, (n,), generator=g)
    return q.tolist(), (q + ctx).tolist()


def _stored(codes):
    """The stored form (uint8 [rows, D / 2]) of INT4 codes in [-7, 7] (int64 [rows, D])."""
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
             "kv_max": max(kv_len), "window": case["window"], "sinks": case["sinks"], "lse": case["lse"],
             "had": _hadamard(d)}
    state["kc"], state["ks"] = _pool(g, pages, case["kv_heads"], page, d, 0.1)
    state["vc"], state["vs"] = _pool(g, pages, case["kv_heads"], page, d, 0.3)
    return state


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "quantize":
        state = _prepare_quantize(case, g)
    elif case["op"] == "gemm":
        qa, sa = _encoded(g, case["M"], case["K"], 0.5)
        qw, sw = _encoded(g, case["N"], case["K"], 0.3)
        state = {"qa": qa, "sa": sa, "qw": qw, "sw": sw, "dtype": getattr(torch, case["dtype"])}
    else:
        state = _prepare_attention(case, g, seed)
    state["op"] = case["op"]
    return state


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------
def _sizes():
    return torch.tensor(SIZES, device=DEV)


def _plain_quantize(s):
    """In 64 bits: values lie next to borders."""
    x = s["x"].t() if s["layout"] == "kn" else s["x"]
    rows, K = x.shape
    y = x.double()
    if s["block"] > 1:
        if s["signs"] is not None:
            y = y * s["signs"]
        y = (y.reshape(-1, s["block"]) @ s["had"]) * s["block"] ** -0.5
    y = y.reshape(rows, K // 32, 32)
    E = _exponent(y)
    v = _sizes()[_index(y, E).int()] * _two(E).float()
    return [torch.where(y < 0, -v, v).reshape(rows, K).to(torch.bfloat16)]


def _opened_mx(q, s):
    """The fp32 values [rows, K] of codes and scales."""
    n = torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1, 32).int()
    v = _sizes()[n & 7]
    v = torch.where((n & 8) != 0, -v, v)
    E = s.transpose(0, 1).reshape(q.shape[0], -1, 1).int() - 127
    return (v * _two(E).float()).reshape(q.shape[0], -1)


def _plain_gemm(s):
    return [torch.matmul(_opened_mx(s["qa"], s["sa"]), _opened_mx(s["qw"], s["sw"]).t()).to(s["dtype"])]


def _i32(u):
    """The int32 with the bits of the 32-bit word u."""
    return u - (1 << 32) if u >= 1 << 31 else u


def _opened(stored):
    """The codes, as float32, of stored INT4 rows [..., D / 2]."""
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


def _plain_attention(s):
    n, rows, keys = s["kv_len"].numel(), s["q_max"], s["kv_max"]
    total, hq, d = s["q"].shape
    hk, page = s["ks"].shape[1:]
    group = hq // hk
    j = torch.arange(keys, device=DEV)
    cell = s["table"].long()[:, j // page]  # [n, keys]
    at = (cell[:, None, :] * hk + torch.arange(hk, device=DEV)[None, :, None]) * page + j % page
    kc = _opened(s["kc"].reshape(-1, d // 2)[at]) * s["ks"].reshape(-1)[at][..., None]
    cu, kv = s["cu"].long(), s["kv_len"].long()
    q_len = (cu[1:] - cu[:-1])[:, None]
    i = torch.arange(rows, device=DEV)[None, :]
    real = i < q_len
    place = (kv[:, None] - q_len + i)[..., None]
    see = (j <= place) & ((j > place - s["window"]) | (j < s["sinks"]))
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
    if s["op"] == "quantize":
        if s["layout"] == "rows":
            q, e = rw4.mx_quantize_act(s["t"], s["x"])
        else:
            q, e = rw4.mx_pack_weight(s["t"], s["x"], layout=s["layout"])
        return [rw4.mx_dequantize(q, e, torch.bfloat16)]
    if s["op"] == "gemm":
        return [rw4.mx_gemm(s["qa"], s["sa"], s["qw"], s["sw"], s["dtype"])]
    cache = rw4.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
    r = rw4.kv_attention(s["q"], cache, s["table"], s["kv_len"], s["cu"], max_q_len=s["q_max"], window=s["window"],
                         sinks=s["sinks"], return_lse=s["lse"])
    return list(r) if s["lse"] else [r]


def run(state):
    if own:
        return _own(state)
    return {"quantize": _plain_quantize, "gemm": _plain_gemm, "sink_attention": _plain_attention}[state["op"]](state)


# --------------------------------------------------------------------------
# Work
# --------------------------------------------------------------------------
def work(case):
    size = 2 if case["dtype"] == BF16 else 4
    if case["op"] == "quantize":
        n = case["rows"] * case["K"]
        # values in, codes and scales out; those read back as bf16 values
        return {"bytes": n * (size + 2 * (1 / 2 + 1 / 32) + 2), "flops": n * (6 + math.log2(case["block"]))}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K * (1 / 2 + 1 / 32) + M * N * size, "flops": 2 * M * N * K}
    d, hq, hk, n = case["dim"], case["heads"], case["kv_heads"], case["batch"]
    q = (case["q_min"] + case["q_max"]) / 2
    kv = q + (case["kv_min"] + case["kv_max"]) / 2
    read = min(kv, case["window"] + q - 1 + case["sinks"])
    seen = min(kv - (q - 1) / 2, case["window"] + case["sinks"])
    return {"bytes": n * (read * hk * (d + 8) + q * hq * (2 * size * d + (4 if case["lse"] else 0))),
            "flops": n * hq * q * seen * 4 * d}


# --------------------------------------------------------------------------
# The definitions in 64 bits, apart from the plain forms
# --------------------------------------------------------------------------
def exact(case, seed):
    def _sylvester(dim):
        h = torch.ones(1, 1, dtype=torch.float64, device=DEV)
        two = torch.tensor([[1.0, 1.0], [1.0, -1.0]], dtype=torch.float64, device=DEV)
        while h.shape[0] < dim:
            h = torch.kron(two, h)
        return h

    def _exact_quantize(s):
        x = s["x"].double()
        if s["layout"] == "kn":
            x = x.t().contiguous()
        if s["signs"] is not None:
            x = x * s["signs"].double()
        b = s["block"]
        y = (x.reshape(-1, b) @ _sylvester(b)) / math.sqrt(b)
        y = y.reshape(-1, 32)
        top = y.abs().max(1, keepdim=True).values
        # the power of two of the largest, two below: its own exponent's bits
        two = (((top.view(torch.int64) >> 52) - 2).clamp(1023 - 127, 1023 + 127) << 52).view(torch.float64)
        a = (y / two).abs().clamp(max=6.0)
        # steps of 1/2 below 2, 1 below 4, 2 from there; rounding to even within a step's numbers
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a.dtype)
        v = torch.round(a / step) * step * two
        return (torch.sign(y) * v).reshape(-1, case["K"])

    def _exact_mx(q, s):
        rows = q.shape[0]
        out = torch.empty(rows, 2 * q.shape[1], dtype=torch.float64, device=DEV)
        for half in (0, 1):
            n = (q >> (4 * half)) & 15
            e, m = ((n >> 1) & 3).double(), (n & 1).double()
            v = torch.where(e > 0, (1 + m / 2) * 2.0 ** (e - 1), m / 2)
            out[:, half::2] = v * (1 - 2 * (n >> 3).double())
        e = s.permute(1, 0, 2).reshape(rows, -1).double() - 127
        two = ((e.long() + 1023) << 52).view(torch.float64)
        return (out.reshape(rows, -1, 32) * two[..., None]).reshape(rows, -1)

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

    def _exact_attention(s):
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
            hidden = (j > place) | ((j <= place - case["window"]) & (j >= case["sinks"]))
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
    if case["op"] == "quantize":
        return [_exact_quantize(s)]
    if case["op"] == "gemm":
        return [_exact_mx(s["qa"], s["sa"]) @ _exact_mx(s["qw"], s["sw"]).t().contiguous()]
    return _exact_attention(s)
