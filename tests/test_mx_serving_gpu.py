"""The MXFP4 calls as a serving loop uses them: a decoder layer of MXFP4 products around
the INT4 cache's attention with a window and sinks, captured steps, two streams at
once, buffers that are reused, tensors beyond 32-bit offsets."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from oracle import kv as okv  # noqa: E402
from oracle import mx as omx  # noqa: E402

if torch.cuda.is_available():
    import rotated_w4a4_amd as rw4  # noqa: E402
    from tests import kv_util as ku  # noqa: E402

F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8


class _Layer:
    """A decoder layer's attention part: MXFP4 projections, an INT4 cache, a window with sinks."""

    def __init__(self, B, pages, page, width, hq=4, hk=2, D=128, K=512, window=24, sinks=3):
        rng = np.random.default_rng(21)
        self.dims, self.page, self.window, self.sinks = (hq, hk, D, K), page, window, sinks
        self.t, self.to = rw4.Transform.hadamard(K, 128), rw4.Transform.hadamard(hq * D, 256)
        n = (hq + 2 * hk) * D
        self.w_qkv = ku.dev((rng.standard_normal((K, n)) * K ** -0.5).astype(np.float32))
        self.w_o = ku.dev((rng.standard_normal((K, hq * D)) * K ** -0.5).astype(np.float32), BF16)
        self.qkv = rw4.mx_pack_weight(self.t, self.w_qkv)
        self.o = rw4.mx_pack_weight(self.to, self.w_o, layout="nk")
        self.wq, self.wk = (ku.dev((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)) for _ in range(2))
        self.rope = rw4.rope_table(4096, D)
        self.cache = rw4.KVCache.empty(pages, page, hk, D)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device=ku.DEV)
        self.ring = torch.arange(pages, dtype=torch.int32, device=ku.DEV)
        self.state = torch.tensor([0, pages], dtype=torch.int32, device=ku.DEV)
        self.kv = torch.zeros(B, dtype=torch.int32, device=ku.DEV)

    def step(self, x, new, most):
        hq, hk, D, K = self.dims
        T = x.shape[0]
        s = rw4.kv_slots(self.kv, new, self.table, self.ring, self.state, self.page, T, kv_len=self.kv,
                         free_state_out=self.state)
        y = rw4.mx_gemm(*rw4.mx_quantize_act(self.t, x), *self.qkv)
        h = y.view(T, hq + 2 * hk, D)
        q = rw4.kv_append(self.cache, h[:, hq:hq + hk], h[:, hq + hk:], s.slot_map, h[:, :hq], self.wq, self.wk,
                          self.rope, s.positions)
        o = rw4.kv_attention(q, self.cache, self.table, self.kv, s.cu_new, max_q_len=most, window=self.window,
                             sinks=self.sinks, out=torch.zeros_like(q))
        z = rw4.mx_gemm(*rw4.mx_quantize_act(self.to, o.view(T, hq * D)), *self.o)
        return y, o, z


def _x(seed, T, K=512):
    return ku.dev(np.random.default_rng(seed).standard_normal((T, K)).astype(np.float32), BF16)


def _product(x, block, w_rows):
    """(product, sums of sizes) of the definition: rows x and weight rows [N, K], both quantized."""
    a, sa = omx.quantize(omx.rotate(x, block))
    w, sw = omx.quantize(omx.rotate(w_rows, block))
    return omx.gemm(a, sa, w, sw)


def _close_product(got, want, size, K, what):
    ku.close(got, want, K * 2.0 ** -23 * size + ku.half_step(BF16) * np.abs(want) + 1e-30, what)


def test_serving_run_matches_oracle():
    layer = _Layer(B=3, pages=30, page=16, width=12)
    hq, hk, D, K = layer.dims
    past = [[], [], []]
    cs, wq, wk = ku.np64(layer.rope), ku.np64(layer.wq), ku.np64(layer.wk)
    w_qkv, w_o = np.ascontiguousarray(ku.np64(layer.w_qkv).T), ku.np64(layer.w_o)
    for n, new in enumerate([[20, 70, 1], [1, 1, 1], [2, 1, 40], [1, -1, 1], [1, 90, 1], [1, 1, 1]]):
        total = sum(max(v, 0) for v in new)
        T = total + 2
        x = _x(n, T)
        y, o, z = layer.step(x, ku.dev(np.array(new, np.int32)), max(new))
        y, o64 = ku.np64(y), ku.np64(o)
        _close_product(y, *_product(ku.np64(x), 128, w_qkv), K, f"step {n} qkv")
        _close_product(ku.np64(z), *_product(o64.reshape(T, hq * D), 256, w_o), hq * D, f"step {n} o")
        rows = y.reshape(T, hq + 2 * hk, D)
        at = 0
        for b, add in enumerate(new):
            past[b] = [] if add < 0 else past[b] + [rows[at + i] for i in range(add)]
            add = max(add, 0)
            if add:
                all_rows = np.stack(past[b])
                L = len(all_rows)
                pos = np.arange(L)
                zk, fk = okv.norm_rope(all_rows[:, hq:hq + hk], wk, 1e-6, cs, pos, False)
                ck, sk = okv.quantize_heads(zk, fk, True)
                cv, sv = okv.quantize_heads(all_rows[:, hq + hk:], np.ones((L, hk, 1)), True)
                zq, fq = okv.norm_rope(all_rows[L - add:, :hq], wq, 1e-6, cs, pos[L - add:], False)
                qb = ku.np64(ku.dev(okv.rotate_heads(zq * fq).astype(np.float32), BF16))
                pages = -(-L // 16)

                def paged(v):
                    v = np.concatenate([v, np.zeros((pages * 16 - L,) + v.shape[1:], v.dtype)])
                    return np.moveaxis(v.reshape((pages, 16) + v.shape[1:]), 1, 2)

                want, _, reach, size = okv.kv_attention(qb, paged(ck), paged(sk), paged(cv), paged(sv), pages,
                                                        np.arange(pages)[None], [L], [0, add], D ** -0.5, True,
                                                        layer.window, True, layer.sinks)
                # a query may round to the neighbouring bf16 where the two evaluations straddle a border: one step,
                # 2 half_step, in one of D products at most enters a score
                tol = ku.attention_tolerance(want, reach, size, BF16, D, L) + (
                    4 * ku.half_step(BF16) * size * reach)[..., None]
                ku.close(o64[at:at + add], want, tol, f"step {n} request {b}")
            at += add


def test_captured_step_replays():
    B = 3
    eager, graphed = (_Layer(B, pages=40, page=16, width=12) for _ in range(2))
    first = np.array([50, 30, 1], np.int32)
    for layer in (eager, graphed):
        layer.step(_x(50, int(first.sum())), ku.dev(first), 50)
    one, x = ku.dev(np.ones(B, np.int32)), _x(51, B)
    keep = [t.clone() for t in (graphed.kv, graphed.state, graphed.table, graphed.ring)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.step(x, one, 1)
    torch.cuda.current_stream().wait_stream(side)
    for t, o in zip((graphed.kv, graphed.state, graphed.table, graphed.ring), keep):
        t.copy_(o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, o, z = graphed.step(x, one, 1)
    for n in range(5):
        x.copy_(_x(60 + n, B))
        g.replay()
        junk = torch.randn(1000, device=ku.DEV).sum()  # unrelated eager work between replays
        torch.cuda.synchronize()
        ey, eo, ez = eager.step(x, one, 1)
        torch.cuda.synchronize()
        assert torch.equal(y, ey) and torch.equal(o, eo) and torch.equal(z, ez) and torch.isfinite(junk)
        assert torch.equal(graphed.kv, eager.kv)
    assert torch.equal(graphed.cache.k, eager.cache.k)


# M: the kernels for few rows, and each size of tile (64, 128, 256 tokens)
@pytest.mark.parametrize("M,N", [(1, 300), (30, 200), (300, 500), (1500, 2100), (3700, 3900)])
def test_captured_product_replays(M, N):
    K = 640
    rng = np.random.default_rng(M)
    t = rw4.Transform.hadamard(K, 128)
    x = ku.dev(rng.standard_normal((M, K)).astype(np.float32), BF16)
    qw, sw = rw4.mx_pack_weight(t, ku.dev(rng.standard_normal((K, N)).astype(np.float32)))
    q, s, out = (torch.empty(M, K // 2, dtype=U8, device=ku.DEV), torch.empty(K // 128, M, 4, dtype=U8, device=ku.DEV),
                 torch.empty(M, N, dtype=BF16, device=ku.DEV))
    calls = [rw4.prepare_mx_quantize_act(t, x, q, s), rw4.prepare_mx_gemm(q, s, qw, sw, out=out),
             rw4.prepare_mx_dequantize(q, s, F32)]
    back = calls[2].result
    for c in calls:
        c()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in calls:
            c()
    for n in range(3):
        x.copy_(ku.dev((rng.standard_normal((M, K)) * 10.0 ** n).astype(np.float32), BF16))
        g.replay()
        torch.cuda.synchronize()
        eq, es = rw4.mx_quantize_act(t, x)
        assert torch.equal(q, eq) and torch.equal(s, es)
        assert torch.equal(out, rw4.mx_gemm(eq, es, qw, sw)) and torch.equal(back, rw4.mx_dequantize(eq, es, F32))


def test_two_streams_at_once():
    rng = np.random.default_rng(30)
    K = 1024
    t = rw4.Transform.hadamard(K, 256)
    xs = [ku.dev(rng.standard_normal((m, K)).astype(np.float32)) for m in (500, 37)]
    qw, sw = rw4.mx_pack_weight(t, ku.dev(rng.standard_normal((K, 700)).astype(np.float32)))
    want = [rw4.mx_gemm(*rw4.mx_quantize_act(t, x), qw, sw) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(4):
        for i, (x, st) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(st):
                got[i].append(rw4.mx_gemm(*rw4.mx_quantize_act(t, x), qw, sw))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_offsets_beyond_32_bits():
    # codes of more than 4 GiB and values of 20: the last rows against calls of their own
    M, K, N, last = 600001, 16384, 40, 77
    x = torch.empty(M, K, dtype=BF16, device=ku.DEV)
    g = torch.Generator(device=ku.DEV)
    g.manual_seed(1)
    x.normal_(generator=g)
    t = rw4.Transform.hadamard(K, 128)
    q, s = rw4.mx_quantize_act(t, x)
    assert q.numel() > 2 ** 32
    for rows in (slice(M - last, M), slice(0, last), slice(262143, 262143 + last)):
        eq, es = rw4.mx_quantize_act(t, x[rows])
        assert torch.equal(q[rows], eq) and torch.equal(s[:, rows], es)
    # weights as [K, N] of the same size: the pack's loads
    wide = x.view(K, M)[:, M - last:]
    pq, ps = rw4.mx_pack_weight(None, wide)
    eq, es = rw4.mx_pack_weight(None, wide.contiguous())
    assert torch.equal(pq, eq) and torch.equal(ps, es)
    del wide
    rw4.mx_dequantize(q, s, out=x)
    eq, es = q[M - last:].contiguous(), s[:, M - last:].contiguous()
    assert torch.equal(x[M - last:], rw4.mx_dequantize(eq, es))
    qw, sw = rw4.mx_quantize_act(None, torch.randn(N, K, device=ku.DEV))
    y = rw4.mx_gemm(q, s, qw, sw, F32)
    ref = x[M - last:].double() @ rw4.mx_dequantize(qw, sw, F32).double().t().contiguous()
    size = x[M - last:].double().abs() @ rw4.mx_dequantize(qw, sw, F32).double().abs().t().contiguous()
    assert ((y[M - last:].double() - ref).abs() <= K * 2.0 ** -23 * size + 1e-30).all()
    # and as the weights
    y = rw4.mx_gemm(qw, sw, q, s, F32)
    assert ((y[:, M - last:].double().t() - ref).abs() <= K * 2.0 ** -23 * size + 1e-30).all()


@pytest.mark.parametrize("M", [1, 8])
def test_single_tokens_times_more_channels_than_a_grid_of_16_holds(M):
    K, N = 128, 2 ** 27 + 40
    g = torch.Generator(device=ku.DEV)
    g.manual_seed(2)
    qw = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=ku.DEV, generator=g)
    sw = torch.randint(124, 130, (1, N, 4), dtype=torch.uint8, device=ku.DEV, generator=g)
    qa, sa = qw[77:77 + M].clone(), sw[:, 77:77 + M].clone()
    y = rw4.mx_gemm(qa, sa, qw, sw, F32)
    a = rw4.mx_dequantize(qa, sa, F32).double()
    for first in (0, 2 ** 26 - 50, 2 ** 27 - 60, N - 100):
        w = rw4.mx_dequantize(qw[first:first + 100].clone(), sw[:, first:first + 100].clone(), F32).double().t()
        w = w.contiguous()
        # fp32 sums of 128 exact products: half a step of at most their sum of sizes each
        tol = K * 2.0 ** -24 * (a.abs() @ w.abs())
        assert ((y[:, first:first + 100].double() - a @ w).abs() <= tol).all(), first


@pytest.mark.parametrize("M,N", [(1, 5), (3, 40), (70, 33)])
def test_longest_rows(M, N):
    # K = 2^23: codes are those of the row's pieces; the product against sums in 64 bits
    K, piece = 2 ** 23, 4096
    g = torch.Generator(device=ku.DEV)
    g.manual_seed(3)
    a = torch.randn(M, K, device=ku.DEV, generator=g).to(BF16)
    w = torch.randn(N, K, device=ku.DEV, generator=g).to(BF16)
    qa, sa = rw4.mx_quantize_act(None, a)
    qw, sw = rw4.mx_pack_weight(None, w, layout="nk")
    eq, es = rw4.mx_quantize_act(None, a.view(-1, piece))
    assert torch.equal(qa.view(-1, piece // 2), eq)
    assert torch.equal(sa.view(K // piece, piece // 128, M, 4), es.view(piece // 128, M, K // piece, 4).permute(2, 0, 1, 3))
    a, w = rw4.mx_dequantize(qa, sa), rw4.mx_dequantize(qw, sw)
    want = torch.zeros(M, N, dtype=torch.float64, device=ku.DEV)
    size = torch.zeros_like(want)
    for k in range(0, K, 2 ** 18):
        x, z = a[:, k:k + 2 ** 18].double(), w[:, k:k + 2 ** 18].double().t().contiguous()
        want += x @ z
        size += x.abs() @ z.abs()
    y = rw4.mx_gemm(qa, sa, qw, sw, F32)
    # a product of 128 channels and its addition round within 128 half steps of what they add; K / 128 of them in a row
    tol = (K / 128 + 128) * 2.0 ** -24 * size
    assert ((y.double() - want).abs() <= tol).all()


def test_results_do_not_depend_on_the_other_rows():
    # a row alone, among others, and beside rows of NaN: the same codes; the product of the same kernel the same bits
    rng = np.random.default_rng(31)
    K = 512
    t = rw4.Transform.hadamard(K, 128)
    x = ku.dev(rng.standard_normal((9, K)).astype(np.float32))
    q, s = rw4.mx_quantize_act(t, x)
    one_q, one_s = rw4.mx_quantize_act(t, x[4:5])
    assert torch.equal(q[4:5], one_q) and torch.equal(s[:, 4:5], one_s)
    qw, sw = rw4.mx_pack_weight(t, ku.dev(rng.standard_normal((K, 50)).astype(np.float32)))
    y = rw4.mx_gemm(q, s, qw, sw)
    x[3], x[5] = float("nan"), float("inf")
    q2, s2 = rw4.mx_quantize_act(t, x)
    y2 = rw4.mx_gemm(q2, s2, qw, sw)
    keep = [0, 1, 2, 4, 6, 7, 8]
    assert torch.equal(y2[keep], y[keep]) and torch.isnan(y2[[3, 5]]).all()


def test_scales_of_a_checkpoint():
    # scales stored by rows, as files of this format hold them
    rng = np.random.default_rng(32)
    N, K = 33, 640
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    s = rng.integers(120, 130, (N, K // 32)).astype(np.uint8)
    qw, sw = ku.dev(omx.pack(codes)), rw4.mx_scale_rows(ku.dev(s))
    assert np.array_equal(ku.np64(rw4.mx_dequantize(qw, sw, F32)), omx.values(codes, s))
