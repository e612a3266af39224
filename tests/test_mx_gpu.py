"""MXFP4 calls on the GPU against the float64 oracle: codes and scales exactly,
values exactly, products within bounds derived from their fp32 sums."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from oracle import mx as omx  # noqa: E402

if torch.cuda.is_available():
    import rotated_w4a4_amd as rw4  # noqa: E402
    from tests.kv_util import DEV, dev, np64  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
U8 = torch.uint8


def _np(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def _rows(kind, rng, M, K):
    """Values by kind; all of them keep exact products and borders in play."""
    g = rng.standard_normal((M, K))
    if kind == "gauss":
        x = g * np.exp(0.5 * rng.standard_normal((M, 1)))
    elif kind == "outliers":
        x = g.copy()
        x[:, rng.integers(0, K, max(1, K // 100))] *= 100
        x.reshape(-1)[rng.integers(0, M * K, max(1, M * K // 5000))] *= 1000
    elif kind == "integers":  # many exact ties and zeros behind blocks of 256
        x = np.rint(3 * g)
    elif kind == "sparse":
        x = np.where(rng.random((M, K)) < 0.02, g, 0.0)
    elif kind == "constant":
        x = np.repeat(np.rint(4 * rng.standard_normal((M, 1))), K, 1)
    elif kind == "tiny":
        x = g * np.exp2(rng.integers(-149, -120, (M, 1)).astype(float))
    elif kind == "huge":
        x = np.clip(g, -3, 3) * 2.0 ** 125
    elif kind == "mixed":  # rows of every magnitude
        x = g * np.exp2(rng.integers(-130, 120, (M, 1)).astype(float))
    else:
        raise KeyError(kind)
    return x.astype(np.float32)


KINDS = ["gauss", "outliers", "integers", "sparse", "constant", "tiny", "huge", "mixed"]


def _check(got, y, what):
    """(q, s) against the definition of y, code by code."""
    codes, s = omx.quantize(y)
    q, sg = _np(got[0]), _np(got[1])
    want = omx.scale_order(s)
    assert np.array_equal(sg, want), f"{what}: {int((sg != want).sum())} scales of {sg.size} differ"
    c = omx.unpack(q)
    assert np.array_equal(c, codes), f"{what}: {int((c != codes).sum())} codes of {c.size} differ"


def _transform(K, block, signed, seed=0):
    if block == 1:
        return None, None
    signs = np.random.default_rng(seed).choice([-1, 1], K) if signed else None
    return rw4.Transform.hadamard(K, block, signs), signs


SHAPES = [(1, 128, 128), (7, 384, 128), (3, 640, 128), (33, 1152, 128), (2, 512, 256), (5, 1024, 256), (9, 2048, 512),
          (4, 512, 512), (1, 128, 1), (6, 896, 1), (130, 4096, 128), (3, 14336, 128), (17, 8192, 256)]


@pytest.mark.parametrize("M,K,block", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("signed", [False, True])
def test_codes(M, K, block, dtype, signed):
    if block == 1 and signed:
        pytest.skip("signs belong to a transform")
    rng = np.random.default_rng(M * K + block)
    t, signs = _transform(K, block, signed)
    for kind in ("gauss", "outliers"):
        x = dev(_rows(kind, rng, M, K), dtype)
        _check(rw4.mx_quantize_act(t, x), omx.rotate(np64(x), block, signs), f"{kind} {M}x{K}/{block}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("block", [1, 128, 256, 512])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_codes_of_values_of_every_kind(kind, block, dtype):
    rng = np.random.default_rng(11)
    M, K = 24, 1024
    t, signs = _transform(K, block, False)
    x = dev(_rows(kind, rng, M, K), dtype)
    if kind == "huge":
        x = x.clamp(-3e38, 3e38)
    _check(rw4.mx_quantize_act(t, x), omx.rotate(np64(x), block, signs), f"{kind} /{block}")


def test_many_codes():
    # 8 million codes: borders that fp32 alone would miss now and then
    rng = np.random.default_rng(5)
    x = dev(_rows("outliers", rng, 2048, 4096), BF16)
    t, _ = _transform(4096, 128, False)
    _check(rw4.mx_quantize_act(t, x), omx.rotate(np64(x), 128), "2048x4096")


@pytest.mark.parametrize("block", [128, 256, 512])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["gauss", "outliers"])
def test_many_codes_of_every_block(kind, block, dtype):
    # a few values of a wave near a border, and exact ties (block 256 of bf16)
    rng = np.random.default_rng(50 + block)
    x = dev(_rows(kind, rng, 515, 4096), dtype)
    t, signs = _transform(4096, block, block == 512)
    y = omx.rotate(np64(x), block, signs)
    _check(rw4.mx_quantize_act(t, x), y, "rows")
    _check(rw4.mx_pack_weight(t, x.t().contiguous()), y, "columns")


@pytest.mark.parametrize("kind", ["gauss", "integers"])
def test_many_rows(kind):
    # rows enough for four at a time, and the last ones fewer: the same rows again in a small call
    rng = np.random.default_rng(60)
    x = dev(_rows(kind, rng, 1003, 512), BF16).repeat(34, 1)[:34101]
    t, signs = _transform(512, 256, False)
    q, s = rw4.mx_quantize_act(t, x)
    _check((q[:1003].contiguous(), s[:, :1003].contiguous()), omx.rotate(np64(x[:1003]), 256), "first")
    assert torch.equal(q[1003:33099].view(-1, 1003, 256), q[:1003].expand(32, 1003, 256))
    assert torch.equal(q[33099:], q[:1002])
    assert torch.equal(s[:, 1003:33099].view(4, -1, 1003, 4), s[:, None, :1003].expand(4, 32, 1003, 4))
    assert torch.equal(s[:, 33099:], s[:, :1002])


@pytest.mark.parametrize("block", [1, 128, 512])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_not_finite(block, dtype):
    rng = np.random.default_rng(6)
    x = dev(_rows("gauss", rng, 5, 1024), dtype)
    x[1, 70], x[2, 600], x[3, 1023], x[4, 0] = float("nan"), float("inf"), float("-inf"), float("inf")
    x[4, 1] = float("-inf")
    t, _ = _transform(1024, block, False)
    y = np64(x)
    if block > 1:
        bad = ~np.isfinite(y.reshape(5, -1, block)).all(-1)
        y = omx.rotate(np.where(np.isfinite(y), y, 0.0), block).reshape(5, -1, block)
        y[bad] = np.nan  # the Hadamard spreads it
        y = y.reshape(5, 1024)
    got = rw4.mx_quantize_act(t, x)
    _check(got, y, "not finite")
    v = rw4.mx_dequantize(*got, F32)
    assert torch.isnan(v).any(1).tolist() == [False, True, True, True, True]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_in_a_wider_tensor(dtype):
    rng = np.random.default_rng(7)
    wide = dev(_rows("gauss", rng, 9, 1024 + 128), dtype)
    x = wide[:, 64:64 + 1024]
    t, _ = _transform(1024, 128, False)
    q = torch.full((9, 512), 0xEE, dtype=U8, device=DEV)
    s = torch.full((8, 9, 4), 0xEE, dtype=U8, device=DEV)
    got = rw4.mx_quantize_act(t, x, q=q, s=s)
    assert got[0] is q and got[1] is s
    _check(got, omx.rotate(np64(x), 128), "a view")


@pytest.mark.parametrize("N,K,block,signed", [(1, 128, 128, False), (5, 384, 128, True), (33, 1024, 256, False),
                                              (64, 512, 512, True), (100, 640, 1, False), (31, 1536, 128, False)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("form", ["kn", "nk", "nk_odd", "kn_wide", "both"])
def test_pack_weight(N, K, block, signed, dtype, form):
    rng = np.random.default_rng(N + K)
    w = _rows("gauss", rng, N, K) * 0.02
    t, signs = _transform(K, block, signed)
    if form == "kn":
        a, layout = dev(w.T, dtype), "kn"
    elif form == "nk":
        a, layout = dev(w, dtype), "nk"
    elif form == "nk_odd":  # rows that are not 16-byte aligned
        a, layout = torch.zeros(N, K + 1, dtype=dtype, device=DEV)[:, 1:], "nk"
        a.copy_(dev(w, dtype))
    elif form == "kn_wide":  # every second channel of a wider matrix
        a, layout = torch.zeros(K, 2 * N + 3, dtype=dtype, device=DEV)[:, 3::2][:, :N], "kn"
        a.copy_(dev(w.T, dtype))
    else:
        a, layout = torch.zeros(2 * K, N, 3, dtype=dtype, device=DEV)[::2, :, 1], "kn"
        a.copy_(dev(w.T, dtype))
    got = rw4.mx_pack_weight(t, a, layout=layout)
    y = np64(a) if layout == "nk" else np64(a).T
    _check(got, omx.rotate(np.ascontiguousarray(y), block, signs), form)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_dequantize_every_code_and_scale(dtype):
    rng = np.random.default_rng(8)
    M, K = 37, 8192
    codes = rng.integers(0, 16, (M, K)).astype(np.uint8)
    s = np.arange(M * K // 32).reshape(M, -1) % 256
    s = s.astype(np.uint8)
    out = torch.full((M, K + 8), 3.0, dtype=dtype, device=DEV)
    rw4.mx_dequantize(dev(omx.pack(codes)), dev(omx.scale_order(s)), out=out[:, :K])
    want = omx.values(codes, s)
    big = np.abs(want) > torch.finfo(dtype).max  # 2^127 times 2 and more leave both types
    got = np64(out[:, :K])
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.isinf(got[big]).all() and np.array_equal(np.sign(got[big]), np.sign(want[big]))
    keep = ~big & ~np.isnan(want)
    assert np.array_equal(got[keep], want[keep])
    assert (out[:, K:] == 3.0).all()


def _operand(rng, rows, K, spread=4):
    codes = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    s = (127 + rng.integers(-spread, spread + 1, (rows, K // 32))).astype(np.uint8)
    return codes, s


def _gemm_check(ca, sa, cw, sw, dtype, ldy=None, what=""):
    M, N, K = ca.shape[0], cw.shape[0], ca.shape[1]
    want, size = omx.gemm(ca, sa, cw, sw)
    wide = torch.full((M + 1, (N if ldy is None else ldy) + 3), 7.0, dtype=dtype, device=DEV)
    out = wide[:M, :N]
    rw4.mx_gemm(dev(omx.pack(ca)), dev(omx.scale_order(sa)), dev(omx.pack(cw)), dev(omx.scale_order(sw)), out=out)
    got = np64(out)
    # K products added in fp32, each addition off by one unit in the last place at most
    # (2^-23, whichever way it rounds) of a partial sum that `size` bounds; then the
    # output's own rounding
    tol = K * 2.0 ** -23 * size + torch.finfo(dtype).eps / 2 * np.abs(want) + 1e-38
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    err = np.where(np.isnan(want), 0.0, np.abs(got - want))
    assert (err <= np.nan_to_num(tol, nan=1.0)).all(), (what, float((err - tol)[err > tol].max()), int((err > tol).sum()))
    assert (wide[M:] == 7.0).all() and (wide[:, N:] == 7.0).all(), what


GEMMS = [(1, 1, 128), (1, 16, 128), (2, 17, 256), (7, 100, 384), (16, 64, 2176), (17, 33, 512), (33, 130, 1152),
         (64, 48, 4096), (65, 129, 128), (100, 1, 640), (128, 128, 256), (129, 257, 384), (200, 513, 2048),
         (257, 300, 640), (300, 1000, 1408), (1000, 72, 896), (511, 511, 1152), (640, 640, 128), (500, 1100, 384),
         (449, 1001, 256), (900, 901, 2176)]


@pytest.mark.parametrize("M,N,K", GEMMS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gemm(M, N, K, dtype):
    rng = np.random.default_rng(M + 3 * N + K)
    _gemm_check(*_operand(rng, M, K), *_operand(rng, N, K), dtype, what=f"{M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", [(5, 40, 14336), (3, 70, 14336), (4, 1001, 8192), (1, 33, 4224), (77, 96, 4224),
                                   (140, 270, 4096), (61, 800, 14336), (600, 520, 1024), (700, 1300, 1152),
                                   (2100, 700, 640), (3841, 4093, 640), (4096, 3588, 384), (1700, 1500, 128)])
def test_gemm_of_whole_numbers_is_exact(M, N, K):
    # scales of 1: products are multiples of 1/4, sums stay below 36 K < 2^22, so fp32 holds each exactly
    rng = np.random.default_rng(M)
    ca, cw = (rng.integers(0, 16, (r, K)).astype(np.uint8) for r in (M, N))
    one_a, one_w = np.full((M, K // 32), 127, np.uint8), np.full((N, K // 32), 127, np.uint8)
    want, _ = omx.gemm(ca, one_a, cw, one_w)
    got = rw4.mx_gemm(dev(omx.pack(ca)), dev(omx.scale_order(one_a)), dev(omx.pack(cw)), dev(omx.scale_order(one_w)), F32)
    assert np.array_equal(np64(got), want)


@pytest.mark.parametrize("M,N,K", [(3, 20, 512), (40, 50, 640), (150, 140, 640), (520, 700, 640)])
def test_gemm_places_every_block(M, N, K):
    # one block of one row of each side is not zero: the product shows where its codes and scales went
    rng = np.random.default_rng(9)
    for b in range(K // 32):
        ca, cw = np.zeros((M, K), np.uint8), np.zeros((N, K), np.uint8)
        m, n = int(rng.integers(M)), int(rng.integers(N))
        ca[m, 32 * b:32 * b + 32] = rng.integers(1, 8, 32)
        cw[n, 32 * b:32 * b + 32] = rng.integers(1, 8, 32)
        sa = rng.integers(100, 150, (M, K // 32)).astype(np.uint8)
        sw = rng.integers(100, 150, (N, K // 32)).astype(np.uint8)
        want, _ = omx.gemm(ca, sa, cw, sw)
        got = rw4.mx_gemm(dev(omx.pack(ca)), dev(omx.scale_order(sa)), dev(omx.pack(cw)), dev(omx.scale_order(sw)), F32)
        assert np.array_equal(np64(got), want), b


@pytest.mark.parametrize("M,N", [(2, 30), (40, 40), (150, 140), (700, 700)])
def test_gemm_scales_at_their_ends(M, N):
    rng = np.random.default_rng(10)
    ca, sa = _operand(rng, M, 256)
    cw, sw = _operand(rng, N, 256)
    sa[0], sw[0] = 254, 1      # 2^127 and 2^-126: their products are ordinary
    sa[1, 3] = 255             # a row of NaN
    sw[5, 0] = 255             # a column of NaN
    sa[0, :] = 254
    sw[1:, :] = rng.integers(1, 20, sw[1:].shape)
    sw[5, 0] = 255
    _gemm_check(ca, sa, cw, sw, F32, what="ends")


def test_empty():
    q0, s0 = torch.empty(0, 64, dtype=U8, device=DEV), torch.empty(1, 0, 4, dtype=U8, device=DEV)
    q1, s1 = torch.zeros(3, 64, dtype=U8, device=DEV), torch.full((1, 3, 4), 127, dtype=U8, device=DEV)
    assert rw4.mx_quantize_act(None, torch.empty(0, 128, device=DEV))[0].shape == (0, 64)
    assert rw4.mx_pack_weight(None, torch.empty(128, 0, device=DEV))[0].shape == (0, 64)
    assert rw4.mx_dequantize(q0, s0).shape == (0, 128)
    assert rw4.mx_gemm(q0, s0, q1, s1).shape == (0, 3)
    assert rw4.mx_gemm(q1, s1, q0, s0).shape == (3, 0)
    torch.cuda.synchronize()


def test_refusals():
    x = torch.zeros(4, 256, device=DEV)
    q, s = rw4.mx_quantize_act(None, x)
    t = rw4.Transform.hadamard(512, 128)
    with pytest.raises(ValueError):
        rw4.mx_quantize_act(t, x)
    with pytest.raises(ValueError):
        rw4.mx_quantize_act(None, x[:, ::2])
    with pytest.raises(ValueError):
        rw4.mx_quantize_act(None, torch.zeros(4, 200, device=DEV))
    with pytest.raises(TypeError):
        rw4.mx_quantize_act(None, x.half())
    with pytest.raises(ValueError):
        rw4.mx_quantize_act(None, x, q=torch.empty(4, 127, dtype=U8, device=DEV))
    with pytest.raises(rw4.RW4Error):
        rw4.mx_quantize_act(None, torch.zeros(4, 257, device=DEV)[:, 1:])  # rows not aligned
    with pytest.raises(rw4.RW4Error, match="UNSUPPORTED"):
        rw4.mx_quantize_act(rw4.Transform.hadamard(1024, 1024), torch.zeros(4, 1024, device=DEV))
    with pytest.raises(ValueError):
        rw4.mx_pack_weight(None, x, layout="mn")
    with pytest.raises(ValueError):
        rw4.mx_gemm(q, s, q[:, :64].contiguous(), s[:1])
    with pytest.raises(ValueError):
        rw4.mx_gemm(q, s[:, :3], q, s)
    with pytest.raises(ValueError):
        rw4.mx_gemm(q, s.float(), q, s)
    with pytest.raises(ValueError):
        rw4.mx_gemm(q, s, q, s, out=torch.empty(4, 5, device=DEV))
    with pytest.raises(TypeError):
        rw4.mx_gemm(q, s, q, s, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        rw4.mx_gemm(q, s, q, s, out_dtype=BF16, out=torch.empty(4, 4, device=DEV))
    with pytest.raises(ValueError):
        rw4.mx_dequantize(q, s, out=torch.empty(4, 255, device=DEV))
