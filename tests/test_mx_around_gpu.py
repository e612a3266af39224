"""The MXFP4 quantizers write their codes and scales and nothing else: outputs between poisoned bytes, rows that end inside
a wave's 512 channels, single and many rows; blocks whose codes are decided beside blocks that are settled in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from oracle import mx as omx  # noqa: E402

if torch.cuda.is_available():
    import rotated_w4a4_amd as rw4  # noqa: E402
    from tests.kv_util import DEV, dev, np64  # noqa: E402

F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8
AROUND = 1 << 16


def _between(*shape):
    """A contiguous uint8 tensor of `shape` with 64 KB of 0xEE on both sides, and the check that those stay."""
    n = int(np.prod(shape))
    flat = torch.full((n + 2 * AROUND + 16,), 0xEE, dtype=U8, device=DEV)

    def stays():
        assert (flat[:AROUND] == 0xEE).all() and (flat[AROUND + n:] == 0xEE).all()

    return flat[AROUND:AROUND + n].view(*shape), stays


@pytest.mark.parametrize("M,K,block", [(1, 128, 1), (1, 384, 128), (3, 640, 128), (2, 512, 256), (5, 512, 512), (257, 1152, 1),
                                       (35003, 640, 128), (33000, 128, 1), (34001, 512, 256)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_outputs_end_where_they_end(M, K, block, dtype):
    rng = np.random.default_rng(M + K)
    few = min(M, 1001)
    x = dev(rng.standard_normal((few, K)).astype(np.float32), dtype).repeat(-(-M // few), 1)[:M]
    t = None if block == 1 else rw4.Transform.hadamard(K, block)
    codes, scales = omx.quantize(omx.rotate(np64(x[:few]), block))
    for call in (lambda **out: rw4.mx_quantize_act(t, x, q=out["q"], s=out["s"]),
                 lambda **out: rw4.mx_pack_weight(t, x.t().contiguous(), qw=out["q"], sw=out["s"])):
        (q, q_stays), (s, s_stays) = _between(M, K // 2), _between(K // 128, M, 4)
        call(q=q, s=s)
        q_stays()
        s_stays()
        want_q, want_s = dev(omx.pack(codes)), dev(omx.scale_order(scales))
        rows = torch.arange(M, device=DEV) % few
        assert torch.equal(q, want_q[rows]) and torch.equal(s, want_s[:, rows])


@pytest.mark.parametrize("block", [128, 256])
def test_settled_blocks_leave_the_others_alone(block):
    # one block of a wave has an exact tie (or a value next to a border), the others are far from any: every value of
    # theirs, the first one too, keeps its code
    rng = np.random.default_rng(block)
    K = 1024
    x = np.zeros((64, K), np.int64)
    for r in range(64):
        b = r % (512 // block)
        x[r] = 7 * rng.integers(1, 1000, K)
        x[r, b * block:(b + 1) * block] = 0
        # block 256: 20 / 16, the border of 4 and 6; block 128: whole numbers next to 5 2^14 sqrt(2)
        x[r, b * block + r] = 20 if block == 256 else round(5 * 2 ** 14 * 2 ** 0.5)
    xf = dev(x.astype(np.float32))
    codes, scales = omx.quantize_whole(x, block, 0)
    t = rw4.Transform.hadamard(K, block)
    for q, s in (rw4.mx_quantize_act(t, xf), rw4.mx_pack_weight(t, xf.t().contiguous())):
        assert np.array_equal(omx.unpack(q.cpu().numpy()), codes) and np.array_equal(s.cpu().numpy(), omx.scale_order(scales))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_beyond_the_types_range(dtype):
    # a Hadamard of finite values that reaches 2^130: codes and scales hold it (saturating at 6 2^127), reading it back
    # gives infinity, the product with small weights is finite again
    K = 256
    x = torch.full((3, K), 2.0 ** 127, dtype=dtype, device=DEV)
    x[1, 128:] = 2.0 ** 124
    x[2] = -x[2]
    q, s = rw4.mx_quantize_act(rw4.Transform.hadamard(K, 128), x)
    codes, scales = omx.quantize(omx.rotate(np64(x), 128))
    assert np.array_equal(omx.unpack(q.cpu().numpy()), codes) and np.array_equal(s.cpu().numpy(), omx.scale_order(scales))
    # sqrt(128) 2^127 = 2^130.5 is 6 at 2^127; sqrt(128) 2^124 = 5.66 2^125
    big = [torch.inf, torch.inf, -torch.inf]
    small = [torch.inf, 6 * 2.0 ** 125, -torch.inf]
    back = rw4.mx_dequantize(q, s, dtype)
    assert back[:, 0].tolist() == big and back[:, 128].tolist() == small
    w = torch.zeros(2, K, device=DEV)
    w[0, 0], w[1, 128] = 2.0 ** -100, 2.0 ** -110
    y = rw4.mx_gemm(q, s, *rw4.mx_quantize_act(None, w), F32)
    assert y.tolist() == [[6 * 2.0 ** 27, 6 * 2.0 ** 17], [6 * 2.0 ** 27, 6 * 2.0 ** 15], [-6 * 2.0 ** 27, -6 * 2.0 ** 17]]
