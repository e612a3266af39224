"""Blocks whose codes are decided in fp32 beside blocks that are settled in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from oracle import mx as omx  # noqa: E402

if torch.cuda.is_available():
    import rotated_w4a4_amd as rw4  # noqa: E402
    from tests.kv_util import dev  # noqa: E402

F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8

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
