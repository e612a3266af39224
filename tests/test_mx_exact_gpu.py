"""Codes of rotated values next to borders, against sums in whole numbers: exact up to 2^46 units a block (2^53 for blocks
of 256), one of the two neighbours beyond."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from oracle import mx as omx  # noqa: E402

if torch.cuda.is_available():
    import rotated_w4a4_amd as rw4  # noqa: E402
    from tests.kv_util import dev  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16


def _check(x, block, unit, dtype, what):
    """Whole numbers x that dtype holds, times 2^unit: both calls' codes and scales."""
    values = dev(np.ldexp(x.astype(np.float64), unit).astype(np.float32), dtype)
    assert np.array_equal(np.ldexp(values.double().cpu().numpy(), -unit), x), "the type holds the numbers"
    codes, scales = omx.quantize_whole(x, block, unit)
    t = rw4.Transform.hadamard(x.shape[1], block)
    for q, s in (rw4.mx_quantize_act(t, values), rw4.mx_pack_weight(t, values.t().contiguous())):
        assert np.array_equal(s.cpu().numpy(), omx.scale_order(scales)), what
        assert np.array_equal(omx.unpack(q.cpu().numpy()), codes), what


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [10, 30, 45, 48])
def test_what_breaks_a_tie(bits, dtype):
    # 20 / 16 is the border between 4 and 6 times 2^-2; 2^-bits more or less decides, up to 2^53 units a block
    x = np.zeros((9, 512), np.int64)
    for r, big in enumerate((20, 12, 28, 5, 24, 10, 14, 31, 1)):
        x[r, 3 * r], x[r, 3 * r + 1] = big << bits, 1
        x[r, 256 + r], x[r, 300 + r] = -((big % 29 + 3) << bits), -1
    assert np.abs(x).reshape(-1, 256).sum(1).max() < 2 ** 53
    _check(x, 256, -bits, dtype, f"2^-{bits}")


@pytest.mark.parametrize("block", [128, 512])
@pytest.mark.parametrize("off", [-2, -1, 0, 1, 2])
def test_sums_next_to_borders(block, off):
    # the whole numbers below 2^46 nearest to m sqrt(2) 2^k: the nearest is off by 2^-46.8 of it; u as two fp32 values
    rows = []
    for near in (6219777023951, 62197770239509, 388736063997, 38873606399694, 1518500249, 5 * 1518500250):
        u = near + off
        for where in (0, 77):
            x = np.zeros(1024, np.int64)
            x[where], x[where + 1] = u >> 23 << 23, u & (1 << 23) - 1
            x[block + where], x[block + where + 33] = -(u >> 23 << 23), (u & (1 << 23) - 1)
            rows.append(x)
    x = np.stack(rows)
    assert np.abs(x).reshape(-1, block).sum(1).max() < 2 ** 46
    _check(x, block, -20, F32, f"{block} {off}")


@pytest.mark.parametrize("block,spread", [(128, 14), (512, 12), (256, 20)])
def test_values_of_many_magnitudes(block, spread):
    # 24-bit values whose exponents lie as far apart as the sums' bound allows
    rng = np.random.default_rng(block)
    x = rng.integers(-2 ** 24 + 1, 2 ** 24, (6, 1024)) << rng.integers(0, spread, (6, 1024))
    assert np.abs(x).reshape(-1, block).sum(1).max() < 2 ** (53 if block == 256 else 46)
    _check(x, block, -30, F32, f"{block}")


def test_beyond_the_bound_codes_are_a_neighbour():
    # 20 and 2^-70 in one block of 256: the exact y lies 2^-74 beside the border of codes 6 and 7
    x = torch.zeros(4, 512, device="cuda")
    x[:, 0], x[:, 1] = 20.0, 2.0 ** -70
    t = rw4.Transform.hadamard(512, 256)
    for q, s in (rw4.mx_quantize_act(t, x), rw4.mx_pack_weight(t, x.t().contiguous())):
        c = omx.unpack(q.cpu().numpy())[:, :256]
        assert set(np.unique(c)) <= {6, 7} and (s[:2] == 125).all()
