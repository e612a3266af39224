"""mx_gemm at the longest rows that the calls take (2^23 channels), with whole-number sums that fp32 holds exactly: the
kernel of every shape has to find each value."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

if torch.cuda.is_available():
    import rotated_w4a4_amd as rw4  # noqa: E402
    from tests.kv_util import DEV  # noqa: E402

K, GROUPS = 2 ** 23, 2 ** 16  # channels, and groups of 128
SHAPES = {"Few4": (3, 40), "Split": (70, 33), "Tile64": (700, 900), "Tile128": (1801, 2101), "Tile256": (3841, 3840)}


def _values(codes):
    """FP4 codes as float64."""
    size = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=codes.device)[(codes & 7).long()]
    return torch.where(codes >= 8, -size, size)


@pytest.mark.parametrize("kernel", list(SHAPES))
@pytest.mark.parametrize("sparse_rows", [True, False])
def test_longest_rows_are_exact(kernel, sparse_rows):
    # One operand has one value in every 16th group of 128 channels, the first and the last group among them, 4096 in
    # all; the other is random throughout.  Products are multiples of 1/4 of at most 36, so all partial sums are
    # multiples of 1/4 below 36 * 4096 < 2^22 and fp32 holds them exactly.
    M, N = SHAPES[kernel]
    g = torch.Generator(device=DEV)
    g.manual_seed(M + sparse_rows)
    rand = lambda low, high, size: torch.randint(low, high, size, dtype=torch.uint8, device=DEV, generator=g)  # noqa: E731
    group = torch.arange(GROUPS // 16, device=DEV) * 16 + torch.randint(0, 16, (GROUPS // 16,), device=DEV, generator=g)
    group[0], group[-1] = 0, GROUPS - 1
    byte = group * 64 + torch.randint(0, 64, (GROUPS // 16,), device=DEV, generator=g)  # its even channel
    thin, full = (M, N) if sparse_rows else (N, M)
    dense = rand(0, 256, (full, K // 2))
    sparse = torch.zeros(thin, K // 2, dtype=torch.uint8, device=DEV)
    sparse[:, byte] = rand(0, 16, (thin, GROUPS // 16))
    ones = [torch.full((GROUPS, n, 4), 127, dtype=torch.uint8, device=DEV) for n in (thin, full)]
    a, w = (sparse, ones[0]), (dense, ones[1])
    want = _values(sparse[:, byte]) @ _values(dense[:, byte] & 15).t().contiguous()
    assert want.abs().max() > 100 and want.unique().numel() > 100
    if sparse_rows:
        got = rw4.mx_gemm(*a, *w, torch.float32)
    else:
        got = rw4.mx_gemm(*w, *a, torch.float32).t()
    assert torch.equal(got.double(), want)
