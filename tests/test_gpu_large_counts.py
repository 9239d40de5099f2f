"""Calls of as many rows as their 32-bit counts hold, where sums of a count and a
tile or a grid's size pass 31 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_mixture_experts_15_b200 as moe

R = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def _memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of device memory")
    moe.moe_reset_device_status()
    yield
    assert moe.moe_device_status() == 0
    torch.cuda.empty_cache()


def ends(t):
    """The first and the last rows."""
    return torch.cat([t[:1000], t[-1000:]])


def test_grouped_product():
    x = torch.zeros(R, 16, dtype=torch.int8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    for part in (x[:1000], x[-1000:]):
        part.copy_(torch.randint(-128, 128, (1000, 16), generator=g, device="cuda"))
    xs = torch.ones(R, device="cuda")
    w = torch.randint(-128, 128, (1, 16), generator=g, device="cuda", dtype=torch.int8)
    y = torch.full((R, 1), 7.0, dtype=torch.float16, device="cuda")
    moe.moe_grouped_gemm_i8(x, xs, w, torch.full((1,), 0.125, device="cuda"), y)
    ref = ends(x).double() @ w.double().T * 0.125
    # the sum is below 2^18 and exact in fp32, the scales are powers of two: one rounding
    assert ((ends(y).double() - ref).abs() <= ref.abs() * 2.0 ** -11).all()
    assert (y[1000:-1000] == 0).all()
