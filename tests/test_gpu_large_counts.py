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


def test_block_norm():
    d, g = 8, torch.Generator(device="cuda").manual_seed(1)
    x = torch.ones(R, d, dtype=torch.bfloat16, device="cuda")
    for part in (x[:1000], x[-1000:]):
        part.copy_(torch.randn(1000, d, generator=g, device="cuda"))
    w = 1 + torch.randn(d, generator=g, device="cuda") * 0.1
    u = torch.full((R, d), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_block_norm_fwd(moe.block_norm(R, d, eps=1e-6), x, w_pre=w, u=u)
    v = ends(x).double()
    ref = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * w.double()
    tol = (2.0 ** -8 + 24 * 2.0 ** -24) * ref.abs() + 2.0 ** -133
    assert ((ends(u).double() - ref).abs() <= tol).all()
    assert (u[1000:-1000].amax(0) == u[1000]).all() and (u[1000:-1000].amin(0) == u[1000]).all()


def test_scored_routing():
    """One expert: its weight is the scale, and its gradient 0 but for d_scores."""
    s, g = moe.shape(R, 8, 1, 1), moe.gating(moe.SCORE_SIGMOID, scale=1.5)
    z = torch.zeros(R, 1, device="cuda")
    z[:3, 0], z[-3:, 0] = torch.tensor([1.0, 2, 3]), torch.tensor([-1.0, -2, -3])
    idx = torch.full((R, 1), 7, dtype=torch.int32, device="cuda")
    w = torch.full((R, 1), 7.0, device="cuda")
    moe.moe_route_select(s, g, z, idx, w)
    assert (idx == 0).all() and (w == 1.5).all()
    dz = torch.full((R, 1), 7.0, device="cuda")
    moe.moe_route_select_bwd(s, g, z, idx, w, dz, d_scores=w)
    v = torch.cat([z[:3], z[-3:]]).double()
    ref = 1.5 * torch.sigmoid(v) * torch.sigmoid(-v)
    got = torch.cat([dz[:3], dz[-3:]]).double()
    assert ((got - ref).abs() <= 128 * 2.0 ** -24 * (ref + 3)).all()
    assert ((dz[3:-3] - 0.375).abs() <= 1e-5).all()
