"""8-bit integer products on the GPU: codes, scales and integer sums exactly,
the scaled values to their roundings (u = 2^-24)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_mixture_experts_15_b200 as moe

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(autouse=True)
def _clean_status():
    moe.moe_reset_device_status()
    yield
    assert moe.moe_device_status() == 0


def quant_ref(x):
    """The definition in fp32 operations on the host."""
    x = x.astype(np.float32)
    amax = np.abs(x).max(1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        s = np.where(amax == 0, np.float32(1), amax * np.float32(1 / 127)).astype(np.float32)
        q = np.clip(np.rint(x / s), -127, 127)
    return np.nan_to_num(q).astype(np.int8), s[:, 0]


def quant(x):
    codes = torch.full(x.shape, 99, dtype=torch.int8, device="cuda")
    scales = torch.full((x.shape[0],), float("nan"), device="cuda")
    moe.moe_quantize_i8_rows(x, codes, scales)
    return codes, scales


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (67, 1040), (5, 4096), (700, 512),
                                       (2, 14336), (3, 40000)])
def test_quantize_rows_exactly(rows, cols, dtype):
    rng = np.random.default_rng(rows + cols)
    x = rng.standard_normal((rows, cols)) * 10.0 ** rng.uniform(-3, 3, (rows, 1))
    if rows > 2:
        x[1] = 0.0
        x[2, 5] = 3e4
        # halves of a step: ties go to the even code (a scale of exactly 1)
        x[0] = (np.arange(cols) % 253 - 126) + 0.5
        x[0, 0] = 127.0
    t = torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).cuda()
    codes, scales = quant(t)
    q, s = quant_ref(t.float().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), s.view(np.uint32))
    assert np.array_equal(codes.cpu().numpy(), q)


def test_quantize_many_rows_exactly():
    """Enough elements that hundreds lie within 2^-14 of a tie between two
    codes, where the product by the reciprocal cannot decide."""
    x = torch.randn(6000, 1040, generator=torch.Generator(device="cuda").manual_seed(1),
                    device="cuda")
    codes, scales = quant(x)
    amax = x.abs().amax(1)
    s = amax * torch.full_like(amax, float(np.float32(1 / 127)))
    assert torch.equal(scales, s)
    assert torch.equal(codes.float(), torch.round(x / s[:, None]))


def test_quantize_keeps_infinities_and_nan_in_the_scale():
    x = torch.randn(4, 64, device="cuda")
    x[1, 3] = float("inf")
    x[2, 60] = float("nan")
    x[3, 0], x[3, 1] = float("nan"), float("-inf")
    codes, scales = quant(x)
    assert scales[0].isfinite() and scales[1].isinf() and scales[2].isnan() and scales[3].isnan()
    w = torch.ones(8, 64, dtype=torch.int8, device="cuda")
    y = torch.empty(4, 8, device="cuda")
    moe.moe_grouped_gemm_i8(codes, scales, w, torch.ones(8, device="cuda"), y)
    assert y[0].isfinite().all() and y[1:].isnan().all()


def case(counts, K, n, seed, extra=0, lowest=False):
    """Codes and scales for groups of `counts` rows, `extra` rows behind them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    R, G = int(sum(counts)) + extra, len(counts)
    c = lambda *s: torch.randint(-128, 128, s, generator=g, device="cuda",  # noqa: E731
                                 dtype=torch.int8)
    x, w = c(R, K), c(G, n, K)
    if lowest:
        x.fill_(-128)
        w.fill_(-128)
    xs = torch.rand(R, generator=g, device="cuda") + 0.5
    ws = torch.rand(G, n, generator=g, device="cuda") * 1e-3 + 1e-4
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    return x, xs, w, ws, off


def product(counts, x, xs, w, ws):
    """The product in 64 bits (each integer sum exactly)."""
    y, at = [], 0
    for e, c in enumerate(counts):
        v = x[at:at + c].double() @ w[e].double().T
        y.append(v * xs[at:at + c].double()[:, None] * ws[e].double())
        at += c
    return torch.cat(y)


def check(counts, K, n, dtype="f32", seed=0, extra=0, lowest=False):
    x, xs, w, ws, off = case(counts, K, n, seed, extra, lowest)
    R = int(sum(counts))
    y = torch.full((R + extra, n), 7.0, dtype=DT[dtype], device="cuda")
    moe.moe_grouped_gemm_i8(x, xs, w, ws, y, offsets=off)
    ref = product(counts, x, xs, w, ws)
    # the sum to fp32 and two products: 3 u (and u for their own product), then
    # the output's rounding
    f = torch.finfo(DT[dtype])
    rel, ab = (4 * U, 0) if dtype == "f32" else (4 * U + f.eps / 2, f.smallest_normal * f.eps / 2)
    assert ((y[:R].double() - ref).abs() <= rel * ref.abs() + ab).all()
    assert (y[R:] == 7.0).all()   # rows behind the last group stay as they were


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("counts", [[1], [2], [7], [16], [33], [130], [300], [0, 1, 0, 5, 0],
                                    [37, 0, 130, 5], [256, 1, 129, 64, 0, 17, 300]])
def test_grouped_product(counts, dtype):
    for i, (K, n) in enumerate(((16, 1), (48, 5), (128, 128), (144, 130), (1040, 257), (512, 640))):
        check(counts, K, n, dtype, seed=i, extra=i % 2 * 9)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("counts,K,n", [([1000, 700, 0, 901], 640, 2570), ([150, 161, 33, 200], 656, 5003),
                                        ([900, 301], 512, 2001), ([2500], 2064, 1000)])
def test_many_tiles(counts, K, n, dtype):
    """Several rounds of tiles over the SMs: on pairs of CTAs, of either width, and
    on single ones."""
    check(counts, K, n, dtype, seed=K)


@pytest.mark.parametrize("rows", [1, 3, 8, 17, 32, 60])
@pytest.mark.parametrize("K,n", [(4096, 4096), (4112, 1000), (14336, 264), (256, 14336), (64, 3)])
def test_few_rows(rows, K, n):
    check([rows], K, n, "bf16", seed=rows)
    x, xs, w, ws, _ = case([rows], K, n, 1)
    y = torch.empty(rows, n, device="cuda")
    moe.moe_grouped_gemm_i8(x, xs, w[0], ws, y)     # one group without offsets
    ref = product([rows], x, xs, w, ws)
    assert ((y.double() - ref).abs() <= 4 * U * ref.abs()).all()


def test_many_groups_with_few_rows():
    rng = np.random.default_rng(0)
    check(rng.integers(0, 4, 64).tolist(), 512, 1032, "f32", extra=3)
    check(rng.integers(0, 60, 64).tolist(), 1040, 264, "bf16")
    check(rng.integers(0, 2, 1024).tolist(), 64, 40, "f16")
    check([0] * 7 + [1], 256, 48, "f32")
    check([0] * 8, 256, 48, "f32", extra=5)


def test_large_product():
    rng = np.random.default_rng(1)
    check(rng.multinomial(4000, [1 / 8] * 8).tolist(), 2048, 3000, "bf16")


@pytest.mark.parametrize("rows", [2, 40])
def test_sums_fill_32_bits(rows):
    """The longest rows of the lowest codes: 131056 * 2^14 just fits s32."""
    check([rows], 131056, 8, "f32", lowest=True)


def test_bad_offsets_are_recorded_and_skipped():
    x, xs, w, ws, off = case([5, 6, 7], 64, 40, 0)
    y = torch.full((18, 40), 7.0, device="cuda")
    bad = off.clone()
    bad[1], bad[2] = 30, 11           # group 0 passes the rows, group 1 runs backwards
    moe.moe_grouped_gemm_i8(x, xs, w, ws, y, offsets=bad)
    assert moe.moe_device_status() == -5
    moe.moe_reset_device_status()
    ref = product([5, 6, 7], x, xs, w, ws)
    assert (y[:11] == 7.0).all()
    assert ((y[11:].double() - ref[11:]).abs() <= 4 * U * ref[11:].abs()).all()


def test_stream_and_graph():
    x, xs, w, ws, off = case([50, 0, 3], 512, 264, 3)
    for rows in (53, 3):
        o = off if rows == 53 else torch.tensor([0, 1, 1, 3], dtype=torch.int32, device="cuda")
        y = torch.empty(rows, 264, device="cuda")
        moe.moe_grouped_gemm_i8(x[:rows], xs[:rows], w, ws, y, offsets=o)
        st, z = torch.cuda.Stream(), torch.empty_like(y)
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            moe.moe_grouped_gemm_i8(x[:rows], xs[:rows], w, ws, z, offsets=o)
        st.synchronize()
        assert torch.equal(y, z)
        gr, z = torch.cuda.CUDAGraph(), torch.empty_like(y)
        with torch.cuda.graph(gr):
            moe.moe_grouped_gemm_i8(x[:rows], xs[:rows], w, ws, z, offsets=o)
        for _ in range(2):
            z.zero_()
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, z)


# ------------------------------------------------------------------- experts
@pytest.mark.parametrize("situ", [False, True])
@pytest.mark.parametrize("width,h,counts", [(128, 128, [37, 0, 130, 5]), (256, 384, [1, 0, 2, 1]),
                                            (512, 256, [300, 1, 64, 129])])
def test_expert_ffn(width, h, counts, situ):
    """Against the same steps in 64 bits with H rounded to bf16 and quantised.

    The pre-activations are exact sums, so H differs from the reference's by
    the activation's error: 2^-20 (SwiGLU) or 2^-10 (the capped one's tanh).
    Its share over a bf16 step of 2^-8 of the values round to the neighbour
    (2^-11, or a quarter), each then off by 2^-8 and by at most one code of the
    row (one in some 30 of a typical code): 1e-3 of the result in the 2-norm,
    and 1.7e-2 for the capped one."""
    N, R = len(counts), int(sum(counts))
    g = torch.Generator(device="cuda").manual_seed(width + h)
    x = torch.randn(R + 3, width, generator=g, device="cuda")
    mats = {}
    for k, (a, b) in dict(gate=(N * h, width), up=(N * h, width), down=(N * width, h)).items():
        mats[k] = quant(torch.randn(a, b, generator=g, device="cuda") * b ** -0.5)
    xc, xs = quant(x)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    s = moe.shape(R + 3, width, N, 1, h)
    act = moe.act(moe.ACT_SITU_GLU, 4.0, 25.0) if situ else moe.act()
    y = torch.full((R + 3, width), 7.0, device="cuda")
    moe.moe_expert_ffn_i8(s, width, xc, xs, off, mats["gate"][0], mats["up"][0], mats["down"][0],
                          mats["gate"][1], mats["up"][1], mats["down"][1], y, a=act)
    assert (y[R:] == 7.0).all()
    val = {k: c.double() * sc.double()[:, None] for k, (c, sc) in mats.items()}
    xv, ref, at = xc.double() * xs.double()[:, None], [], 0
    for e, c in enumerate(counts):
        r = xv[at:at + c]
        a, b = (r @ val[k][e * h:(e + 1) * h].T for k in ("gate", "up"))
        if situ:
            a, b = 4 * torch.tanh(a / 4), 25 * torch.tanh(b / 25)
        H = (a * torch.sigmoid(a) * b).to(torch.bfloat16).float()
        q, sc = quant_ref(H.cpu().numpy()) if c else (np.zeros((0, h), np.int8), np.zeros(0, "f4"))
        Hv = torch.from_numpy(q).cuda().double() * torch.from_numpy(sc).cuda().double()[:, None]
        ref.append(Hv @ val["down"][e * width:(e + 1) * width].T)
        at += c
    ref = torch.cat(ref)
    off_by = float((y[:R].double() - ref).norm() / ref.norm())
    assert off_by <= (1.7e-2 if situ else 1e-3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_tiny_rows_exactly(dtype):
    """Rows whose scale is subnormal, or rounds to 0, where the product by its
    reciprocal cannot be used: the definition's codes, held within 127."""
    top = [1e-35, 2e-36, 1.495e-36, 1.49e-36, 1e-36, 1e-37, 1e-39, 1e-40, 5e-42, 3e-43, 2e-44, 1e-44,
           3e-45, 1.5e-45]
    rng = np.random.default_rng(6)
    x = rng.uniform(-1, 1, (len(top), 96))
    x[:, 7] = -1.0
    x = (x * np.array(top)[:, None]).astype(np.float32)
    x[:, 9], x[:, 10] = 0.0, -0.0
    t = torch.from_numpy(x).to(DT[dtype]).cuda()
    codes, scales = quant(t)
    q, s = quant_ref(t.float().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), s.view(np.uint32))
    assert np.array_equal(codes.cpu().numpy(), q)
    if dtype == "f32":
        assert (s == 0).any() and ((0 < s) & (s < 2.0 ** -126)).any() and (np.abs(q) == 127).any()


def test_quantize_codes_of_rows_that_are_not_finite():
    """A row with an infinity or a NaN has nothing but zero codes: its scale holds it."""
    x = torch.randn(3, 64, device="cuda")
    x[0, 3] = float("inf")
    x[1, 60] = float("nan")
    x[2, 0], x[2, 1], x[2, 2] = float("nan"), float("-inf"), float("inf")
    for dt in DT.values():
        codes, _ = quant(x.to(dt))
        assert (codes == 0).all()
