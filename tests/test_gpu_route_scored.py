"""Scored routing on the GPU against the definition in 64 bits: the selection
exactly, the scores to one rounding, the weights and gradients to bounds that
count fp32 roundings (u = 2^-24 each)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_mixture_experts_15_b200 as moe

U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _clean_status():
    moe.moe_reset_device_status()
    yield
    assert moe.moe_device_status() == 0


def exact_scores(z, sigmoid):
    z = z.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            return 1 / (1 + np.exp(-z))
        m = z.max(1, keepdims=True)
        e = np.where(z == -np.inf, 0.0, np.exp(z - np.where(np.isinf(m) & (m < 0), 0, m)))
        S = e.sum(1, keepdims=True)
        return np.divide(e, S, out=np.where(np.isnan(S), np.nan, np.zeros_like(e)), where=S != 0)


def order(v):
    """Rows' indices by descending value, NaN last, ties to the lower index."""
    return np.lexsort((np.broadcast_to(np.arange(v.shape[-1]), v.shape), -np.where(
        np.isnan(v), 0, v), np.isnan(v)), axis=-1)


def select(z, bias, k, sigmoid, G=1, top_group=1, group_top=1, renorm=True, scale=1.0):
    s = exact_scores(z, sigmoid)
    s32 = s.astype(np.float32)
    c = s32 if bias is None else s32 + bias
    T, N = c.shape
    keep = np.ones((T, N), bool)
    if G > 1:
        per = c.reshape(T, G, N // G)
        best = np.take_along_axis(per, order(per), 2)[:, :, :group_top]
        gs = best[:, :, 0] if group_top == 1 else best[:, :, 0] + best[:, :, 1]
        kept = order(gs)[:, :top_group]
        keep = np.zeros((T, G), bool)
        np.put_along_axis(keep, kept, True, 1)
        keep = np.repeat(keep, N // G, 1)
    # kept experts first, then the order of c among them
    idx = np.lexsort((np.broadcast_to(np.arange(N), c.shape), -np.where(np.isnan(c), 0, c),
                      np.isnan(c), ~keep), axis=-1)[:, :k]
    a = np.take_along_axis(s32.astype(np.float64), idx, 1)  # of the scores as rounded
    if renorm:
        S = a.sum(1, keepdims=True)
        with np.errstate(invalid="ignore"):
            a = np.where(S == 0, 0.0, a / np.where(S == 0, 1, S))
    return s, idx, a * scale


def run(z, bias, k, sigmoid, G=1, top_group=1, group_top=1, renorm=True, scale=1.0, scores=True):
    T, N = z.shape
    zt = torch.from_numpy(z).cuda()
    bt = None if bias is None else torch.from_numpy(bias).cuda()
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    sc = torch.full((T, N), float("nan"), device="cuda") if scores else None
    g = moe.gating(moe.SCORE_SIGMOID if sigmoid else moe.SCORE_SOFTMAX, G, top_group, group_top,
                   scale)
    moe.moe_route_select(moe.shape(T, 8, N, k, renorm=int(renorm)), g, zt, idx, w, bias=bt,
                         scores=sc)
    return idx.cpu().numpy(), w.cpu().numpy(), None if sc is None else sc.cpu().numpy()


def check(z, bias, k, sigmoid, **kw):
    idx, w, sc = run(z, bias, k, sigmoid, **kw)
    s, ref_idx, ref_w = select(z, bias, k, sigmoid, **kw)
    assert np.array_equal(idx, ref_idx)
    # one rounding, where the double value lies within 2^-41 of a midpoint either neighbour
    tiny = 2.0 ** -149
    assert np.all(np.isnan(sc) == np.isnan(s))
    assert np.all((np.abs(sc - s) <= U * (1 + 2.0 ** -16) * s + tiny) | np.isnan(s))
    # a score's rounding, five additions of the sum, the sum's scores, a
    # division and the product by the scale: 9 roundings, and 1 for their products
    assert np.all((np.abs(w - ref_w) <= 10 * U * np.abs(ref_w) + 8 * tiny) | np.isnan(ref_w))
    assert np.all(np.isnan(w) == np.isnan(ref_w))
    idx2, w2, _ = run(z, bias, k, sigmoid, scores=False, **kw)   # without the scores
    assert np.array_equal(idx2, ref_idx)
    assert np.all((np.abs(w2 - ref_w) <= 10 * U * np.abs(ref_w) + 8 * tiny) | np.isnan(ref_w))
    assert np.all(np.isnan(w2) == np.isnan(ref_w))
    return idx, w, sc


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,N,k", [(1, 1, 1), (1, 4, 2), (3, 31, 5), (5, 33, 32), (17, 64, 8),
                                   (2, 65, 6), (7, 127, 4), (9, 128, 32), (33, 250, 6),
                                   (12, 384, 8), (6, 500, 1), (4, 512, 10), (3, 640, 3),
                                   (5, 768, 9), (21, 896, 16), (2, 1021, 31), (8, 1024, 32)])
def test_selection_and_weights(T, N, k, sigmoid):
    rng = np.random.default_rng(T * 1000 + N)
    z = (rng.standard_normal((T, N)) * 2).astype(np.float32)
    b = (rng.standard_normal(N) * 0.2).astype(np.float32)
    check(z, b, k, sigmoid)
    check(z, None, k, sigmoid, renorm=False, scale=2.5)


@pytest.mark.parametrize("N,G,top_group,group_top,k", [
    (64, 8, 4, 2, 8), (256, 8, 4, 2, 8), (256, 8, 1, 2, 32), (160, 8, 3, 1, 6), (90, 3, 2, 2, 7),
    (1024, 32, 5, 2, 16), (1022, 2, 1, 1, 32), (32, 32, 9, 1, 9), (35, 7, 7, 2, 3), (24, 12, 4, 2, 8)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_groups(N, G, top_group, group_top, k, sigmoid):
    rng = np.random.default_rng(N + G)
    z = (rng.standard_normal((67, N)) * 2).astype(np.float32)
    b = (rng.standard_normal(N) * 0.3).astype(np.float32)
    kw = dict(G=G, top_group=top_group, group_top=group_top)
    idx, _, _ = check(z, b, k, sigmoid, **kw)
    assert max(len(set(r // (N // G))) for r in idx) <= top_group
    check(z, None, k, sigmoid, scale=0.5, **kw)


def test_many_tokens_select_exactly():
    """Enough tokens that scores one rounding apart meet at the border."""
    rng = np.random.default_rng(5)
    z = rng.standard_normal((20000, 256)).astype(np.float32)
    b = (rng.standard_normal(256) * 0.05).astype(np.float32)
    check(z, b, 8, True, G=8, top_group=4, group_top=2)
    check(z[:6000], b, 8, False)


def test_values_a_rounding_apart_are_ordered():
    """Rows whose scores differ in their last bits, group scores among them, so
    that every decision hangs on them."""
    rng = np.random.default_rng(9)
    z = (0.7 + rng.integers(-40, 40, (3000, 128)) * 2.0 ** -23).astype(np.float32)
    z[1000:2000] = (-3.0 + rng.integers(-9, 9, (1000, 128)) * 2.0 ** -21).astype(np.float32)
    z[2000:, ::2] = rng.standard_normal((1000, 64)).astype(np.float32)
    check(z, None, 8, True)
    check(z, None, 8, True, G=8, top_group=3, group_top=2)
    b = (rng.integers(-8, 8, 128) * 2.0 ** -24).astype(np.float32)
    check(z, b, 5, True, G=16, top_group=4, group_top=1)


def test_ties_go_to_the_lower_expert():
    z = np.zeros((3, 96), np.float32)
    z[1, 40:44] = 1.0
    z[2] = 40.0  # sigmoid 1 in fp32 for different logits
    z[2, ::2] = 30.0
    for sigmoid in (False, True):
        idx, _, _ = check(z, None, 6, sigmoid)
        assert list(idx[0]) == [0, 1, 2, 3, 4, 5]
        assert list(idx[1]) == [40, 41, 42, 43, 0, 1]
    assert list(run(z, None, 6, True)[0][2]) == [0, 1, 2, 3, 4, 5]
    idx, _, _ = check(z, None, 6, True, G=4, top_group=2, group_top=2)
    assert list(idx[0]) == [0, 1, 2, 3, 4, 5] and list(idx[1][:4]) == [40, 41, 42, 43]


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("G,top_group", [(1, 1), (4, 2)])
def test_masked_and_non_finite_logits(sigmoid, G, top_group):
    """Masked experts (-infinity, the type's lowest value), rows that leave
    nothing, infinities, NaN, and biases of -infinity: indices stay distinct
    and in range, and everything follows the definition."""
    rng = np.random.default_rng(1)
    N, k = 40, 6
    z = rng.standard_normal((12, N)).astype(np.float32)
    z[0, 3:] = -np.inf                     # fewer experts left than k
    z[1] = -np.inf                         # none left
    z[2] = np.finfo(np.float32).min
    z[3, ::3] = np.finfo(np.float32).min
    z[4, 5] = np.nan
    z[5] = np.nan
    z[6, 2] = np.inf
    z[7, :20] = 200.0
    z[8] = -200.0
    z[9, 1] = 1e38
    b = (rng.standard_normal(N) * 0.1).astype(np.float32)
    kw = dict(G=G, top_group=top_group, group_top=2 if G > 1 else 1)
    for bias in (None, b):
        if not sigmoid:  # softmax of a row with NaN or +infinity is NaN
            zz, rest = z[[4, 5, 6]], np.delete(z, [4, 5, 6], 0)
            idx, w, sc = run(zz, bias, k, False, **kw)
            assert np.isnan(sc).all() and np.isnan(w).all()
            assert all(len(set(r)) == k and r.min() >= 0 and r.max() < N for r in idx)
            check(rest, bias, k, False, **kw)
        else:
            check(z, bias, k, True, **kw)
    b[4::5] = -np.inf
    idx, _, _ = check(z[7:], b, k, sigmoid, **kw)
    assert all(len(set(r)) == k for r in idx)


def test_scores_in_place_of_the_logits():
    rng = np.random.default_rng(3)
    z = rng.standard_normal((50, 200)).astype(np.float32)
    zt = torch.from_numpy(z).cuda()
    idx = torch.empty(50, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(50, 4, device="cuda")
    moe.moe_route_select(moe.shape(50, 8, 200, 4), moe.gating(moe.SCORE_SIGMOID), zt, idx, w,
                         scores=zt)
    ref_idx, ref_w, ref_s = run(z, None, 4, True)
    assert np.array_equal(zt.cpu().numpy(), ref_s) and np.array_equal(idx.cpu().numpy(), ref_idx)
    assert np.array_equal(w.cpu().numpy(), ref_w)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("T,d,N,k", [(1, 64, 8, 2), (37, 264, 160, 6)])
def test_route_scored_is_the_routers_logits_and_the_selection(T, d, N, k, dtype):
    torch.manual_seed(T)
    u = torch.randn(T, d, device="cuda").to(getattr(torch, dtype))
    wr = torch.randn(N, d, device="cuda") * 0.1
    b = torch.randn(N, device="cuda") * 0.1
    s, g = moe.shape(T, d, N, k), moe.gating(moe.SCORE_SIGMOID, 4 if N > 8 else 1, 2 if N > 8 else 1,
                                             2 if N > 8 else 1, 1.5)
    z0 = torch.empty(T, N, device="cuda")
    i0, w0 = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_route(s, u, wr, i0, w0, logits=z0)  # the softmax router, for its logits
    outs = []
    for keep in (True, False):
        z = torch.empty(T, N, device="cuda") if keep else None
        i, w = torch.empty_like(i0), torch.empty_like(w0)
        moe.moe_route_scored(s, g, u, wr, i, w, bias=b, logits=z)
        if keep:
            assert torch.equal(z, z0)
        outs.append((i, w))
    i, w = torch.empty_like(i0), torch.empty_like(w0)
    moe.moe_route_select(s, g, z0, i, w, bias=b)
    for a, c in outs:
        assert torch.equal(a, i) and torch.equal(c, w)


def test_softmax_top_k_is_the_softmax_router():
    """Without bias and groups the selection is moe_route's."""
    torch.manual_seed(0)
    s = moe.shape(64, 128, 32, 4)
    u, wr = torch.randn(64, 128, device="cuda"), torch.randn(32, 128, device="cuda") * 0.1
    i0, w0 = torch.empty(64, 4, dtype=torch.int32, device="cuda"), torch.empty(64, 4, device="cuda")
    i1, w1 = torch.empty_like(i0), torch.empty_like(w0)
    moe.moe_route(s, u, wr, i0, w0)
    moe.moe_route_scored(s, moe.gating(), u, wr, i1, w1)
    assert torch.equal(i0, i1)
    assert torch.allclose(w0, w1, rtol=2e-6, atol=0)


# ------------------------------------------------------------------ gradient
def grad_ref(z, idx, da, ds, sigmoid, renorm, scale):
    """dz in 64 bits from the formula, and the size of the terms it adds."""
    z = z.astype(np.float64)
    s = exact_scores(z, sigmoid)
    T, k = idx.shape
    row = np.arange(T)[:, None]
    si = np.take_along_axis(s, idx, 1)
    g = np.zeros_like(s) if ds is None else ds.astype(np.float64).copy()
    m = np.abs(g)
    da = da.astype(np.float64) * scale
    if renorm:
        S = si.sum(1, keepdims=True)
        S1 = np.where(S == 0, 1, S)
        add = np.where(S == 0, 0, (da - (da * si).sum(1, keepdims=True) / S1) / S1)
        mag = np.where(S == 0, 0, (np.abs(da) + (np.abs(da) * si).sum(1, keepdims=True) / S1) / S1)
    else:
        add, mag = da, np.abs(da)
    np.add.at(g, (row, idx), add)
    np.add.at(m, (row, idx), mag)
    if sigmoid:
        f = s * (1 / (1 + np.exp(z)))
        return g * f, m * f
    return (s * (g - (g * s).sum(1, keepdims=True)), s * (m + (m * s).sum(1, keepdims=True)))


def run_bwd(z, idx, da, ds, sigmoid, renorm, scale, in_place=False):
    T, N = z.shape
    c = lambda v: None if v is None else torch.from_numpy(v).cuda()  # noqa: E731
    d = c(ds)
    dz = d if in_place else torch.full((T, N), float("nan"), device="cuda")
    g = moe.gating(moe.SCORE_SIGMOID if sigmoid else moe.SCORE_SOFTMAX, scale=scale)
    moe.moe_route_select_bwd(moe.shape(T, 8, N, idx.shape[1], renorm=int(renorm)), g, c(z),
                             c(idx.astype(np.int32)), c(da), dz, d_scores=d)
    return dz.cpu().numpy()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm,dense", [(True, False), (True, True), (False, True)])
@pytest.mark.parametrize("T,N,k", [(1, 1, 1), (3, 31, 5), (17, 64, 8), (33, 250, 6), (5, 384, 32),
                                   (21, 896, 16), (2, 1021, 31)])
def test_gradient_formula(T, N, k, renorm, dense, sigmoid):
    """Each dz to 128 u of the terms it adds: the exponential of a rounded
    difference (|z - max| below 20 here: 24 u), a sum of at most 32 + 5, its
    reciprocal, the slots' sums (10) and the products (10)."""
    rng = np.random.default_rng(N + k)
    z = (rng.standard_normal((T, N)) * 2).astype(np.float32)
    idx = np.argsort(-z, 1)[:, :k]
    da = rng.standard_normal((T, k)).astype(np.float32)
    ds = rng.standard_normal((T, N)).astype(np.float32) if dense else None
    ref, mag = grad_ref(z, idx, da, ds, sigmoid, renorm, 2.5)
    got = run_bwd(z, idx, da, ds, sigmoid, renorm, 2.5)
    assert np.all(np.abs(got - ref) <= 128 * U * mag + 2.0 ** -140)
    if dense:
        assert np.array_equal(got, run_bwd(z, idx, da, ds, sigmoid, renorm, 2.5, in_place=True))


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(sigmoid, renorm):
    """Along a random direction, against central differences of the forward in
    64 bits (step 1e-5: their own error is below 1e-8 of the terms)."""
    rng = np.random.default_rng(8)
    T, N, k = 9, 100, 7
    z = rng.standard_normal((T, N)).astype(np.float32)
    idx = np.argsort(-z, 1)[:, :k]
    da, ds = (rng.standard_normal(s).astype(np.float32) for s in ((T, k), (T, N)))
    v = rng.standard_normal((T, N))

    def L(h):
        s = exact_scores(z + h * v, sigmoid)
        a = np.take_along_axis(s, idx, 1)
        a = a / a.sum(1, keepdims=True) if renorm else a
        return 1.5 * (a * da).sum() + (s * ds).sum()

    quotient = (L(1e-5) - L(-1e-5)) / 2e-5
    got = run_bwd(z, idx, da, ds, sigmoid, renorm, 1.5).astype(np.float64)
    _, mag = grad_ref(z, idx, da, ds, sigmoid, renorm, 1.5)
    assert abs((got * v).sum() - quotient) <= (128 * U + 1e-7) * (mag * np.abs(v)).sum()


def test_gradient_of_repeated_and_masked_experts():
    rng = np.random.default_rng(2)
    z = rng.standard_normal((6, 20)).astype(np.float32)
    idx = np.array([[1, 1, 1], [0, 5, 0], [3, 4, 5], [2, 1, 0], [19, 18, 17], [7, 7, 8]])
    z[2, 3:6] = -np.inf          # every selected score is 0
    z[3, 5:] = -np.inf
    da = rng.standard_normal((6, 3)).astype(np.float32)
    for sigmoid in (False, True):
        for renorm in (True, False):
            with np.errstate(over="ignore"):
                ref, mag = grad_ref(z, idx, da, None, sigmoid, renorm, 1.0)
            got = run_bwd(z, idx, da, None, sigmoid, renorm, 1.0)
            assert np.isfinite(got).all()
            assert np.all(np.abs(got - ref) <= 128 * U * mag + 2.0 ** -140)
    z[:] = -np.inf
    for sigmoid in (False, True):
        assert np.all(run_bwd(z, idx, da, None, sigmoid, True, 1.0) == 0)


def renorm_grad64(z, idx, da, ds, sigmoid, scale):
    """dz in 64 bits with the weights from logits relative to the largest selected
    one, so that no score underflows, and the size of the terms it adds."""
    z = z.astype(np.float64)
    row, zs = np.arange(len(z))[:, None], np.take_along_axis(z, idx, 1)
    m = zs.max(1, keepdims=True)
    top = np.minimum(m, 0) if sigmoid else m
    with np.errstate(over="ignore"):
        w = np.exp(zs - top) / (1 + np.exp(zs)) if sigmoid else np.exp(zs - top)
        w = w / w.sum(1, keepdims=True)
        s = exact_scores(z, sigmoid)
        f = 1 / (1 + np.exp(z)) if sigmoid else np.ones_like(z)
    da = da.astype(np.float64) * scale
    wda, wma = (w * da).sum(1, keepdims=True), (w * np.abs(da)).sum(1, keepdims=True)
    fs = np.take_along_axis(f, idx, 1)
    g = np.zeros_like(z) if ds is None else ds.astype(np.float64)
    dot, dotm = ((0.0, 0.0) if sigmoid else
                 ((g * s).sum(1, keepdims=True), (np.abs(g) * s).sum(1, keepdims=True)))
    # softmax: the terms w_i (da_i - sum da w) of sum g s, at most 2 sum |da| w in
    # all, add up to 0 but each is rounded, and every dz_j takes s_j of their sum
    slots = 0.0 if sigmoid else 2 * wma
    dz, mag = s * f * (g - dot), s * f * (np.abs(g) + dotm + slots)
    np.add.at(dz, (row, idx), w * fs * (da - wda))
    np.add.at(mag, (row, idx), w * fs * (np.abs(da) + wma))
    return dz, mag


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dense", [False, True])
def test_gradient_of_tiny_selected_scores(sigmoid, dense):
    """Selected experts whose scores are near fp32's smallest values or between
    them (a bias or the groups chose them): the renormalised weights stay of
    order 1, and so does their gradient.  Bounds: the exponential of a rounded
    difference (|z_i - max| below 20 among the selected: 24 u), 10 roundings of
    the sums, 10 of the products and the reciprocal, twice; the dense part as
    elsewhere, with 2^-140 for its subnormal scores."""
    rng = np.random.default_rng(12)
    T, N, k = 19, 70, 6
    base = np.linspace(-103.5, -20.0, T)[:, None]      # the largest of a row's selected
    z = rng.standard_normal((T, N)).astype(np.float32)
    z[:, 0] = 2.0
    idx = np.stack([1 + rng.permutation(N - 1)[:k] for _ in range(T)])
    drop = rng.uniform(0, 17, (T, k))
    drop[:, 3] = 0
    low = (base - drop) + (0 if sigmoid else np.log(np.exp(z.astype(np.float64)).sum(1,
                                                                               keepdims=True)))
    np.put_along_axis(z, idx, low.astype(np.float32), 1)
    da = rng.standard_normal((T, k)).astype(np.float32)
    ds = rng.standard_normal((T, N)).astype(np.float32) if dense else None
    ref, mag = renorm_grad64(z, idx, da, ds, sigmoid, 2.5)
    got = run_bwd(z, idx, da, ds, sigmoid, True, 2.5)
    assert np.median(np.abs(ref).max(1)) > 0.1
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - ref) <= 128 * U * mag + 2.0 ** -140)
    if dense:
        assert np.array_equal(got, run_bwd(z, idx, da, ds, sigmoid, True, 2.5, in_place=True))
    # the same index twice, and one that is no expert's beside them
    idx[:, 4] = idx[:, 3]
    ref, mag = renorm_grad64(z, idx, da, ds, sigmoid, 2.5)
    got = run_bwd(z, idx, da, ds, sigmoid, True, 2.5)
    assert np.all(np.abs(got - ref) <= 128 * U * mag + 2.0 ** -140)
    bad = np.concatenate([idx, np.full((T, 1), N)], 1)
    got2 = run_bwd(z, bad, np.concatenate([da, np.ones((T, 1), np.float32)], 1), ds, sigmoid, True,
                   2.5)
    assert moe.moe_device_status() == -5
    moe.moe_reset_device_status()
    assert np.all(np.abs(got2 - ref) <= 128 * U * mag + 2.0 ** -140)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_gradient_ends_where_the_forwards_weights_do(sigmoid):
    """The weights are 0, and have no gradient, exactly where every selected
    score rounds to 0 in fp32 (150 ln 2 = 103.97208 below the sigmoid's 0)."""
    edge = np.float32(-150 * np.log(2.0))
    steps = np.arange(-4, 5) * np.spacing(np.abs(edge))
    z = np.full((len(steps), 40), 1.0, np.float32)
    lift = 0.0 if sigmoid else 1 + np.log(37.0)
    z[:, 5:8] = (edge + lift + steps.astype(np.float32)[:, None]).astype(np.float32)
    if not sigmoid:   # clear of the edge: the logarithm of the sum is rounded, too
        z[:, 5:8] += np.where(steps < 0, -1e-3, 1e-3).astype(np.float32)[:, None]
    idx = np.tile(np.array([5, 6, 7]), (len(z), 1))
    da = np.tile(np.array([1.0, 2.0, 4.0], np.float32), (len(z), 1))
    b = np.zeros(40, np.float32)
    b[5:8] = 2.0
    _, w, _ = run(z, b, 3, sigmoid)
    got = run_bwd(z, idx, da, None, sigmoid, True, 1.0)
    alive = (w != 0).any(1)
    assert alive.any() and not alive.all()
    assert np.array_equal(alive, (np.abs(got[:, 5:8]).max(1) > 0.1))
    assert np.all(got[~alive] == 0)


def test_gradient_refuses_bad_indices():
    """An index out of range is recorded and its slot counts as absent."""
    rng = np.random.default_rng(4)
    z = rng.standard_normal((2, 10)).astype(np.float32)
    da = np.ones((2, 2), np.float32)
    got = run_bwd(z, np.array([[3, 10], [-1, 4]]), da, None, True, False, 1.0)
    assert moe.moe_device_status() == -5
    moe.moe_reset_device_status()
    ref, _ = grad_ref(z, np.array([[3], [4]]), da[:, :1], None, True, False, 1.0)
    assert np.allclose(got, ref, rtol=1e-5, atol=0)


def test_empty_batch_stream_and_graph():
    s, g = moe.shape(0, 8, 16, 2), moe.gating()
    e = torch.empty(0, device="cuda")
    moe.moe_route_select(s, g, e, torch.empty(0, dtype=torch.int32, device="cuda"), e)
    T, N, k = 300, 256, 8
    s, g = moe.shape(T, 8, N, k), moe.gating(moe.SCORE_SIGMOID, 8, 4, 2)
    z = torch.randn(T, N, device="cuda")
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    dz = torch.empty(T, N, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        moe.moe_route_select(s, g, z, idx, w)
        moe.moe_route_select_bwd(s, g, z, idx, w, dz)
    torch.cuda.current_stream().wait_stream(st)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        moe.moe_route_select(s, g, z, idx, w)
        moe.moe_route_select_bwd(s, g, z, idx, w, dz)
    z.copy_(torch.randn(T, N, device="cuda"))
    gr.replay()
    i2, w2, d2 = torch.empty_like(idx), torch.empty_like(w), torch.empty_like(dz)
    moe.moe_route_select(s, g, z, i2, w2)
    moe.moe_route_select_bwd(s, g, z, i2, w2, d2)
    assert torch.equal(idx, i2) and torch.equal(w, w2) and torch.equal(dz, d2)
