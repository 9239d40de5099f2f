"""Block norms on the GPU against their formulas in 64 bits.  A value of a type
with unit roundoff eps/2 is held to eps/2 of itself plus fp32 roundings
(u = 2^-24) of the terms it is made of."""
import itertools

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_mixture_experts_15_b200 as moe

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


@pytest.fixture(autouse=True)
def _clean_status():
    moe.moe_reset_device_status()
    yield
    assert moe.moe_device_status() == 0


def half_step(dt):
    """Relative and absolute part of one rounding (fp32: counted in u)."""
    if dt == torch.float32:
        return 0.0, 2.0 ** -149
    f = torch.finfo(dt)
    return f.eps / 2, f.smallest_normal * f.eps / 2


def inputs(T, d, dt, gate, post, pre, seed, branch=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, sd=1.0: torch.randn(s, generator=g, device="cuda") * sd  # noqa: E731
    t = {"x": n(T, d, sd=2).to(dt), "y": n(T, d, sd=0.5).to(dt) if branch else None,
         "w_post": 1 + n(d, sd=0.2) if post else None, "w_pre": 1 + n(d, sd=0.2) if pre else None}
    t["gate"] = {"none": None, "channel": n(d), "token": n(T), "full": n(T, d).to(dt)}[gate]
    t["desc"] = moe.block_norm(T, d, {"none": 0, "channel": 1, "token": 2, "full": 3}[gate], 0.9,
                               -0.7, EPS)
    t["kind"] = gate
    return t


def d64(t):
    return None if t is None else t.double()


def gate64(t):
    if t["gate"] is None:
        return torch.ones((), dtype=torch.float64, device="cuda")
    return d64(t["gate"])[:, None] if t["kind"] == "token" else d64(t["gate"])


def rnorm(v):
    return 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def forward(t, x_out=None):
    e = dict(device="cuda", dtype=t["x"].dtype)
    T, d = t["x"].shape
    xo = torch.full((T, d), float("nan"), **e) if x_out is None and t["y"] is not None else x_out
    u = torch.full((T, d), float("nan"), **e) if t["w_pre"] is not None else None
    moe.moe_block_norm_fwd(t["desc"], t["x"], y=t["y"], w_post=t["w_post"], gate=t["gate"],
                           w_pre=t["w_pre"], x_out=xo, u=u)
    return xo, u


def check_forward(t):
    xo, u = forward(t)
    dt, x, y = t["x"].dtype, d64(t["x"]), d64(t["y"])
    rel, ab = half_step(dt)
    if y is not None:
        n = y if t["w_post"] is None else y * rnorm(y) * d64(t["w_post"])
        b = -0.7 * gate64(t) * n
        ref = 0.9 * x + b
        # the norm's factor: a sum of 8 + 5 + 4 + 4 steps halved by the root, the
        # root's 2, the products' 4, the sum's 1 and the constants' own: below 24
        tol = rel * ref.abs() + 24 * U * ((0.9 * x).abs() + b.abs()) + ab
        assert ((xo.double() - ref).abs() <= tol).all()
        x = xo.double()
    if u is not None:
        ref = x * rnorm(x) * d64(t["w_pre"])
        assert ((u.double() - ref).abs() <= rel * ref.abs() + 24 * U * ref.abs() + ab).all()
    return xo, u


SIZES = [(1, 8), (3, 24), (1, 512), (67, 256), (5, 264), (33, 1000), (9, 2056), (150, 4096),
         (3, 4104), (2, 8192), (41, 12296), (1, 16384)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,d", SIZES)
def test_forward(T, d, dtype):
    for i, (gate, (post, pre)) in enumerate(itertools.product(
            ("none", "channel", "token", "full"), ((True, True), (False, True), (True, False),
                                                   (False, False)))):
        check_forward(inputs(T, d, DT[dtype], gate, post, pre, 10 * d + i))


@pytest.mark.parametrize("dtype", list(DT))
def test_pre_norm_alone(dtype):
    for T, d in ((1, 8), (70, 520), (5, 4104)):
        check_forward(inputs(T, d, DT[dtype], "none", False, True, d, branch=False))


@pytest.mark.parametrize("dtype", list(DT))
def test_many_rows(dtype):
    """More rows than the grid holds at once, in teams that do not divide them."""
    check_forward(inputs(5003, 136, DT[dtype], "channel", True, True, 1))
    check_forward(inputs(1203, 4096, DT[dtype], "full", True, True, 2))
    check_forward(inputs(301, 8200, DT[dtype], "token", True, True, 3))


@pytest.mark.parametrize("T,d", [(7, 512), (40, 4096), (3, 5000)])
def test_one_pass_equals_its_two_halves(T, d):
    """Post and next pre norm in one call equal two calls bit for bit, and
    x_out may be x."""
    t = inputs(T, d, torch.bfloat16, "channel", True, True, 7)
    xo, u = forward(t)
    a, _ = forward({**t, "w_pre": None})
    _, b = forward({**t, "x": a, "y": None, "w_post": None, "gate": None, "kind": "none",
                    "desc": moe.block_norm(T, d, eps=EPS)})
    assert torch.equal(xo, a) and torch.equal(u, b)
    x = t["x"].clone()
    forward({**t, "x": x}, x_out=x)
    assert torch.equal(x, xo)


def test_zero_rows_and_non_finite_rows():
    t = inputs(6, 520, torch.bfloat16, "none", True, True, 3)
    t["x"][0] = 0
    t["y"][0] = 0
    t["y"][1] = 0
    t["x"][3, 7] = float("inf")
    t["y"][4, 9] = float("nan")
    xo, u = forward(t)
    assert (xo[0] == 0).all() and (u[0] == 0).all()
    assert torch.isfinite(xo[1]).all() and torch.isfinite(u[[1, 2, 5]]).all()
    assert xo[3, 7].isinf() and xo[3].isfinite().sum() == 519   # its own element only
    assert xo[4].isnan().all() and u[4].isnan().all()           # the norm spreads a NaN
    ok = [0, 1, 2, 5]
    check_forward({**t, "x": t["x"][ok], "y": t["y"][ok], "desc": moe.block_norm(
        4, 520, 0, 0.9, -0.7, EPS)})


# ------------------------------------------------------------------ backward
def backward(t, x_out, dx_out, du, gt, branch=True, in_place=False):
    T, d = t["x"].shape
    nan = lambda *s, dtype=torch.float32: torch.full(s, float("nan"), device="cuda",  # noqa: E731
                                                     dtype=dtype)
    dt = t["x"].dtype
    g = {"dx": dx_out if in_place else nan(T, d, dtype=gt)}
    if branch:
        g["dy"] = nan(T, d, dtype=dt)
    if t["gate"] is not None:
        g["dgate"] = nan(*t["gate"].shape, dtype=t["gate"].dtype)
    if t["w_post"] is not None:
        g["dw_post"] = nan(d)
    if t["w_pre"] is not None:
        g["dw_pre"] = nan(d)
    moe.moe_block_norm_bwd(t["desc"], dx_out, g, x_out=x_out, y=t["y"], w_post=t["w_post"],
                           gate=t["gate"], w_pre=t["w_pre"], du=du)
    return g


def backward64(t, x_out, dx_out, du, branch=True):
    """The gradients in 64 bits and, for each, the size of the terms it adds."""
    xo, y, dxo = d64(x_out), d64(t["y"]), d64(dx_out)
    T, d = t["x"].shape
    dxt = torch.zeros(T, d, dtype=torch.float64, device="cuda") if dxo is None else dxo
    mag, ref = dxt.abs(), {}
    if t["w_pre"] is not None:
        r, w, g = rnorm(xo), d64(t["w_pre"]), d64(du)
        xh, wd = xo * r, w * g
        dxt = dxt + r * (wd - xh * (xh * wd).mean(1, keepdim=True))
        mag = mag + r * (wd.abs() + xh.abs() * (xh * wd).abs().mean(1, keepdim=True))
        ref["dw_pre"] = ((g * xh).sum(0), (g * xh).abs().sum(0))
    if not branch:
        ref["dx"] = (dxt, mag)
        return ref
    ref["dx"] = (0.9 * dxt, 0.9 * mag)
    b, bm, gt = -0.7 * dxt, 0.7 * mag, gate64(t)
    n = yh = y
    dn, dnm = b * gt, bm * gt.abs()
    if t["w_post"] is not None:
        r, w = rnorm(y), d64(t["w_post"])
        yh = y * r
        n = yh * w
        ref["dw_post"] = ((dn * yh).sum(0), (dnm * yh.abs()).sum(0))
        ref["dy"] = (r * (w * dn - yh * (n * dn).mean(1, keepdim=True)),
                     r * ((w * dnm).abs() + yh.abs() * (n.abs() * dnm).mean(1, keepdim=True)))
    else:
        ref["dy"] = (dn.expand(T, d), dnm.expand(T, d))
    if t["gate"] is not None:
        dg, dm = b * n, bm * n.abs()
        ref["dgate"] = ((dg.sum(0), dm.sum(0)) if t["kind"] == "channel" else
                        (dg.sum(1), dm.sum(1)) if t["kind"] == "token" else (dg, dm))
    return ref


def grads_in(t, gt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, d = t["x"].shape
    xo = (torch.randn(T, d, generator=g, device="cuda") * 2).to(t["x"].dtype)
    dxo = torch.randn(T, d, generator=g, device="cuda").to(gt)
    du = torch.randn(T, d, generator=g, device="cuda").to(gt) if t["w_pre"] is not None else None
    return xo, dxo, du


def check_backward(t, gt, seed, dxo_none=False, branch=True):
    xo, dxo, du = grads_in(t, gt, seed)
    if dxo_none:
        dxo = None
    g = backward(t, xo, dxo, du, gt, branch)
    ref = backward64(t, xo, dxo, du, branch)
    assert set(g) == set(ref)
    T = t["x"].shape[0]
    for k, (v, m) in ref.items():
        rel, ab = half_step(g[k].dtype)
        # two row sums (21 steps each) and some 20 products and factors, each one
        # u of its terms; sums over the tokens add a step for each token at most
        steps = 96 + (T + 32 if v.dim() == 1 else 0)
        err = (g[k].double() - v).abs()
        assert (err <= rel * v.abs() + steps * U * m + ab).all(), (k, float(err.max()))
    return g, ref


@pytest.mark.parametrize("dtype,grad", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"),
                                        ("f16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("T,d", SIZES)
def test_backward(T, d, dtype, grad):
    for i, (gate, (post, pre)) in enumerate(itertools.product(
            ("none", "channel", "token", "full"), ((True, True), (False, True), (True, False),
                                                   (False, False)))):
        check_backward(inputs(T, d, DT[dtype], gate, post, pre, d + i), DT[grad], T + i)


@pytest.mark.parametrize("T,d,gate", [(5003, 136, "channel"), (1203, 4096, "channel"),
                                      (301, 8200, "token"), (700, 1000, "full")])
def test_backward_many_rows(T, d, gate):
    check_backward(inputs(T, d, torch.bfloat16, gate, True, True, 4), torch.float32, 5)


@pytest.mark.parametrize("T,d", [(301, 4104), (331, 8192), (70, 8200), (230, 16384)])
def test_wide_rows(T, d):
    """Rows of one CTA and of a cluster, more and fewer than run at once."""
    for dtype, grad, gate in (("bf16", "bf16", "full"), ("bf16", "f32", "token"),
                              ("f16", "f16", "channel"), ("f32", "f32", "none")):
        t = inputs(T, d, DT[dtype], gate, True, True, d + T)
        check_forward(t)
        check_backward(t, DT[grad], T)


@pytest.mark.parametrize("T,d", [(200, 8192), (3, 16384)])
def test_wide_rows_captured(T, d):
    """Clusters in a graph, as a call outside it does."""
    t = inputs(T, d, torch.float16, "token", True, True, 3)
    want = forward(t)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = forward(t)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_backward_without_stream_gradient_or_branch():
    t = inputs(33, 1000, torch.bfloat16, "channel", True, True, 1)
    check_backward(t, torch.float32, 2, dxo_none=True)
    t = inputs(33, 1000, torch.bfloat16, "none", False, True, 1, branch=False)
    check_backward(t, torch.float32, 2, branch=False)
    check_backward(t, torch.float32, 2, dxo_none=True, branch=False)


def test_backward_in_place_and_reproducible():
    t = inputs(777, 1000, torch.bfloat16, "channel", True, True, 1)
    xo, dxo, du = grads_in(t, torch.float32, 3)
    a = backward(t, xo, dxo, du, torch.float32)
    b = backward(t, xo, dxo, du, torch.float32)
    c = backward(t, xo, dxo.clone(), du, torch.float32, in_place=True)
    for k in a:
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k])


def test_backward_against_differences():
    """The gradients along random directions of x, y, the gains and the gate
    against central differences of the forward in 64 bits (step 1e-6)."""
    T, d = 6, 264
    t = inputs(T, d, torch.float32, "channel", True, True, 5)
    names = ["x", "y", "w_post", "gate", "w_pre"]
    g = torch.Generator(device="cuda").manual_seed(1)
    v = {k: torch.randn(t[k].shape, generator=g, device="cuda", dtype=torch.float64) for k in names}
    dxo = torch.randn(T, d, generator=g, device="cuda")
    du = torch.randn(T, d, generator=g, device="cuda")

    def stream(h):
        p = {k: d64(t[k]) + h * v[k] for k in names}
        xo = 0.9 * p["x"] - 0.7 * p["gate"] * p["y"] * rnorm(p["y"]) * p["w_post"]
        return xo, xo * rnorm(xo) * p["w_pre"]

    def L(h):
        xo, u = stream(h)
        return float((xo * d64(dxo)).sum() + (u * d64(du)).sum())
    quotient = (L(1e-6) - L(-1e-6)) / 2e-6
    xo = stream(0)[0].float()   # the stored stream: within u of the exact one
    got = backward(t, xo, dxo, du, torch.float32)
    ref = backward64(t, xo, dxo, du)
    of = {"x": "dx", "y": "dy", "w_post": "dw_post", "gate": "dgate", "w_pre": "dw_pre"}
    total = sum(float((got[of[k]].double() * v[k]).sum()) for k in names)
    size = sum(float((ref[of[k]][1] * v[k].abs()).sum()) for k in names)
    assert abs(total - quotient) <= (200 * U + 1e-8) * size


def test_empty_batch_streams_and_graph():
    b = moe.block_norm(0, 64, moe.GATE_CHANNEL)
    e = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    moe.moe_block_norm_fwd(b, e, y=e, w_post=w, gate=w, w_pre=w, x_out=e, u=e)
    out = {k: torch.full((64,), 3.0, device="cuda") for k in ("dgate", "dw_post", "dw_pre")}
    moe.moe_block_norm_bwd(b, e, {"dx": e, "dy": e, **out}, x_out=e, y=e, w_post=w, gate=w, w_pre=w,
                           du=e)
    assert all((o == 0).all() for o in out.values())
    t = inputs(300, 1000, torch.bfloat16, "channel", True, True, 1)
    xo, dxo, du = grads_in(t, torch.float32, 3)
    ref_f, ref_b = forward(t), backward(t, xo, dxo, du, torch.float32)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        f, g = forward(t), backward(t, xo, dxo, du, torch.float32)
    st.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(f, ref_f))
    assert all(torch.equal(g[k], ref_b[k]) for k in g)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        f, g = forward(t), backward(t, xo, dxo, du, torch.float32)
    for _ in range(2):
        gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(f, ref_f))
    assert all(torch.equal(g[k], ref_b[k]) for k in g)
