"""The operators around and inside a block run together, as a program uses them:
a serving step (norm, scored routing, permutation, 8-bit experts, combine, norm
with the residual) and a training step (norms around the bf16 layer and its
backward, the router's gradient from the experts' rows)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_mixture_experts_15_b200 as moe

EPS = 1e-6


@pytest.fixture(autouse=True)
def _clean_status():
    moe.moe_reset_device_status()
    yield
    assert moe.moe_device_status() == 0


def randn(g, *s, sd=1.0):
    return torch.randn(*s, generator=g, device="cuda") * sd


def rms(v, w):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * w.double()


class ServingStep:
    """x_out, u_next for a stream x: one block with 8-bit experts."""

    def __init__(self, T, d, N, k, h, groups, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.d, self.N, self.k, self.h = T, d, N, k, h
        self.x = randn(g, T, d).bfloat16()
        self.w_pre, self.w_post, self.w_next = (1 + randn(g, d, sd=0.1) for _ in range(3))
        self.layer_scale = randn(g, d, sd=0.5)
        self.w_route, self.bias = randn(g, N, d, sd=d ** -0.5), randn(g, N, sd=0.05)
        self.mats = {}
        for name, (a, b) in dict(gate=(N * h, d), up=(N * h, d), down=(N * d, h)).items():
            w = randn(g, a, b, sd=b ** -0.5).bfloat16()
            q = torch.empty(a, b, dtype=torch.int8, device="cuda")
            s = torch.empty(a, device="cuda")
            moe.moe_quantize_i8_rows(w, q, s)
            self.mats[name] = (q, s)
        self.s = moe.shape(T, d, N, k, h)
        self.gating = moe.gating(moe.SCORE_SIGMOID, groups, max(1, groups // 2), min(2, N // groups),
                                 1.5)
        self.pre = moe.block_norm(T, d, eps=EPS)
        self.post = moe.block_norm(T, d, moe.GATE_CHANNEL, 1.0, 0.8, EPS)
        bf, i32 = dict(device="cuda", dtype=torch.bfloat16), dict(device="cuda", dtype=torch.int32)
        R = T * k
        self.u, self.y = torch.empty(T, d, **bf), torch.empty(T, d, **bf)
        self.x_out, self.u_next = torch.empty(T, d, **bf), torch.empty(T, d, **bf)
        self.idx, self.w = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda")
        self.counts, self.over = torch.empty(N, **i32), torch.empty(N, **i32)
        self.off, self.perm = torch.empty(N + 1, **i32), torch.empty(R, **i32)
        self.row_of, self.totals = torch.empty(T, k, **i32), torch.empty(3, **i32)
        self.rows = torch.empty(R, d, **bf)
        self.codes = torch.empty(R, d, dtype=torch.int8, device="cuda")
        self.scales = torch.empty(R, device="cuda")
        self.y_rows = torch.empty(R, d, device="cuda")
        byte = lambda n: torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")  # noqa: E731
        self.ws_ffn = byte(moe.moe_expert_ffn_i8_workspace_bytes(self.s))
        self.ws_route = torch.empty(T, N, device="cuda")
        self.ws_perm = byte(1 << 22)

    def __call__(self):
        m, s = self.mats, self.s
        moe.moe_block_norm_fwd(self.pre, self.x, w_pre=self.w_pre, u=self.u)
        moe.moe_route_scored(s, self.gating, self.u, self.w_route, self.idx, self.w,
                             bias=self.bias, logits=self.ws_route)
        moe.moe_permute(s, self.idx, self.counts, self.off, self.perm, self.row_of, self.over,
                        self.totals, ws=self.ws_perm)
        moe.moe_gather(s, self.d, self.u, self.perm, self.off, self.rows)
        moe.moe_quantize_i8_rows(self.rows, self.codes, self.scales)
        moe.moe_expert_ffn_i8(s, self.d, self.codes, self.scales, self.off, m["gate"][0],
                              m["up"][0], m["down"][0], m["gate"][1], m["up"][1], m["down"][1],
                              self.y_rows, ws=self.ws_ffn)
        moe.moe_combine(s, self.d, self.y_rows, self.row_of, self.w, self.y)
        moe.moe_block_norm_fwd(self.post, self.x, y=self.y, w_post=self.w_post,
                               gate=self.layer_scale, w_pre=self.w_next, x_out=self.x_out,
                               u=self.u_next)

    def reference(self):
        """The same block in 64 bits from the kernel's own routing: u rounded to
        bf16 and quantised, H rounded to bf16 and quantised."""
        val = {n: q.double() * s.double()[:, None] for n, (q, s) in self.mats.items()}
        x = self.x.double()
        u = rms(x, self.w_pre).bfloat16().float()

        def q8(v):
            s = v.abs().amax(1, keepdim=True) * torch.full_like(v[:, :1], float(np.float32(1 / 127)))
            s = torch.where(s > 0, s, torch.ones_like(s))
            return torch.round(v / s).clamp(-127, 127).double() * s.double()
        uq, y, h, d = q8(u), torch.zeros_like(x), self.h, self.d
        for e in range(self.N):
            t, slot = (self.idx == e).nonzero(as_tuple=True)
            if len(t):
                a = uq[t] @ val["gate"][e * h:(e + 1) * h].T
                b = uq[t] @ val["up"][e * h:(e + 1) * h].T
                H = q8((a * torch.sigmoid(a) * b).bfloat16().float())
                y.index_add_(0, t, self.w[t, slot].double()[:, None]
                             * (H @ val["down"][e * d:(e + 1) * d].T))
        y = y.bfloat16().double()
        xo = x + 0.8 * self.layer_scale.double() * rms(y, self.w_post)
        return xo, rms(xo, self.w_next)


@pytest.mark.parametrize("T,d,N,k,h,groups", [(1, 256, 8, 2, 128, 1), (3, 512, 64, 8, 128, 8),
                                              (130, 256, 16, 4, 256, 4)])
def test_serving_step(T, d, N, k, h, groups):
    """The stream within 2^-7 in the 2-norm: its own rounding to bf16 (2^-9 rms),
    the block's output rounded to bf16 before its norm (2^-9), and the codes of u
    and H that fall on the other side of a tie (1e-3 of the experts' output,
    as for the FFN alone); routing ids exactly, given the kernel's u."""
    step = ServingStep(T, d, N, k, h, groups, seed=T + N)
    step()
    # routing from the kernel's own u, by the definition in 64 bits
    z = step.ws_route.double()
    c = (1 / (1 + torch.exp(-z))).float() + step.bias
    if groups > 1:
        per = c.view(T, groups, -1)
        gs = per.topk(min(2, N // groups), dim=2).values.sum(2)
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(
            1, torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :groups // 2], True)
        c = torch.where(keep[:, :, None], per, -torch.inf).view(T, N)
    idx = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(idx.int(), step.idx)
    for got, ref in zip((step.x_out, step.u_next), step.reference()):
        assert float((got.double() - ref).norm() / ref.norm()) <= 2.0 ** -7


def test_serving_step_captured():
    """The step captured once and replayed on another stream's contents equals
    the calls made one by one, also with two steps' graphs in turn."""
    a, b = ServingStep(40, 256, 16, 4, 128, 4, 1), ServingStep(2, 256, 16, 4, 128, 4, 2)
    graphs = []
    for step in (a, b):
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for seed in (5, 6):
        for step in (a, b):
            step.x.copy_(randn(torch.Generator(device="cuda").manual_seed(seed), step.T, step.d))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for step in (a, b):
            got = [t.clone() for t in (step.idx, step.w, step.x_out, step.u_next)]
            step()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in
                       zip(got, (step.idx, step.w, step.x_out, step.u_next)))


def test_training_step():
    """x' = x + gate norm(layer(norm(x))) and its gradients, the layer's and the
    norms' kernels chained, against differentiation in 64 bits with the kernel's
    selected experts.  Each gradient passes the layer's bf16 roundings (bounded
    by 1e-2 in the 2-norm for the layer alone) and two more of bf16 rows (dy and
    u, 2^-9 rms each)."""
    T, d, N, k, h = 192, 256, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    x = randn(g, T, d).bfloat16()
    w_pre, w_post, gate = 1 + randn(g, d, sd=0.1), 1 + randn(g, d, sd=0.1), randn(g, d, sd=0.5)
    wr = randn(g, N, d, sd=d ** -0.5)
    wg, wu = (randn(g, N, h, d, sd=d ** -0.5).bfloat16() for _ in range(2))
    wd = randn(g, N, d, h, sd=h ** -0.5).bfloat16()
    dxo = randn(g, T, d)
    s = moe.shape(T, d, N, k, h)
    pre, post = moe.block_norm(T, d, eps=EPS), moe.block_norm(T, d, moe.GATE_CHANNEL, eps=EPS)
    bf, f32 = dict(device="cuda", dtype=torch.bfloat16), dict(device="cuda")
    i32 = dict(device="cuda", dtype=torch.int32)
    u, y, xo = (torch.empty(T, d, **bf) for _ in range(3))
    fwd = dict(top_idx=torch.empty(T, k, **i32), top_w=torch.empty(T, k, **f32),
               probs=torch.empty(T, N, **f32), offsets=torch.empty(N + 1, **i32),
               perm_tok=torch.empty(T * k, **i32), row_of=torch.empty(T, k, **i32))
    moe.moe_block_norm_fwd(pre, x, w_pre=w_pre, u=u)
    moe.moe_layer_fwd(s, wr, wg, wu, wd, u, y, outputs=fwd)
    moe.moe_block_norm_fwd(post, x, y=y, w_post=w_post, gate=gate, x_out=xo)
    dx, dy, dx2 = torch.empty(T, d, **f32), torch.empty(T, d, **bf), torch.empty(T, d, **f32)
    dw_post, dgate, dw_pre = (torch.empty(d, **f32) for _ in range(3))
    moe.moe_block_norm_bwd(post, dxo, dict(dx=dx, dy=dy, dgate=dgate, dw_post=dw_post), y=y,
                           w_post=w_post, gate=gate)
    lg = dict(du=torch.empty(T, d, **f32), dz=torch.empty(T, N, **f32),
              dw_route=torch.empty(N, d, **f32), dw_gate=torch.empty(N, h, d, **f32),
              dw_up=torch.empty(N, h, d, **f32), dw_down=torch.empty(N, d, h, **f32))
    moe.moe_layer_bwd(s, wr, wg, wu, wd, u, dy, fwd, lg)
    moe.moe_block_norm_bwd(pre, dx, dict(dx=dx2, dw_pre=dw_pre), x_out=x, w_pre=w_pre,
                           du=lg["du"])

    leaf = {n: v.double().requires_grad_(True) for n, v in
            dict(x=x, w_pre=w_pre, w_post=w_post, gate=gate, wr=wr, wg=wg, wu=wu, wd=wd).items()}
    un = leaf["x"] / torch.sqrt((leaf["x"] ** 2).mean(1, keepdim=True) + EPS) * leaf["w_pre"]
    p = torch.softmax(un @ leaf["wr"].T, 1)
    idx = fwd["top_idx"].long()
    a = p.gather(1, idx)
    a = a / a.sum(1, keepdim=True)
    out = torch.zeros_like(un)
    for e in range(N):
        t, slot = (idx == e).nonzero(as_tuple=True)
        gt, up = un[t] @ leaf["wg"][e].T, un[t] @ leaf["wu"][e].T
        out = out.index_add(0, t, a[t, slot][:, None]
                            * ((gt * torch.sigmoid(gt) * up) @ leaf["wd"][e].T))
    yn = out / torch.sqrt((out ** 2).mean(1, keepdim=True) + EPS) * leaf["w_post"]
    total = ((leaf["x"] + leaf["gate"] * yn) * dxo.double()).sum()
    ref = dict(zip(leaf, torch.autograd.grad(total, list(leaf.values()))))
    got = dict(x=dx2, w_pre=dw_pre, w_post=dw_post, gate=dgate, wr=lg["dw_route"],
               wg=lg["dw_gate"], wu=lg["dw_up"], wd=lg["dw_down"])
    for n, r in ref.items():
        assert float((got[n].double() - r).norm() / r.norm()) <= 1e-2 + 2 * 2.0 ** -8, n

    # the router's gradient alone, from the experts' rows: da_s = dy . F_s(u)
    rows, y_rows = torch.empty(T * k, d, **bf), torch.empty(T * k, d, **f32)
    moe.moe_gather(s, d, u, fwd["perm_tok"], fwd["offsets"], rows)
    moe.moe_expert_ffn(s, d, rows, fwd["offsets"], wg, wu, wd, y_rows)
    da = (y_rows[fwd["row_of"].long()] * dy.float()[:, None, :]).sum(2)
    z, dz = torch.empty(T, N, **f32), torch.empty(T, N, **f32)
    idx2, w2 = torch.empty(T, k, **i32), torch.empty(T, k, **f32)
    moe.moe_route_scored(s, moe.gating(), u, wr, idx2, w2, logits=z)
    assert torch.equal(idx2, fwd["top_idx"])
    moe.moe_route_select_bwd(s, moe.gating(), z, idx2, da, dz)
    assert float((dz - lg["dz"]).norm() / lg["dz"].norm()) <= 1e-2


def test_two_steps_at_once():
    """Two steps on two streams at the same time, each with its own buffers,
    give what they give alone; tensors made on another stream are used after it."""
    steps = [ServingStep(300, 512, 16, 4, 128, 4, 1), ServingStep(2, 512, 64, 8, 128, 8, 2)]
    alone = []
    for step in steps:
        step()
        torch.cuda.synchronize()
        alone.append([t.clone() for t in (step.idx, step.w, step.x_out, step.u_next)])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for st, step in zip(streams, steps):
            with torch.cuda.stream(st):
                step()
    torch.cuda.synchronize()
    for step, ref in zip(steps, alone):
        got = (step.idx, step.w, step.x_out, step.u_next)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_a_stream_given_by_its_handle():
    """A call on a stream that is not the current one, its workspace made by the
    call: the workspace's memory is not given to the next tensor meanwhile."""
    T, d = 2000, 1024
    g = torch.Generator(device="cuda").manual_seed(0)
    x, y, dxo, du = (randn(g, T, d).bfloat16() for _ in range(4))
    w = 1 + randn(g, d, sd=0.1)
    b = moe.block_norm(T, d, eps=EPS)

    def grads(stream=None):
        out = dict(dx=torch.empty_like(x), dy=torch.empty_like(x),
                   dw_post=torch.empty(d, device="cuda"), dw_pre=torch.empty(d, device="cuda"))
        torch.cuda.synchronize()
        moe.moe_block_norm_bwd(b, dxo, out, x_out=x, y=y, w_post=w, w_pre=w, du=du,
                               stream=None if stream is None else stream.cuda_stream)
        junk = [torch.full((1 << 22,), 7.0, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        del junk
        return out
    ref = grads()
    for _ in range(5):
        got = grads(torch.cuda.Stream())
        assert all(torch.equal(ref[k], got[k]) for k in ref)
