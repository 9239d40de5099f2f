"""Which stream the workspace of a call belongs to: memory that a call allocates
for itself must be the allocator's for the stream that the call runs on.  From
another stream's memory it may be a block whose last user, still queued there,
writes while the call reads.  On the host, with the allocator's calls recorded."""
import contextlib
import ctypes
import types

import pytest
import torch

import sparse_mixture_experts_15_b200 as moe

CURRENT, SIDE, DEFAULT = 0x7100, 0x7200, 0


class Recorder:
    """torch as the binding uses it for a workspace; `used` is the streams that
    were current when memory was taken."""

    uint8 = torch.uint8

    def __init__(self):
        self.now, self.used = [CURRENT], []
        self.cuda = types.SimpleNamespace(
            device=lambda dev: contextlib.nullcontext(), stream=self._stream,
            ExternalStream=lambda handle, device=None: self._known(handle),
            default_stream=lambda device=None: DEFAULT,
            current_stream=lambda device=None: types.SimpleNamespace(cuda_stream=self.now[-1]))

    @staticmethod
    def _known(handle):
        assert handle != 0  # an ExternalStream of no handle is a stream of its own
        return handle

    @contextlib.contextmanager
    def _stream(self, s):
        self.now.append(s)
        yield
        self.now.pop()

    def empty(self, n, dtype=None, device=None):
        self.used.append(self.now[-1])
        t = types.SimpleNamespace(is_cuda=True, is_contiguous=lambda: True, data_ptr=lambda: 4096,
                                  numel=lambda: n, element_size=lambda: 1)
        return t


@pytest.fixture
def fake(monkeypatch):
    r = Recorder()
    moe._t.act  # looks torch up, so that nothing is set again below
    monkeypatch.setattr(moe._t, "torch", r)
    monkeypatch.setattr(moe._t, "raw_stream", lambda dev: r.now[-1])
    return r


@pytest.mark.parametrize("stream,owner", [(None, CURRENT), (CURRENT, CURRENT), (SIDE, SIDE),
                                          (0, DEFAULT)])
def test_a_workspace_is_of_the_calls_stream(fake, stream, owner):
    b = moe.block_norm(64, 256)
    p, n, ws = moe._workspace(None, 0, stream, moe._lib.moe_block_norm_bwd_workspace_bytes,
                              ctypes.byref(b))
    assert p == 4096 and n >= 2 * 256 * 4 and ws is not None
    assert fake.used == [owner]
    assert fake.now == [CURRENT]


@pytest.mark.gpu
@pytest.mark.parametrize("side", ["own", "default"])
def test_calls_on_two_streams_do_not_share_a_workspace(side):
    """A call on the current stream, its kernels still queued, then one on another
    stream: each takes its workspace itself, and nothing orders the two streams."""
    T, d = 3000, 1024
    g = torch.Generator(device="cuda").manual_seed(0)
    x, y, dxo, du = (torch.randn(T, d, generator=g, device="cuda").bfloat16() for _ in range(4))
    w = 1 + torch.randn(d, generator=g, device="cuda") * 0.1
    x2, du2 = (3 * torch.randn(T, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    b = moe.block_norm(T, d)

    def outputs():
        return dict(dx=torch.empty_like(x), dy=torch.empty_like(x),
                    dw_post=torch.empty(d, device="cuda"), dw_pre=torch.empty(d, device="cuda"))

    def call(out, x_out, grad, stream=None):
        moe.moe_block_norm_bwd(b, dxo, out, x_out=x_out, y=y, w_post=w, w_pre=w, du=grad,
                               stream=stream)

    ref, ref2 = outputs(), outputs()
    call(ref, x, du)
    call(ref2, x2, du2)
    a, c = outputs(), outputs()
    torch.cuda.synchronize()
    here = torch.cuda.Stream()
    there = torch.cuda.Stream().cuda_stream if side == "own" else 0
    with torch.cuda.stream(here):
        for _ in range(20):
            call(a, x, du)
            call(c, x2, du2, there)
    torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(a[k], ref[k]) and torch.equal(c[k], ref2[k])
    assert moe.moe_device_status() == 0


@pytest.mark.gpu
def test_calls_on_a_forked_stream_of_a_capture():
    """Calls that make their workspaces on a stream that a capture forked, beside one
    on the captured stream: the graph holds the memory, and replays repeat them."""
    T, d, N, k = 2000, 512, 64, 8
    g = torch.Generator(device="cuda").manual_seed(2)
    x, y, dxo, du = (torch.randn(T, d, generator=g, device="cuda").bfloat16() for _ in range(4))
    w, wr = 1 + torch.randn(d, generator=g, device="cuda") * 0.1, torch.randn(N, d, generator=g,
                                                                             device="cuda") * 0.05
    b, s, gt = moe.block_norm(T, d), moe.shape(T, d, N, k), moe.gating(moe.SCORE_SIGMOID)

    def outputs():
        return dict(dx=torch.empty_like(x), dy=torch.empty_like(x),
                    dw_post=torch.empty(d, device="cuda"), dw_pre=torch.empty(d, device="cuda"),
                    idx=torch.empty(T, k, dtype=torch.int32, device="cuda"),
                    w=torch.empty(T, k, device="cuda"))

    def calls(out, stream=None):
        moe.moe_block_norm_bwd(b, dxo, out, x_out=x, y=y, w_post=w, w_pre=w, du=du, stream=stream)
        moe.moe_route_scored(s, gt, x, wr, out["idx"], out["w"], stream=stream)
        moe.moe_route(s, x, wr, out["idx2"], out["w2"], stream=stream)

    outs = [outputs() for _ in range(3)]
    for o in outs:
        o.update(idx2=torch.empty_like(o["idx"]), w2=torch.empty_like(o["w"]))
    calls(outs[0])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        calls(outs[1])
        calls(outs[2], side.cuda_stream)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for o in outs[1:]:
            for v in o.values():
                v.fill_(3)
        junk = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(8)]
        graph.replay()
        torch.cuda.synchronize()
        del junk
        for o in outs[1:]:
            assert all(torch.equal(v, outs[0][n]) for n, v in o.items())
    assert moe.moe_device_status() == 0


class Tensor:
    """A CUDA tensor as the binding sees it."""

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.device, self.is_cuda = dtype, shape, "cuda:0", True

    def numel(self):
        return int(torch.Size(self.shape).numel())

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


@pytest.mark.parametrize("name,args", [
    ("moe_route", lambda s, f, i, h: (s, f(16, 64), f(8, 64), i(16, 2), f(16, 2))),
    ("moe_aux_stats", lambda s, f, i, h: (f(16, 8), i(16, 2), f(8))),
    ("moe_permute", lambda s, f, i, h: (s, i(16, 2), i(8), i(9), i(32), i(32), i(8), i(3))),
    ("moe_expert_ffn", lambda s, f, i, h: (s, 128, h(32, 128), i(9), *(h(8, 128, 128),) * 3,
                                           f(32, 128))),
    ("moe_layer_fwd", lambda s, f, i, h: (s, f(8, 64), *(h(8, 128, 64),) * 3, h(16, 64),
                                          h(16, 64))),
    ("moe_quantile_balance", lambda s, f, i, h: (f(16, 8), 2, 4, f(8))),
])
@pytest.mark.parametrize("stream,owner", [(None, CURRENT), (CURRENT, CURRENT), (SIDE, SIDE),
                                          (0, DEFAULT)])
def test_every_calls_workspace_is_of_its_stream(fake, monkeypatch, name, args, stream, owner):
    """The layer's own calls, with the library's launch left out."""
    make = [lambda *n, dt=dt: Tensor(dt, *n) for dt in (torch.float32, torch.int32, torch.bfloat16)]
    launched = []
    monkeypatch.setattr(moe._lib, name, lambda *a: launched.append(a[-1]) or 0)
    for attr in ("cuda", "empty"):
        monkeypatch.setattr(torch, attr, getattr(fake, attr))
    getattr(moe, name)(*args(moe.shape(16, 64, 8, 2, 128), *make), stream=stream)
    assert fake.used == [owner]
    assert launched == [CURRENT if stream is None else stream]
