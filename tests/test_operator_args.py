"""Refusals of the scored-routing, block-norm and 8-bit integer entry points,
on the host: every bad size, kind, combination, alignment or tensor is an
error before anything is launched."""
import ctypes

import pytest
import torch

import sparse_mixture_experts_15_b200 as moe

P = 4096  # a non-NULL, aligned address: the checks run before any device work
lib = moe._lib
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -6


def _select(s, g, logits=P, bias=None, idx=P, w=P, scores=None):
    return lib.moe_route_select(ctypes.byref(s), ctypes.byref(g), logits, bias, idx, w, scores,
                                None)


@pytest.mark.parametrize("N,k,kw", [
    (64, 8, dict(score=2)), (64, 8, dict(score=-1)),
    (64, 8, dict(n_group=0)), (64, 8, dict(n_group=3)), (1024, 8, dict(n_group=64)),
    (64, 8, dict(n_group=8, top_group=0)), (64, 8, dict(n_group=8, top_group=9)),
    (64, 9, dict(n_group=8, top_group=1)),               # 8 experts cannot give 9
    (64, 8, dict(n_group=8, top_group=4, group_top=0)),
    (64, 8, dict(n_group=8, top_group=4, group_top=3)),
    (8, 2, dict(n_group=8, top_group=4, group_top=2)),   # one expert a group has no second
    (1025, 8, {}), (0, 1, {}), (64, 33, {}), (4, 5, {}), (64, 0, {}),
])
def test_gating_refused(N, k, kw):
    s, g = moe.shape(16, 64, N, k), moe.gating(**kw)
    assert _select(s, g) == INVALID
    assert lib.moe_route_select_bwd(ctypes.byref(s), ctypes.byref(g), P, P, P, None, P,
                                    None) == INVALID
    assert lib.moe_route_scored(ctypes.byref(s), ctypes.byref(g), P, moe.BF16, P, None, P, P, None,
                                P, None, 0, None) == INVALID


def test_select_pointers():
    s, g = moe.shape(16, 64, 64, 8), moe.gating()
    assert _select(s, g, logits=None) == INVALID
    assert _select(s, g, idx=None) == INVALID
    assert _select(s, g, w=None) == INVALID
    assert _select(s, g, logits=P + 4) == INVALID
    assert _select(s, g, scores=P + 8) == INVALID
    assert _select(s, g, bias=P + 2) == INVALID
    assert _select(moe.shape(-1, 64, 64, 8), g) == INVALID
    assert _select(moe.shape(0, 64, 64, 8), g, None, None, None, None) == 0
    args = [P, P, P, None, P]
    for at in (0, 1, 2, 4):
        bad = list(args)
        bad[at] = None
        assert lib.moe_route_select_bwd(ctypes.byref(s), ctypes.byref(g), *bad, None) == INVALID
    assert lib.moe_route_scored(ctypes.byref(s), ctypes.byref(g), P, moe.BF16, P, None, P, P, None,
                                None, P, 16, None) == WORKSPACE
    assert lib.moe_route_scored(ctypes.byref(s), ctypes.byref(g), P, moe.E4M3, P, None, P, P, None,
                                P, None, 0, None) == INVALID
    assert lib.moe_route_scored_workspace_bytes(ctypes.byref(s)) >= 16 * 64 * 4


def _fwd(b, dtype=moe.BF16, x=P, y=P, w_post=P, gate=None, w_pre=P, x_out=P, u=P):
    return lib.moe_block_norm_fwd(ctypes.byref(b), dtype, x, y, w_post, gate, w_pre, x_out, u, None)


def _bwd(b, dtype=moe.BF16, gdt=moe.F32, x_out=P, y=P, w_post=P, gate=None, w_pre=P, dxo=P, du=P,
         dx=P, dy=P, dgate=None, dw_post=P, dw_pre=P, ws=P, wlen=1 << 30):
    g = moe.MoeBlockNormGrads(dx, dy, dgate, dw_post, dw_pre)
    return lib.moe_block_norm_bwd(ctypes.byref(b), dtype, gdt, x_out, y, w_post, gate, w_pre, dxo,
                                  du, ctypes.byref(g), ws, wlen, None)


@pytest.mark.parametrize("T,d,kw", [(4, 12, {}), (4, 0, {}), (4, -8, {}), (-1, 64, {}),
                                    (4, 16392, {}), (4, 64, dict(gate=4)), (4, 64, dict(gate=-1)),
                                    (4, 64, dict(eps=0.0)), (4, 64, dict(eps=-1e-6)),
                                    (4, 64, dict(eps=float("nan")))])
def test_norm_sizes(T, d, kw):
    b = moe.block_norm(T, d, **kw)
    assert _fwd(b) == INVALID
    assert _bwd(b) == INVALID
    assert lib.moe_block_norm_bwd_workspace_bytes(ctypes.byref(b)) == 0


def test_norm_combinations():
    b, c = moe.block_norm(4, 64), moe.block_norm(4, 64, gate=moe.GATE_CHANNEL)
    assert _fwd(b, dtype=moe.E4M3) == INVALID
    assert _fwd(b, x=None) == INVALID
    assert _fwd(b, x_out=None) == INVALID            # y without a place for the sum
    assert _fwd(b, u=None) == INVALID                # w_pre without a place for u
    assert _fwd(b, y=None, w_post=None, w_pre=None) == INVALID   # nothing to do
    assert _fwd(b, y=None) == INVALID                # a post norm of nothing
    assert _fwd(c, y=None, w_post=None, gate=P) == INVALID
    assert _fwd(c) == INVALID                        # a gate kind without a gate
    assert _fwd(b, gate=P) == INVALID                # a gate without its kind
    for name in ("x", "y", "w_post", "w_pre", "x_out", "u"):
        assert _fwd(b, **{name: P + 8}) == INVALID
    assert _fwd(c, gate=P + 4) == INVALID
    assert _fwd(moe.block_norm(0, 64), x=None, y=None, w_post=None, x_out=None, u=None) == 0

    assert _bwd(b, gdt=moe.F16) == UNSUPPORTED
    assert _bwd(b, dtype=moe.F32, gdt=moe.BF16) == UNSUPPORTED
    assert _bwd(b, dx=None) == INVALID
    assert _bwd(b, x_out=None) == INVALID
    assert _bwd(b, du=None) == INVALID
    assert _bwd(b, y=None) == INVALID
    assert _bwd(b, dw_post=None) == INVALID
    assert _bwd(b, dw_pre=None) == INVALID
    assert _bwd(b, w_post=None) == INVALID           # dw_post without w_post
    assert _bwd(b, dgate=P) == INVALID
    assert _bwd(c, gate=P) == INVALID                # gate without dgate
    assert _bwd(b, dy=None) == INVALID               # a post norm of no branch
    assert _bwd(b, dy=None, w_post=None, dw_post=None, w_pre=None, dw_pre=None) == INVALID
    assert _bwd(b, w_pre=None, dw_pre=None, dxo=None) == INVALID  # no gradient comes in
    assert _bwd(b, ws=None) == WORKSPACE
    assert _bwd(b, wlen=1024) == WORKSPACE
    for name in ("x_out", "y", "w_post", "w_pre", "dxo", "du", "dx", "dy", "dw_post", "dw_pre",
                 "ws"):
        assert _bwd(b, **{name: P + 8}) == INVALID


def _gemm(rows=4, G=1, K=64, n=8, x=P, xs=P, off=None, w=P, wsc=P, y=P, ydt=moe.F32):
    return lib.moe_grouped_gemm_i8(rows, G, K, n, x, xs, off, w, wsc, y, ydt, P, 1 << 30, None)


def test_i8_arguments():
    q = lib.moe_quantize_i8_rows
    assert q(4, 24, P, moe.BF16, P, P, None) == INVALID
    assert q(4, 0, P, moe.BF16, P, P, None) == INVALID
    assert q(-1, 32, P, moe.BF16, P, P, None) == INVALID
    assert q(4, 32, P, moe.E4M3, P, P, None) == UNSUPPORTED
    assert q(4, 32, None, moe.BF16, P, P, None) == INVALID
    assert q(4, 32, P, moe.F16, P + 8, P, None) == INVALID
    assert q(4, 32, P + 2, moe.F16, P, P, None) == INVALID
    assert q(4, 32, P, moe.F16, P, P + 2, None) == INVALID
    assert q(0, 32, None, moe.F32, None, None, None) == 0
    assert _gemm(K=24) == INVALID
    assert _gemm(K=0) == INVALID
    assert _gemm(K=131072) == INVALID                # the s32 sum could pass its range
    assert _gemm(n=0) == INVALID
    assert _gemm(G=0, off=P) == INVALID
    assert _gemm(G=1025, off=P) == INVALID
    assert _gemm(G=2) == INVALID                     # groups without their offsets
    assert _gemm(rows=-1) == INVALID
    assert _gemm(G=1024, n=1 << 22, off=P) == INVALID
    assert _gemm(ydt=moe.E4M3) == UNSUPPORTED
    for name in ("x", "xs", "w", "wsc", "y"):
        assert _gemm(**{name: None}) == INVALID
        assert _gemm(**{name: P + 2}) == INVALID
    assert _gemm(rows=0, x=None, xs=None, y=None) == 0


def test_ffn_i8_arguments():
    s, a = moe.shape(16, 128, 4, 2, 128), moe.act()
    sc = moe.MoeI8Scales(P, P, P)

    def call(s=s, width=128, x=P, xs=P, off=P, wg=P, sc=sc, a=a, y=P, ws=P, n=1 << 30):
        return lib.moe_expert_ffn_i8(ctypes.byref(s), width, x, xs, off, wg, P, P,
                                     ctypes.byref(sc), ctypes.byref(a), y, ws, n, None)
    assert call(width=64) == UNSUPPORTED
    assert call(s=moe.shape(16, 128, 4, 2, 64)) == UNSUPPORTED
    assert call(off=None) == INVALID
    assert call(x=None) == INVALID
    assert call(wg=None) == INVALID
    assert call(wg=P + 8) == INVALID
    assert call(sc=moe.MoeI8Scales(P, None, P)) == INVALID
    assert call(a=moe.act(moe.ACT_SITU_GLU, 0.0, 25.0)) == INVALID
    assert call(n=64) == WORKSPACE
    assert call(s=moe.shape(0, 128, 4, 2, 128), x=None, xs=None, y=None, ws=None, n=0) == 0
    assert lib.moe_expert_ffn_i8_workspace_bytes(ctypes.byref(s)) >= 32 * 128 * 3 + 32 * 4


def test_binding_refuses_bad_tensors():
    s, g = moe.shape(4, 64, 8, 2), moe.gating()
    f, i = torch.zeros, torch.int32
    with pytest.raises(ValueError, match="logits: 31 elements, the call needs at least 32"):
        moe.moe_route_select(s, g, f(31), f(8, dtype=i), f(8))
    with pytest.raises(ValueError, match="logits: dtype bfloat16"):
        moe.moe_route_select(s, g, f(32, dtype=torch.bfloat16), f(8, dtype=i), f(8))
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.moe_route_select(s, g, f(32), f(8, dtype=i), f(8))
    b = moe.block_norm(4, 64)
    with pytest.raises(ValueError, match="x: 255 elements"):
        moe.moe_block_norm_fwd(b, f(255), w_pre=f(64), u=f(256))
    with pytest.raises(ValueError, match="dx: dtype int32"):
        moe.moe_block_norm_bwd(b, f(256), {"dx": f(256, dtype=i)})
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.moe_quantize_i8_rows(f((4, 16)), f(64, dtype=torch.int8), f(4))
    with pytest.raises(ValueError, match="x: dtype int8"):
        moe.moe_quantize_i8_rows(f((4, 16), dtype=torch.int8), f(64, dtype=torch.int8), f(4))
    with pytest.raises(ValueError, match="rows of 32 codes, x has rows of 16"):
        moe.moe_grouped_gemm_i8(f((4, 16), dtype=torch.int8), f(4),
                                f((2, 8, 32), dtype=torch.int8), f(16), f((4, 8)))


def test_norm_gradients_of_a_type_without_a_kernel_are_refused():
    """The storage type is taken from x_out, y or dy: another type is a refusal
    that names the tensor."""
    b, f = moe.block_norm(4, 64), torch.zeros
    for kw, grads, what in ((dict(x_out=f(256, dtype=torch.int32)), {}, "x_out"),
                            (dict(y=f(256, dtype=torch.float64)), {}, "y"),
                            ({}, dict(dy=f(256, dtype=torch.int8)), "dy")):
        with pytest.raises(ValueError, match=f"{what}: dtype (int32|float64|int8)"):
            moe.moe_block_norm_bwd(b, f(256), {"dx": f(256), **grads}, **kw)
