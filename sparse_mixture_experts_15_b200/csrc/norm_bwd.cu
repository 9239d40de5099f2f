// The gradients of the block norms: the entry, CTAs of 256 threads and the sums
// over the tokens (norm_bwd.cuh has the formulas and the kernel of the rows).
#include "norm_bwd.cuh"

namespace moe {
namespace {

// The gains' gradients from the parts: 32 columns for a block, 32 runs of parts
// summed at once (the loads of a run are in flight together), then the runs by
// a shuffle tree.
struct NormSums {
  int parts, d;
  const float *part_pre, *part_q, *w_post, *gate_ch;
  float beta;
  float *dw_pre, *dw_post, *dgate_ch;
};
__global__ void __launch_bounds__(1024) block_norm_sums(const __grid_constant__ NormSums p) {
  pdl_wait();
  pdl_allow_next();
  __shared__ float run[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const float* src = blockIdx.y == 0 ? p.part_pre : p.part_q;
  if (!src) return;
  float a = 0.0f;
  if (blockIdx.x * 32 + lane < p.d) {
    src += blockIdx.x * 32 + lane;
#pragma unroll 10
    for (int i = w; i < p.parts; i += 32) a += src[(size_t)i * p.d];
  }
  run[w][lane] = a;
  __syncthreads();
  a = run[lane][w];  // column w of the block
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  const int c = blockIdx.x * 32 + w;
  if (lane != 0 || c >= p.d) return;
  if (blockIdx.y == 0) {
    p.dw_pre[c] = a;
  } else {
    if (p.dw_post) p.dw_post[c] = p.beta * (p.gate_ch ? p.gate_ch[c] : 1.0f) * a;
    if (p.dgate_ch) p.dgate_ch[c] = p.beta * (p.w_post ? p.w_post[c] : 1.0f) * a;
  }
}

}  // namespace

int block_norm_bwd_256(NormBwd p, int dtype, int grad_dtype, int* parts, cudaStream_t st) {
  return bwd_typed<kNormThreads>(p, dtype, grad_dtype, parts, st);
}

}  // namespace moe

extern "C" size_t moe_block_norm_bwd_workspace_bytes(const moe_block_norm* norm) {
  if (!moe::norm_ok(norm)) return 0;
  return moe::align_up((size_t)2 * moe::kBwdParts * norm->d * 4, 256);
}

extern "C" int moe_block_norm_bwd(const moe_block_norm* norm, int32_t dtype, int32_t grad_dtype,
                                  const void* x_out, const void* y, const float* w_post,
                                  const void* gate, const float* w_pre, const void* dx_out,
                                  const void* du, const moe_block_norm_grads* grads, void* ws,
                                  size_t ws_bytes, void* stream) {
  using namespace moe;
  if (!norm_ok(norm) || !grads || !valid_act_dtype(dtype)) return MOE_ERR_INVALID_ARG;
  if (grad_dtype != MOE_F32 && grad_dtype != dtype) return MOE_ERR_UNSUPPORTED;
  const moe_block_norm& b = *norm;
  const moe_block_norm_grads& g = *grads;
  cudaStream_t st = as_stream(stream);
  if (b.T == 0) {  // empty tensors may have no address; sums over no tokens
    float* out[3] = {g.dw_post, g.dw_pre,
                     b.gate == MOE_GATE_CHANNEL ? static_cast<float*>(g.dgate) : nullptr};
    cudaError_t e = cudaSuccess;
    for (float* o : out) {
      if (!aligned16(o)) return MOE_ERR_INVALID_ARG;
      if (o && e == cudaSuccess) e = cudaMemsetAsync(o, 0, (size_t)b.d * 4, st);
    }
    return cuda_status(e);
  }
  const bool branch = g.dy != nullptr;
  if ((gate != nullptr) != (b.gate != MOE_GATE_NONE) || (g.dgate != nullptr) != (gate != nullptr) ||
      (g.dw_post != nullptr) != (w_post != nullptr) || (g.dw_pre != nullptr) != (w_pre != nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!branch && (w_post || gate || !w_pre)) return MOE_ERR_INVALID_ARG;
  if (!g.dx || (w_pre && (!x_out || !du)) || (!w_pre && !dx_out) || ((w_post || gate) && !y))
    return MOE_ERR_INVALID_ARG;
  const void* al[] = {x_out, y, w_post, w_pre, dx_out, du, g.dx, g.dy, g.dw_post, g.dw_pre,
                      b.gate == MOE_GATE_TOKEN ? nullptr : gate,
                      b.gate == MOE_GATE_TOKEN ? nullptr : g.dgate};
  for (const void* q : al)
    if (!aligned16(q)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(ws)) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < moe_block_norm_bwd_workspace_bytes(norm)) return MOE_ERR_WORKSPACE;
  NormBwd p{};
  p.T = b.T;
  p.d = b.d;
  p.x_out = w_pre ? x_out : nullptr;
  p.y = w_post || gate ? y : nullptr;
  p.gate_full = b.gate == MOE_GATE_FULL ? gate : nullptr;
  p.gate_ch = b.gate == MOE_GATE_CHANNEL ? static_cast<const float*>(gate) : nullptr;
  p.gate_tok = b.gate == MOE_GATE_TOKEN ? static_cast<const float*>(gate) : nullptr;
  p.branch = branch;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.dx_out = dx_out;
  p.du = w_pre ? du : nullptr;
  p.alpha = b.res_scale;
  p.beta = b.out_scale;
  p.eps = b.eps;
  p.inv_d = 1.0f / (float)b.d;
  p.dx = g.dx;
  p.dy = g.dy;
  p.dgate_full = b.gate == MOE_GATE_FULL ? g.dgate : nullptr;
  p.dgate_tok = b.gate == MOE_GATE_TOKEN ? static_cast<float*>(g.dgate) : nullptr;
  p.status = status_word();
  float* parts = static_cast<float*>(ws);
  NormSums s{};
  s.d = p.d;
  s.w_post = p.w_post;
  s.gate_ch = p.gate_ch;
  s.beta = p.beta;
  s.dw_pre = g.dw_pre;
  s.dw_post = g.dw_post;
  s.dgate_ch = p.gate_ch ? static_cast<float*>(g.dgate) : nullptr;
  const bool q_sum = s.dw_post || s.dgate_ch;
  s.part_pre = p.part_pre = s.dw_pre ? parts : nullptr;
  s.part_q = p.part_q = q_sum ? parts + (size_t)kBwdParts * p.d : nullptr;
  const int row = bwd_row_bytes(dtype == MOE_F32 ? 4 : 2, grad_dtype == MOE_F32 ? 4 : 2, p.w_pre,
                                p.y, p.gate_full);
  const int rc = norm_wide(p.T, p.d, 5120) && bwd_fits(row, kWideThreads)
                     ? block_norm_bwd_512(p, dtype, grad_dtype, &s.parts, st)
                     : block_norm_bwd_256(p, dtype, grad_dtype, &s.parts, st);
  if (rc != MOE_OK || (!s.dw_pre && !q_sum)) return rc;
  MOE_PREFER_SHARED((block_norm_sums));
  launch_pdl(block_norm_sums, dim3((p.d + 31) / 32, q_sum ? 2 : 1), dim3(1024), 0, st, s);
  return launch_status();
}
