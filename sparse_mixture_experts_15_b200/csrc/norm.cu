// The norms around a block of the residual stream, with the block's gate and
// the residual scale, in one pass over the rows:
//   n  = y / sqrt(mean(y^2) + eps) * w_post      (w_post NULL: n = y)
//   x' = res_scale x + out_scale gate n          rounded to the storage type
//   u  = x' / sqrt(mean(x'^2) + eps) * w_pre     of x' as stored
// Sums over a row are fp32 in a fixed order.  Bound by the rows' bytes.
#include "norm.cuh"

namespace moe {
namespace {

constexpr int kFwdCtas = 3;  // CTAs per SM

struct NormFwd {
  int T, d, C;             // C: CTAs of a cluster, each with its share of a row's columns
  int nt;                  // threads per row in a CTA
  const void *x, *y, *gate_full;
  const float *w_post, *w_pre, *gate_ch, *gate_tok;
  float alpha, beta, eps, inv_d;
  void *x_out, *u;
};

// HASY: a block's output comes in (POST: normed first; FULL: gated by element;
// a channel's gate is part of coef, a token's of the row's factor).
template <typename T, int S, bool HASY, bool POST, bool FULL, bool PRE>
__global__ void __launch_bounds__(kNormThreads, kFwdCtas)
    block_norm_fwd(const __grid_constant__ NormFwd p) {
  extern __shared__ __align__(16) char fifo_mem[];
  __shared__ SumBuffers sum_mem;
  pdl_wait();
  pdl_allow_next();
  const Place q = place_of(p.nt, p.C, p.d, p.T);
  RowSum sums{&sum_mem, q.team, p.nt, p.nt / 32, p.C, 0};
  if (p.C > 1) cluster_barrier();  // every CTA of the cluster runs before its memory is written
  constexpr int P = planes<T>();
  const uint32_t step = blockDim.x * 16, stage = P * (1 + HASY + FULL) * step;
  const uint32_t base = smem_addr(fifo_mem + threadIdx.x * 16);
  const size_t skip = (size_t)q.step * p.d;
  Stream<T> sx, sy, sg;
  sx.start(p.x, q, p.d, 0);
  if (HASY) sy.start(p.y, q, p.d, P);
  if (FULL) sg.start(p.gate_full, q, p.d, 2 * P);
  int uncopied = q.count;
  auto issue = [&](uint32_t at) {
    if (uncopied > 0) {
      sx.copy(q, at, step, skip);
      if (HASY) sy.copy(q, at, step, skip);
      if (FULL) sg.copy(q, at, step, skip);
      --uncopied;
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(base + s * stage);
  Pair coef[8], wpre[8];  // out_scale times the post gain and a channel gate
  if (HASY) gains(q, p.w_post, p.gate_ch, p.beta, coef);
  if (PRE) gains(q, p.w_pre, nullptr, 1.0f, wpre);
  const Pair alpha = pair(p.alpha, p.alpha);
  T* xo = static_cast<T*>(p.x_out) + (size_t)q.first * p.d;
  T* u = static_cast<T*>(p.u) + (size_t)q.first * p.d;
  uint32_t at = base, last = base + (S - 1) * stage;  // this row's stage, the one before it
  uint32_t t = q.first;
  for (int left = q.count; left > 0; --left, t += q.step) {
    issue(last);
    float r = 1.0f;
    if (HASY && p.gate_tok) r = p.gate_tok[t];
    cp_wait<S - 1>();
    Pair x[8];
#pragma unroll
    for (int v = 0; v < 2; ++v) sx.get(v, at, step, x + 4 * v);
    if (HASY) {
      Pair y[8];
#pragma unroll
      for (int v = 0; v < 2; ++v) sy.get(v, at, step, y + 4 * v);
      if (POST) {
        Pair a = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) a = fma2(y[i], y[i], a);
        float ss[1] = {sum2(a)};
        row_sum<1>(sums, ss);
        r *= rsqrtf(fmaf(ss[0], p.inv_d, p.eps));
      }
      const Pair rr = pair(r, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = mul2(y[i], rr);
      if (FULL) {
        Pair g[4];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          sg.get(v, at, step, g);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[4 * v + i] = mul2(y[4 * v + i], g[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fma2(y[i], coef[i], mul2(x[i], alpha));
      // rounded here: the next norm reads the stream as it is stored
#pragma unroll
      for (int v = 0; v < 2; ++v) store_chunk<T>(xo + q.c[v], q.on[v], x + 4 * v);
      xo += skip;
    }
    if (PRE) {
      Pair a = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) a = fma2(x[i], x[i], a);
      float ss[1] = {sum2(a)};
      row_sum<1>(sums, ss);
      const float r1 = rsqrtf(fmaf(ss[0], p.inv_d, p.eps));
      const Pair rr = pair(r1, r1);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = mul2(mul2(x[i], rr), wpre[i]);
#pragma unroll
      for (int v = 0; v < 2; ++v) store_chunk<T>(u + q.c[v], q.on[v], x + 4 * v);
      u += skip;
    }
    last = at;
    at = at == base + (S - 1) * stage ? base : at + stage;
  }
}

template <typename T, int S, bool HASY, bool POST, bool FULL, bool PRE>
int run_fwd(const NormFwd& p0, cudaStream_t st) {
  static std::atomic<bool> configured[kMaxDevices];
  NormFwd p = p0;
  const NormPlan q = norm_plan(p.T, p.d, S * 16 * planes<T>() * (1 + HASY + FULL), kFwdCtas);
  p.C = q.C;
  p.nt = q.nt;
  return launch_norm(block_norm_fwd<T, S, HASY, POST, FULL, PRE>, configured, p, q, st);
}

template <typename T, int S>
int fwd_of(const NormFwd& p, cudaStream_t st) {
  const bool post = p.w_post, full = p.gate_full, pre = p.w_pre;
  if (!p.y) return run_fwd<T, S, false, false, false, true>(p, st);
  if (post)
    return full ? (pre ? run_fwd<T, S, true, true, true, true>(p, st)
                       : run_fwd<T, S, true, true, true, false>(p, st))
                : (pre ? run_fwd<T, S, true, true, false, true>(p, st)
                       : run_fwd<T, S, true, true, false, false>(p, st));
  return full ? (pre ? run_fwd<T, S, true, false, true, true>(p, st)
                     : run_fwd<T, S, true, false, true, false>(p, st))
              : (pre ? run_fwd<T, S, true, false, false, true>(p, st)
                     : run_fwd<T, S, true, false, false, false>(p, st));
}

}  // namespace
}  // namespace moe

extern "C" int moe_block_norm_fwd(const moe_block_norm* norm, int32_t dtype, const void* x,
                                  const void* y, const float* w_post, const void* gate,
                                  const float* w_pre, void* x_out, void* u, void* stream) {
  using namespace moe;
  if (!norm_ok(norm) || !valid_act_dtype(dtype)) return MOE_ERR_INVALID_ARG;
  const moe_block_norm& b = *norm;
  if (b.T == 0) return MOE_OK;  // empty tensors may have no address
  if ((gate != nullptr) != (b.gate != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
  if (!x || (y && !x_out) || (w_pre && !u) || (!y && !w_pre)) return MOE_ERR_INVALID_ARG;
  // without a block's output there is nothing to norm or gate
  if (!y && (w_post || gate)) return MOE_ERR_INVALID_ARG;
  const void* al[] = {x, y, w_post, w_pre, x_out, u,
                      b.gate == MOE_GATE_TOKEN ? nullptr : gate};
  for (const void* q : al)
    if (!aligned16(q)) return MOE_ERR_INVALID_ARG;
  NormFwd p{};
  p.T = b.T;
  p.d = b.d;
  p.x = x;
  p.y = y;
  p.gate_full = b.gate == MOE_GATE_FULL ? gate : nullptr;
  p.gate_ch = b.gate == MOE_GATE_CHANNEL ? static_cast<const float*>(gate) : nullptr;
  p.gate_tok = b.gate == MOE_GATE_TOKEN ? static_cast<const float*>(gate) : nullptr;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.alpha = b.res_scale;
  p.beta = b.out_scale;
  p.eps = b.eps;
  p.inv_d = 1.0f / (float)b.d;
  p.x_out = x_out;
  p.u = u;
  cudaStream_t st = as_stream(stream);
  if (dtype == MOE_F32) return fwd_of<float, 2>(p, st);
  if (dtype == MOE_BF16) return fwd_of<__nv_bfloat16, 4>(p, st);
  return fwd_of<__half, 4>(p, st);
}
