// Gradients of the block norms (norm.cu).  With A = sum x'^2, B = sum x' w_pre du
// and r1 = 1 / sqrt(A/d + eps):
//   dx' = dx_out + r1 (w_pre du - x' r1^2 B / d)         dx = res_scale dx'
//   dw_pre = sum_t du x' r1
// and with yh = y r2, k = out_scale w_post gate_ch, g the row's own gate (a
// token's or the full one, else 1), D = sum yh k g dx':
//   dy = r2 (k g dx' - yh D / d)          Q = sum_t g dx' yh
//   dw_post = out_scale gate_ch Q         dgate_ch = out_scale w_post Q
//   dgate_tok = sum yh k dx'              dgate_full = yh k dx'
// so two sums over the tokens carry all three gains' gradients.  The norms'
// factors are formed again from x' and y, which the row needs anyway.
//
// Bound by the rows' bytes.  A row's arrays are read from the FIFO again for
// each of the passes that need them, which costs less than the registers to
// keep them.  The sums over the tokens stay in registers for all rows of a
// team; the teams' and then the CTAs' parts are added in order.
#include "norm.cuh"

namespace moe {
namespace {

constexpr int kBwdCtas = 2;                 // CTAs per SM
constexpr int kBwdParts = 148 * kBwdCtas;   // CTAs (clusters), at most

struct NormBwd {
  int T, d, C, nt;
  const void *x_out, *y, *gate_full, *dx_out, *du;
  const float *w_post, *w_pre, *gate_ch, *gate_tok;
  int branch;
  float alpha, beta, eps, inv_d;
  void *dx, *dy, *dgate_full;
  float* dgate_tok;
  float *part_pre, *part_q;  // [parts][d], nullable
};

enum RowGate { ROW_ONE = 0, ROW_TOKEN = 1, ROW_FULL = 2 };

// HASY: y is read (POST, or a gate's gradient).
template <typename T, typename G, int S, bool PRE, bool HASY, bool POST, int GATE>
__global__ void __launch_bounds__(kNormThreads, kBwdCtas)
    block_norm_bwd(const __grid_constant__ NormBwd p) {
  extern __shared__ __align__(16) char fifo_mem[];
  __shared__ SumBuffers sum_mem;
  pdl_wait();
  pdl_allow_next();
  const Place q = place_of(p.nt, p.C, p.d, p.T);
  RowSum sums{&sum_mem, q.team, p.nt, p.nt / 32, p.C, 0};
  if (p.C > 1) cluster_barrier();  // every CTA of the cluster runs before its memory is written
  constexpr bool FULL = GATE == ROW_FULL, TOKEN = GATE == ROW_TOKEN;
  constexpr int P = planes<T>(), PG = planes<G>();
  constexpr int ay = P * PRE, ag = ay + P * HASY, au = ag + P * FULL, ad = au + PG * PRE;
  const bool has_d = p.dx_out != nullptr;
  const uint32_t step = blockDim.x * 16, stage = (ad + PG) * step;
  const uint32_t base = smem_addr(fifo_mem + threadIdx.x * 16);
  const size_t skip = (size_t)q.step * p.d;
  Stream<T> sx, sy, sg;
  Stream<G> su, sd;
  if (PRE) sx.start(p.x_out, q, p.d, 0);
  if (HASY) sy.start(p.y, q, p.d, ay);
  if (FULL) sg.start(p.gate_full, q, p.d, ag);
  if (PRE) su.start(p.du, q, p.d, au);
  sd.start(p.dx_out, q, p.d, ad);
  int uncopied = q.count;
  auto issue = [&](uint32_t at) {
    if (uncopied > 0) {
      if (PRE) sx.copy(q, at, step, skip);
      if (HASY) sy.copy(q, at, step, skip);
      if (FULL) sg.copy(q, at, step, skip);
      if (PRE) su.copy(q, at, step, skip);
      if (has_d) sd.copy(q, at, step, skip);
      --uncopied;
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(base + s * stage);
  Pair coef[8], wpre[8], a_pre[8], a_q[8];
  gains(q, p.w_post, p.gate_ch, p.beta, coef);
  if (PRE) gains(q, p.w_pre, nullptr, 1.0f, wpre);
#pragma unroll
  for (int i = 0; i < 8; ++i) a_pre[i] = a_q[i] = 0;
  const float af = p.branch ? p.alpha : 1.0f;
  const Pair alpha = pair(af, af);
  G* dx = static_cast<G*>(p.dx) + (size_t)q.first * p.d;
  T* dy = static_cast<T*>(p.dy) + (size_t)q.first * p.d;
  T* dg = static_cast<T*>(p.dgate_full) + (size_t)q.first * p.d;
  uint32_t at = base, last = base + (S - 1) * stage;  // this row's stage, the one before it
  uint32_t t = q.first;
  for (int left = q.count; left > 0; --left, t += q.step) {
    issue(last);
    const float gt = TOKEN ? p.gate_tok[t] : 1.0f;
    cp_wait<S - 1>();
    float s3[3] = {0.0f, 0.0f, 0.0f};
    {
      Pair sa = 0, sb = 0, sc = 0;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        Pair x[4], u[4];
        if (PRE) {
          sx.get(v, at, step, x);
          su.get(v, at, step, u);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sa = fma2(x[i], x[i], sa);
            sb = fma2(mul2(x[i], wpre[4 * v + i]), u[i], sb);
          }
        }
        if (POST) {
          sy.get(v, at, step, x);
#pragma unroll
          for (int i = 0; i < 4; ++i) sc = fma2(x[i], x[i], sc);
        }
      }
      s3[0] = sum2(sc), s3[1] = sum2(sa), s3[2] = sum2(sb);
    }
    if (PRE) row_sum<3>(sums, s3);
    else if (POST) row_sum<1>(sums, s3);
    Pair dv[8];
    if (has_d) {
#pragma unroll
      for (int v = 0; v < 2; ++v) sd.get(v, at, step, dv + 4 * v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) dv[i] = 0;
    }
    if (PRE) {
      const float r1 = rsqrtf(fmaf(s3[1], p.inv_d, p.eps)), m = -s3[2] * p.inv_d * r1 * r1;
      const Pair rr = pair(r1, r1), mm = pair(m, m);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        Pair x[4], u[4];
        sx.get(v, at, step, x);
        su.get(v, at, step, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = 4 * v + i;
          dv[k] = fma2(fma2(x[i], mm, mul2(wpre[k], u[i])), rr, dv[k]);
          a_pre[k] = fma2(u[i], mul2(x[i], rr), a_pre[k]);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      Pair z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = mul2(dv[4 * v + i], alpha);
      store_chunk<G>(dx + q.c[v], q.on[v], z);
    }
    dx += skip;
    if (p.branch) {
      const float r2 = POST ? rsqrtf(fmaf(s3[0], p.inv_d, p.eps)) : 1.0f;
      const Pair rr = pair(r2, r2);
      Pair sum = 0;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        Pair y[4], g[4];
        if (HASY) {
          sy.get(v, at, step, y);
          if (POST)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], rr);
        }
        if (FULL) {
          sg.get(v, at, step, g);
          Pair z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            z[i] = mul2(mul2(coef[4 * v + i], dv[4 * v + i]), y[i]);
            dv[4 * v + i] = mul2(dv[4 * v + i], g[i]);
          }
          store_chunk<T>(dg + q.c[v], q.on[v], z);
        }
        // dv becomes k g dx', but for a token's gate, which comes in below
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = 4 * v + i;
          if (HASY) a_q[k] = fma2(TOKEN ? mul2(dv[k], pair(gt, gt)) : dv[k], y[i], a_q[k]);
          dv[k] = mul2(dv[k], coef[k]);
          if (HASY) sum = fma2(dv[k], y[i], sum);
        }
      }
      dg += skip;
      float m = 0.0f;
      if (POST || TOKEN) {
        float s1[1] = {sum2(sum)};
        row_sum<1>(sums, s1);
        if (TOKEN && q.lane_t == 0 && (p.C == 1 || blockIdx.x % p.C == 0)) p.dgate_tok[t] = s1[0];
        m = -s1[0] * gt * p.inv_d * r2 * r2;
      }
      const float ro = r2 * gt;
      const Pair mm = pair(m, m), rg = pair(ro, ro);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        Pair y[4];
        if (POST) sy.get(v, at, step, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = 4 * v + i;
          if (POST || TOKEN) dv[k] = mul2(dv[k], rg);
          if (POST) dv[k] = fma2(y[i], mm, dv[k]);
        }
        store_chunk<T>(dy + q.c[v], q.on[v], dv + 4 * v);
      }
      dy += skip;
    }
    last = at;
    at = at == base + (S - 1) * stage ? base : at + stage;
  }
  // The CTA's teams add their columns' sums in team order, through the FIFO's
  // memory once every copy into it has landed.
  cp_wait<0>();
  const int teams = blockDim.x / p.nt;
  Pair* mem = reinterpret_cast<Pair*>(fifo_mem);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float* out = k == 0 ? p.part_pre : p.part_q;
    Pair* a = k == 0 ? a_pre : a_q;
    if (!out) continue;
    if (teams > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) mem[i * blockDim.x + threadIdx.x] = a[i];
      __syncthreads();
      if (q.team == 0)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          for (int m = 1; m < teams; ++m)
            a[i] = fma2(mem[i * blockDim.x + m * p.nt + q.lane_t], pair(1.0f, 1.0f), a[i]);
    }
    if (q.team == 0)
#pragma unroll
      for (int v = 0; v < 2; ++v)
        store_chunk<float>(out + (size_t)(blockIdx.x / p.C) * p.d + q.c[v], q.on[v], a + 4 * v);
  }
}

// The gains' gradients from the parts: 32 columns for a block, 8 runs of parts
// summed at once and the runs then in order.
struct NormSums {
  int parts, d;
  const float *part_pre, *part_q, *w_post, *gate_ch;
  float beta;
  float *dw_pre, *dw_post, *dgate_ch;
};
__global__ void __launch_bounds__(256) block_norm_sums(const __grid_constant__ NormSums p) {
  pdl_wait();
  pdl_allow_next();
  __shared__ float run[8][32];
  const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, r = threadIdx.x >> 5;
  const float* src = blockIdx.y == 0 ? p.part_pre : p.part_q;
  if (!src) return;
  float a = 0.0f;
  if (c < p.d) {
    src += c;
#pragma unroll 8
    for (int i = r; i < p.parts; i += 8) a += src[(size_t)i * p.d];
  }
  run[r][lane] = a;
  __syncthreads();
  if (r == 0 && c < p.d) {
#pragma unroll
    for (int i = 1; i < 8; ++i) a += run[i][lane];
    if (blockIdx.y == 0) {
      p.dw_pre[c] = a;
    } else {
      if (p.dw_post) p.dw_post[c] = p.beta * (p.gate_ch ? p.gate_ch[c] : 1.0f) * a;
      if (p.dgate_ch) p.dgate_ch[c] = p.beta * (p.w_post ? p.w_post[c] : 1.0f) * a;
    }
  }
}

// Stages of the FIFO: as many as leave room for two CTAs per SM, 2 or 3.
template <typename T, typename G, bool PRE, bool HASY, bool POST, int GATE>
int run_bwd(const NormBwd& p0, const moe_block_norm_grads& g, float* parts, cudaStream_t st) {
  static std::atomic<bool> configured[kMaxDevices];
  constexpr int row = 16 * (planes<T>() * (PRE + HASY + (GATE == ROW_FULL)) + planes<G>() * (PRE + 1));
  constexpr int S = 3 * row * kNormThreads * kBwdCtas <= kNormSmem ? 3 : 2;
  NormBwd p = p0;
  NormPlan q = norm_plan(p.T, p.d, S * row, kBwdCtas);
  if (q.grid > kBwdParts * q.C) q.grid = kBwdParts * q.C;
  p.C = q.C;
  p.nt = q.nt;
  NormSums s{};
  s.parts = q.grid / q.C;
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
  const int rc =
      launch_norm(block_norm_bwd<T, G, S, PRE, HASY, POST, GATE>, configured, p, q, st);
  if (rc != MOE_OK || (!s.dw_pre && !q_sum)) return rc;
  MOE_PREFER_SHARED((block_norm_sums));
  launch_pdl(block_norm_sums, dim3((p.d + 31) / 32, q_sum ? 2 : 1), dim3(256), 0, st, s);
  return launch_status();
}

template <typename T, typename G, bool PRE>
int bwd_gate(const NormBwd& p, const moe_block_norm_grads& g, float* parts, cudaStream_t st) {
  if (p.w_post)
    return p.gate_full  ? run_bwd<T, G, PRE, true, true, ROW_FULL>(p, g, parts, st)
           : p.gate_tok ? run_bwd<T, G, PRE, true, true, ROW_TOKEN>(p, g, parts, st)
                        : run_bwd<T, G, PRE, true, true, ROW_ONE>(p, g, parts, st);
  return p.gate_full  ? run_bwd<T, G, PRE, true, false, ROW_FULL>(p, g, parts, st)
         : p.gate_tok ? run_bwd<T, G, PRE, true, false, ROW_TOKEN>(p, g, parts, st)
         : p.gate_ch  ? run_bwd<T, G, PRE, true, false, ROW_ONE>(p, g, parts, st)
                      : run_bwd<T, G, PRE, false, false, ROW_ONE>(p, g, parts, st);
}

template <typename T, typename G>
int bwd_of(const NormBwd& p, const moe_block_norm_grads& g, float* parts, cudaStream_t st) {
  return p.w_pre ? bwd_gate<T, G, true>(p, g, parts, st)
                 : bwd_gate<T, G, false>(p, g, parts, st);
}

}  // namespace
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
  float* parts = static_cast<float*>(ws);
  if (dtype == MOE_F32) return bwd_of<float, float>(p, g, parts, st);
  if (dtype == MOE_BF16)
    return grad_dtype == MOE_F32 ? bwd_of<__nv_bfloat16, float>(p, g, parts, st)
                                 : bwd_of<__nv_bfloat16, __nv_bfloat16>(p, g, parts, st);
  return grad_dtype == MOE_F32 ? bwd_of<__half, float>(p, g, parts, st)
                               : bwd_of<__half, __half>(p, g, parts, st);
}
