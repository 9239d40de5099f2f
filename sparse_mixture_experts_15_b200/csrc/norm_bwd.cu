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
// factors are formed again from x' and y, which the row needs anyway.  D comes
// from sums of the inputs as well,
//   sum yh k g dx' = r2 (sum y k g dx_out + r1 (sum y k g w_pre du
//                    - r1^2 B / d sum y k g x')),
// so a row needs one round of sums: one pass over its arrays forms all six, a
// second one the outputs.
//
// Bound by the rows' bytes.  The second pass reads the row's arrays from
// shared memory again, which costs less than the registers to keep them.  The
// sums over the tokens stay in registers for all rows of a team; the teams' and
// then the CTAs' parts are added in order.
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
  int* status;
};

// Six sums over the threads of a row at once.  In a warp a lane hands on half of
// its values at each of three steps, so that lane 4 i ends with value i's sum
// after 9 shuffles instead of 30; the team's warps and then the cluster's CTAs
// are added from shared memory by lanes that each take one value.  Two buffers
// taken in turn: a thread writes a buffer again only after a barrier that every
// reader of its last contents has reached.
struct RowSumMem {
  float warp_part[2][kNormThreads / 32][8];
  float rank_part[2][4][8];
  uint64_t bar[2];
};
struct RowSum6 {
  RowSumMem* m;
  int team, nt, warps, C;  // warps: of this team
  uint32_t uses;
  Exchange cluster;
};
__device__ __forceinline__ void row_sums(RowSum6& r, float* v) {
  const int lane = threadIdx.x & 31;
  const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
  float h[4], a, c;
  h[0] = (b4 ? v[4] : v[0]) + __shfl_xor_sync(0xffffffffu, b4 ? v[0] : v[4], 16);
  h[1] = (b4 ? v[5] : v[1]) + __shfl_xor_sync(0xffffffffu, b4 ? v[1] : v[5], 16);
  h[2] = (b4 ? 0.0f : v[2]) + __shfl_xor_sync(0xffffffffu, b4 ? v[2] : 0.0f, 16);
  h[3] = (b4 ? 0.0f : v[3]) + __shfl_xor_sync(0xffffffffu, b4 ? v[3] : 0.0f, 16);
  a = (b3 ? h[2] : h[0]) + __shfl_xor_sync(0xffffffffu, b3 ? h[0] : h[2], 8);
  c = (b3 ? h[3] : h[1]) + __shfl_xor_sync(0xffffffffu, b3 ? h[1] : h[3], 8);
  a = (b2 ? c : a) + __shfl_xor_sync(0xffffffffu, b2 ? a : c, 4);
  a += __shfl_xor_sync(0xffffffffu, a, 2);
  a += __shfl_xor_sync(0xffffffffu, a, 1);  // the sum of value lane / 4
  int from = 4;                             // lanes between the values
  const int b = r.uses & 1;
  if (r.warps > 1) {
    if ((lane & 3) == 0) r.m->warp_part[b][threadIdx.x >> 5][lane >> 2] = a;
    team_sync(r.team, r.nt);
    const float* p = &r.m->warp_part[b][r.team * r.warps][lane & 7];
    const int w = lane >> 3;
    a = (w < r.warps ? p[8 * w] : 0.0f) + (w + 4 < r.warps ? p[8 * (w + 4)] : 0.0f);
    a += __shfl_xor_sync(0xffffffffu, a, 8);
    a += __shfl_xor_sync(0xffffffffu, a, 16);
    from = 1;
  }
  if (r.C > 1) {  // warps > 1: rows this wide fill their teams
    const int rank = blockIdx.x % r.C;
    if (threadIdx.x == 0) r.cluster.expect(b, 8 * 4 * r.C);
    if (threadIdx.x < 8)
      for (int to = 0; to < r.C; ++to) r.cluster.send(b, &r.m->rank_part[b][rank][lane], to, a);
    r.cluster.wait(b, (r.uses >> 1) & 1);
    a = r.m->rank_part[b][0][lane & 7];
    for (int k = 1; k < r.C; ++k) a += r.m->rank_part[b][k][lane & 7];
  }
#pragma unroll
  for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xffffffffu, a, from * i);
  ++r.uses;
}

enum RowGate { ROW_ONE = 0, ROW_TOKEN = 1, ROW_FULL = 2 };

// HASY: y is read (POST, or a gate's gradient).
template <typename T, typename G, int S, bool PRE, bool HASY, bool POST, int GATE>
__global__ void __launch_bounds__(kNormThreads, kBwdCtas)
    block_norm_bwd(const __grid_constant__ NormBwd p) {
  extern __shared__ __align__(128) char ring_mem[];
  __shared__ RowSumMem sum_mem;
  __shared__ uint64_t full_bar[kMaxTeams][S];
  constexpr bool FULL = GATE == ROW_FULL, TOKEN = GATE == ROW_TOKEN;
  constexpr bool SUMS = PRE || POST || TOKEN;
  constexpr int W = chunk_width<T, G>(), NV = kCols / W, ET = sizeof(T), EG = sizeof(G), H = W / 2;
  constexpr int NT = PRE + HASY + FULL, NG = PRE + 1;  // arrays of T, of G
  const int nt = p.nt;
  const Place q = place_of(nt, p.C, p.d, p.T);
  RowSum6 sums{&sum_mem, q.team, nt, nt / 32, p.C, 0, {smem_addr(sum_mem.bar), true, p.status}};
  if (p.C > 1) sums.cluster.init();
  // a stage: x', y, the full gate, then du, dx_out
  const uint32_t st_t = nt * kCols * ET, st_g = nt * kCols * EG;  // bytes of an array in a stage
  const uint32_t stage = NT * st_t + NG * st_g;
  const uint32_t oy = PRE * st_t, og = oy + HASY * st_t, ou = NT * st_t, od = ou + PRE * st_g;
  const uint32_t ring = smem_addr(ring_mem) + q.team * S * stage;
  const uint32_t bar = smem_addr(full_bar[q.team]);
  const bool leader = q.lane_t == 0, has_d = p.dx_out != nullptr;
  if (leader) {
    for (int s = 0; s < S; ++s) tc::mbar_init(bar + 8 * s, 1);
    tc::fence_barrier_init();
  }
  for (int s = 0; s < S; ++s) {
    for (int k = 0; k < NT; ++k) zero_tail(q, nt, ring + s * stage + k * st_t, ET);
    for (int k = 0; k < NG; ++k) zero_tail(q, nt, ring + s * stage + ou + k * st_g, EG);
  }
  team_sync(q.team, nt);
  if (p.C > 1) cluster_barrier();  // every CTA of the cluster runs before its memory is written
  pdl_wait();
  pdl_allow_next();
  auto issue = [&](uint32_t row, int s) {  // by the leader
    const size_t e = (size_t)row * (uint32_t)p.d + q.begin;
    const uint32_t at = ring + s * stage, bt = q.cols * ET, bg = q.cols * EG, b = bar + 8 * s;
    tc::mbar_arrive_expect_tx(b, NT * bt + (PRE + has_d) * bg);
    if (q.cols == 0) return;
    if (PRE) bulk_copy(at, static_cast<const T*>(p.x_out) + e, bt, b);
    if (HASY) bulk_copy(at + oy, static_cast<const T*>(p.y) + e, bt, b);
    if (FULL) bulk_copy(at + og, static_cast<const T*>(p.gate_full) + e, bt, b);
    if (PRE) bulk_copy(at + ou, static_cast<const G*>(p.du) + e, bg, b);
    if (has_d) bulk_copy(at + od, static_cast<const G*>(p.dx_out) + e, bg, b);
  };
  if (leader)
    for (int s = 0; s < S && s < q.count; ++s) issue(q.first + s * q.step, s);
  Pair coef[8], wpre[8], a_pre[8], a_q[8];
  gains<W>(q, nt, p.w_post, p.gate_ch, p.beta, coef);
  if (PRE) gains<W>(q, nt, p.w_pre, nullptr, 1.0f, wpre);
#pragma unroll
  for (int i = 0; i < 8; ++i) a_pre[i] = a_q[i] = 0;
  const float af = p.branch ? p.alpha : 1.0f;
  const Pair alpha = pair(af, af);
  const uint32_t mt = q.lane_t * W * ET, mg = q.lane_t * W * EG;  // this thread's first chunk
  const uint32_t nx = nt * W * ET, ng = nt * W * EG;              // from a chunk to the next
  uint32_t t = q.first;
  Ring at_row{bar, S, 0, 0, true, 0, 0};
  for (int row = 0; row < q.count; ++row, t += q.step) {
    const float gt = TOKEN ? p.gate_tok[t] : 1.0f;
    at_row.wait(p.status);
    const int s = at_row.s;
    const uint32_t ax = ring + s * stage + mt, ay = ax + oy, ag = ax + og;
    const uint32_t au = ring + s * stage + ou + mg, ad = ring + s * stage + od + mg;
    // pass 1: the sums over the row
    float r1 = 1.0f, r2 = 1.0f, m1 = 0.0f, D = 0.0f;  // D without a token's gate
    if (SUMS) {
      Pair sums6[6] = {0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        Pair x[H], u[H], y[H], d[H];
        if (PRE) {
          get<W, T>(ax + v * nx, x);
          get<W, G>(au + v * ng, u);
        }
        if (HASY) get<W, T>(ay + v * nx, y);
        if (HASY && (POST || TOKEN) && has_d) get<W, G>(ad + v * ng, d);
        if (POST)
#pragma unroll
          for (int i = 0; i < H; ++i) sums6[2] = fma2(y[i], y[i], sums6[2]);
        if (FULL && POST) {
          Pair g[H];
          get<W, T>(ag + v * nx, g);
#pragma unroll
          for (int i = 0; i < H; ++i) y[i] = mul2(y[i], g[i]);
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
          const int k = H * v + i;
          Pair w = 0;
          if (PRE) {
            w = mul2(u[i], wpre[k]);
            sums6[0] = fma2(x[i], x[i], sums6[0]);
            sums6[1] = fma2(x[i], w, sums6[1]);
          }
          if (POST || TOKEN) {
            const Pair z = mul2(y[i], coef[k]);
            if (has_d) sums6[3] = fma2(z, d[i], sums6[3]);
            if (PRE) {
              sums6[4] = fma2(z, w, sums6[4]);
              sums6[5] = fma2(z, x[i], sums6[5]);
            }
          }
        }
      }
      float s6[6];
#pragma unroll
      for (int i = 0; i < 6; ++i) s6[i] = sum2(sums6[i]);
      row_sums(sums, s6);
      if (PRE) {
        r1 = rsqrtf(fmaf(s6[0], p.inv_d, p.eps));
        m1 = -s6[1] * p.inv_d * r1 * r1;
      }
      if (POST) r2 = rsqrtf(fmaf(s6[2], p.inv_d, p.eps));
      D = fmaf(r1, fmaf(m1, s6[5], s6[4]), s6[3]) * r2;
    } else {
      team_sync(q.team, nt);
    }
    // every thread of the team is past the row before this one: its stage is free
    if (nt == 32) __syncwarp();
    if (leader && at_row.ok && row > 0 && row - 1 + S < q.count)
      issue(t + (S - 1) * q.step, s == 0 ? S - 1 : s - 1);
    if (TOKEN && q.begin + q.lane_t == 0) p.dgate_tok[t] = D;
    // pass 2: the outputs
    const float my = POST ? -D * gt * p.inv_d * r2 * r2 : 0.0f;
    const Pair rr1 = pair(r1, r1), mm1 = pair(m1, m1), rr2 = pair(r2, r2), mm2 = pair(my, my);
    const size_t e = (size_t)t * (uint32_t)p.d + q.begin + q.lane_t * W;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const bool on = (v * nt + q.lane_t) * W < q.cols;
      const size_t ev = e + v * nt * W;
      Pair dv[H], y[H], z[H];
      if (has_d) {
        get<W, G>(ad + v * ng, dv);
      } else {
#pragma unroll
        for (int i = 0; i < H; ++i) dv[i] = 0;
      }
      if (PRE) {
        Pair x[H], u[H];
        get<W, T>(ax + v * nx, x);
        get<W, G>(au + v * ng, u);
#pragma unroll
        for (int i = 0; i < H; ++i) {
          const int k = H * v + i;
          dv[i] = fma2(fma2(x[i], mm1, mul2(wpre[k], u[i])), rr1, dv[i]);
          a_pre[k] = fma2(u[i], mul2(x[i], rr1), a_pre[k]);
        }
      }
#pragma unroll
      for (int i = 0; i < H; ++i) z[i] = mul2(dv[i], alpha);
      put<W>(static_cast<G*>(p.dx) + ev, on, z);
      if (!p.branch) continue;
      if (HASY) {
        get<W, T>(ay + v * nx, y);
        if (FULL) {
          Pair g[H];
          get<W, T>(ag + v * nx, g);
#pragma unroll
          for (int i = 0; i < H; ++i) {
            z[i] = mul2(mul2(coef[H * v + i], dv[i]), mul2(y[i], rr2));
            dv[i] = mul2(dv[i], g[i]);
          }
          put<W>(static_cast<T*>(p.dgate_full) + ev, on, z);
        } else if (TOKEN) {
#pragma unroll
          for (int i = 0; i < H; ++i) dv[i] = mul2(dv[i], pair(gt, gt));
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
          const int k = H * v + i;
          a_q[k] = fma2(dv[i], POST ? mul2(y[i], rr2) : y[i], a_q[k]);
          z[i] = mul2(dv[i], coef[k]);
          if (POST) z[i] = fma2(z[i], rr2, mul2(y[i], mm2));
        }
      } else {
#pragma unroll
        for (int i = 0; i < H; ++i) z[i] = mul2(dv[i], coef[H * v + i]);
      }
      put<W>(static_cast<T*>(p.dy) + ev, on, z);
    }
    at_row.next();
  }
  if (leader) at_row.drain();
  if (p.C > 1) cluster_barrier();  // no CTA leaves while another may write to it
  // The CTA's teams add their columns' sums in team order, through the ring's
  // memory: every copy into it has been waited for.
  const int teams = blockDim.x / nt;
  Pair* mem = reinterpret_cast<Pair*>(ring_mem);
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
            a[i] = fma2(mem[i * blockDim.x + m * nt + q.lane_t], pair(1.0f, 1.0f), a[i]);
    }
    if (q.team == 0)
#pragma unroll
      for (int v = 0; v < NV; ++v)
        put<W>(out + (size_t)(blockIdx.x / p.C) * p.d + q.begin + (v * nt + q.lane_t) * W,
               (v * nt + q.lane_t) * W < q.cols, a + H * v);
  }
}

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

// Stages of the ring: three where they leave room for two CTAs per SM, else two.
// Two stages of wide elements still fit only one CTA per SM, whose waits nothing
// covers (8192 x 4096 with fp32 stream gradients: bf16 with a channel gate 101 us, the
// bytes 92; bf16 with a full gate 173 and 113, fp32 175 and 123, fp32 with a full
// gate 229 and 164).
template <typename T, typename G, bool PRE, bool HASY, bool POST, int GATE>
int run_bwd(const NormBwd& p0, const moe_block_norm_grads& g, float* parts, cudaStream_t st) {
  static NormSetup setup;
  constexpr int row =
      kCols * ((int)sizeof(T) * (PRE + HASY + (GATE == ROW_FULL)) + (int)sizeof(G) * (PRE + 1));
  constexpr int S = 3 * row * kNormThreads * kBwdCtas <= kNormSmem ? 3 : 2;
  NormBwd p = p0;
  NormPlan q = norm_plan(p.T, p.d, S * row, kBwdCtas);
  if (q.grid > kBwdParts * q.C) q.grid = kBwdParts * q.C;
  const auto kernel = block_norm_bwd<T, G, S, PRE, HASY, POST, GATE>;
  int rc = prepare_norm(kernel, setup, q);
  if (rc != MOE_OK) return rc;
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
  rc = launch_norm(kernel, p, q, st);
  if (rc != MOE_OK || (!s.dw_pre && !q_sum)) return rc;
  MOE_PREFER_SHARED((block_norm_sums));
  launch_pdl(block_norm_sums, dim3((p.d + 31) / 32, q_sum ? 2 : 1), dim3(1024), 0, st, s);
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
  p.status = status_word();
  float* parts = static_cast<float*>(ws);
  if (dtype == MOE_F32) return bwd_of<float, float>(p, g, parts, st);
  if (dtype == MOE_BF16)
    return grad_dtype == MOE_F32 ? bwd_of<__nv_bfloat16, float>(p, g, parts, st)
                                 : bwd_of<__nv_bfloat16, __nv_bfloat16>(p, g, parts, st);
  return grad_dtype == MOE_F32 ? bwd_of<__half, float>(p, g, parts, st)
                               : bwd_of<__half, __half>(p, g, parts, st);
}
