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
#pragma once

#include "norm.cuh"

namespace moe {

constexpr int kBwdParts = 148 * (kSmThreads / kNormThreads);  // CTAs (clusters), at most

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

// Bytes of a thread's columns in a stage of the ring, and whether two stages of
// a CTA of `threads` have room (512 threads: not with fp32 data, nor with a full
// gate of 16 bits next to fp32 gradients).
constexpr int bwd_row_bytes(size_t t, size_t g, bool pre, bool has_y, bool full) {
  return kCols * (int)(t * (pre + has_y + full) + g * (pre + 1));
}
constexpr bool bwd_fits(int row, int threads) { return 2 * row * threads <= kNormSmem; }

// The kernel's instances for CTAs of 256 and of 512 threads, each in a
// translation unit of its own.  parts: how many parts the sums over the tokens
// are in.
int block_norm_bwd_256(NormBwd p, int dtype, int grad_dtype, int* parts, cudaStream_t st);
int block_norm_bwd_512(NormBwd p, int dtype, int grad_dtype, int* parts, cudaStream_t st);

namespace {

// Six sums over the threads of a row at once.  In a warp a lane hands on half of
// its values at each of three steps, so that lane 4 i ends with value i's sum
// after 9 shuffles instead of 30; the team's warps and then the cluster's CTAs
// are added from shared memory by lanes that each take one value.  Two buffers
// taken in turn: a thread writes a buffer again only after a barrier that every
// reader of its last contents has reached.
struct RowSumMem {
  float warp_part[2][kWideThreads / 32][8];
  float rank_part[2][4][8];
  uint64_t bar[2];
};
struct RowSum6 {
  RowSumMem* m;
  int team, nt, warps, C;  // warps: of this team
  uint32_t uses;
  Exchange cluster;
};
template <int THREADS>
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
    if (THREADS > 256)
      a += (w + 8 < r.warps ? p[8 * (w + 8)] : 0.0f) + (w + 12 < r.warps ? p[8 * (w + 12)] : 0.0f);
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
template <typename T, typename G, int THREADS, int S, bool PRE, bool HASY, bool POST, int GATE>
__global__ void __launch_bounds__(THREADS, kSmThreads / THREADS)
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
      row_sums<THREADS>(sums, s6);
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

// Stages of the ring: as many as leave room for an SM's threads, 2 or 3.
template <int THREADS, typename T, typename G, bool PRE, bool HASY, bool POST, int GATE>
int run_bwd(NormBwd p, int* parts, cudaStream_t st) {
  constexpr int row = bwd_row_bytes(sizeof(T), sizeof(G), PRE, HASY, GATE == ROW_FULL);
  constexpr int S = 3 * row * kSmThreads <= kNormSmem ? 3 : 2;
  if constexpr (bwd_fits(row, THREADS)) {
    static std::atomic<bool> configured[kMaxDevices];
    NormPlan q = norm_plan(p.T, p.d, S * row, THREADS);
    if (q.grid > kBwdParts * q.C) q.grid = kBwdParts * q.C;
    p.C = q.C;
    p.nt = q.nt;
    *parts = q.grid / q.C;
    return launch_norm(block_norm_bwd<T, G, THREADS, S, PRE, HASY, POST, GATE>, configured, p, q,
                       st);
  }
  return MOE_ERR_UNSUPPORTED;  // the entry asks for no such instance
}

template <int THREADS, typename T, typename G, bool PRE>
int bwd_gate(const NormBwd& p, int* parts, cudaStream_t st) {
  if (p.w_post)
    return p.gate_full  ? run_bwd<THREADS, T, G, PRE, true, true, ROW_FULL>(p, parts, st)
           : p.gate_tok ? run_bwd<THREADS, T, G, PRE, true, true, ROW_TOKEN>(p, parts, st)
                        : run_bwd<THREADS, T, G, PRE, true, true, ROW_ONE>(p, parts, st);
  return p.gate_full  ? run_bwd<THREADS, T, G, PRE, true, false, ROW_FULL>(p, parts, st)
         : p.gate_tok ? run_bwd<THREADS, T, G, PRE, true, false, ROW_TOKEN>(p, parts, st)
         : p.gate_ch  ? run_bwd<THREADS, T, G, PRE, true, false, ROW_ONE>(p, parts, st)
                      : run_bwd<THREADS, T, G, PRE, false, false, ROW_ONE>(p, parts, st);
}

template <int THREADS, typename T, typename G>
int bwd_of(const NormBwd& p, int* parts, cudaStream_t st) {
  return p.w_pre ? bwd_gate<THREADS, T, G, true>(p, parts, st)
                 : bwd_gate<THREADS, T, G, false>(p, parts, st);
}

template <int THREADS>
int bwd_typed(const NormBwd& p, int dtype, int grad_dtype, int* parts, cudaStream_t st) {
  if (dtype == MOE_F32) return bwd_of<THREADS, float, float>(p, parts, st);
  if (dtype == MOE_BF16)
    return grad_dtype == MOE_F32 ? bwd_of<THREADS, __nv_bfloat16, float>(p, parts, st)
                                 : bwd_of<THREADS, __nv_bfloat16, __nv_bfloat16>(p, parts, st);
  return grad_dtype == MOE_F32 ? bwd_of<THREADS, __half, float>(p, parts, st)
                               : bwd_of<THREADS, __half, __half>(p, parts, st);
}

}  // namespace
}  // namespace moe
