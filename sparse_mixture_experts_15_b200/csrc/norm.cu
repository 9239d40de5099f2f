// The norms around a block of the residual stream, with the block's gate and
// the residual scale, in one pass over the rows:
//   n  = y / sqrt(mean(y^2) + eps) * w_post      (w_post NULL: n = y)
//   x' = res_scale x + out_scale gate n          rounded to the storage type
//   u  = x' / sqrt(mean(x'^2) + eps) * w_pre     of x' as stored
// Sums over a row are fp32 in a fixed order.  Bound by the rows' bytes.
#include "norm.cuh"

namespace moe {
namespace {

// CTAs per SM (three, of 80 registers a thread, spill and take 59 us where two
// take 45: 8192 x 4096 bf16, both norms)
constexpr int kFwdCtas = 2;

// Stages of a team's ring.  More of them let the reads run ahead of the stores,
// and the memory serves the two worse: 16384 x 4096 bf16, both norms, 83.4 us, with
// four stages 96.4 (the pre norm alone 82.3 and 90.9; 2048 rows 13.8 and 14.1, the
// pre norm alone 12.8 and 12.3).  A row's stage is filled again once the first
// sum's barrier shows that its threads have read it (at the row's end: 86.4).
constexpr int kFwdStages = 2;

struct NormFwd {
  int T, d, C;             // C: CTAs of a cluster, each with its share of a row's columns
  int nt;                  // threads per row in a CTA
  const void *x, *y, *gate_full;
  const float *w_post, *w_pre, *gate_ch, *gate_tok;
  float alpha, beta, eps, inv_d;
  void *x_out, *u;
  int* status;
};

// A sum over the threads of a row: lanes by a shuffle tree, the team's warps from
// shared memory in a fixed order, then the CTAs of the cluster in rank order through
// distributed shared memory.  Two buffers taken in turn: a thread writes a buffer
// again only after a barrier that every reader of its last contents has reached.
struct RowSumMem {
  // by team, whose warps' parts are padded with zeros to a multiple of four: at
  // most four teams of two warps, two of three or four, one of more
  float4 warp_part[2][4];
  float rank_part[2][4];
  uint64_t bar[2];
};
struct RowSum {
  RowSumMem* m;
  int team, nt, warps, C;  // warps: of this team
  uint32_t uses;
  Exchange cluster;
};
__device__ __forceinline__ float row_sum(RowSum& r, float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int b = r.uses & 1;
  if (r.warps > 1) {
    const float4* p = &r.m->warp_part[b][r.team];
    if ((threadIdx.x & 31) == 0)
      reinterpret_cast<float*>(r.m->warp_part[b] + r.team)[(threadIdx.x >> 5) - r.team * r.warps] = v;
    team_sync(r.team, r.nt);
    const float4 a = p[0];
    v = (a.x + a.y) + (a.z + a.w);
    if (r.warps > 4) {
      const float4 c = p[1];
      v += (c.x + c.y) + (c.z + c.w);
    }
  }
  if (r.C > 1) {  // warps > 1: rows this wide fill their teams
    if (threadIdx.x == 0) r.cluster.expect(b, 4 * r.C);
    if ((int)threadIdx.x < r.C)
      r.cluster.send(b, &r.m->rank_part[b][blockIdx.x % r.C], threadIdx.x, v);
    r.cluster.wait(b, (r.uses >> 1) & 1);
    v = r.m->rank_part[b][0];
    for (int c = 1; c < r.C; ++c) v += r.m->rank_part[b][c];
  }
  ++r.uses;
  return v;
}

// HASY: a block's output comes in (POST: normed first; FULL: gated by element;
// a channel's gate is part of coef, a token's of the row's factor).
template <typename T, bool HASY, bool POST, bool FULL, bool PRE>
__global__ void __launch_bounds__(kNormThreads, kFwdCtas)
    block_norm_fwd(const __grid_constant__ NormFwd p) {
  constexpr int S = kFwdStages;
  extern __shared__ __align__(128) char ring_mem[];
  __shared__ RowSumMem sum_mem;
  __shared__ uint64_t full_bar[kMaxTeams][S];
  constexpr int W = chunk_width<T, T>(), NV = kCols / W, E = sizeof(T), A = 1 + HASY + FULL;
  const int nt = p.nt;
  const Place q = place_of(nt, p.C, p.d, p.T);
  RowSum sums{&sum_mem, q.team, nt, nt / 32, p.C, 0, {smem_addr(sum_mem.bar), true, p.status}};
  if (p.C > 1) sums.cluster.init();
  const uint32_t slot = nt * kCols * E;  // bytes of an array in a stage
  const uint32_t ring = smem_addr(ring_mem) + q.team * S * A * slot;
  const uint32_t bar = smem_addr(full_bar[q.team]);
  const bool leader = q.lane_t == 0;
  if (threadIdx.x < 8) sum_mem.warp_part[threadIdx.x >> 2][threadIdx.x & 3] = make_float4(0, 0, 0, 0);
  __syncthreads();
  if (leader) {
    for (int s = 0; s < S; ++s) tc::mbar_init(bar + 8 * s, 1);
    tc::fence_barrier_init();
  }
  for (int s = 0; s < S * A; ++s) zero_tail(q, nt, ring + s * slot, E);
  team_sync(q.team, nt);
  if (p.C > 1) cluster_barrier();  // every CTA of the cluster runs before its memory is written
  pdl_wait();
  pdl_allow_next();
  auto issue = [&](uint32_t row, int s) {  // by the leader
    const size_t e = (size_t)row * (uint32_t)p.d + q.begin;
    const uint32_t at = ring + s * A * slot, bytes = q.cols * E;
    tc::mbar_arrive_expect_tx(bar + 8 * s, A * bytes);
    if (bytes == 0) return;
    bulk_copy(at, static_cast<const T*>(p.x) + e, bytes, bar + 8 * s);
    if (HASY) bulk_copy(at + slot, static_cast<const T*>(p.y) + e, bytes, bar + 8 * s);
    if (FULL)
      bulk_copy(at + 2 * slot, static_cast<const T*>(p.gate_full) + e, bytes, bar + 8 * s);
  };
  if (leader)
    for (int s = 0; s < S && s < q.count; ++s) issue(q.first + s * q.step, s);
  Pair coef[8], wpre[8];  // out_scale times the post gain and a channel gate
  if (HASY) gains<W>(q, nt, p.w_post, p.gate_ch, p.beta, coef);
  if (PRE) gains<W>(q, nt, p.w_pre, nullptr, 1.0f, wpre);
  const Pair alpha = pair(p.alpha, p.alpha);
  const uint32_t mine = q.lane_t * W * E, next = nt * W * E;  // this thread's first chunk, its step
  uint32_t t = q.first;
  Ring at_row{bar, S, 0, 0, true, 0, 0};
  // the row S on into the stage of row i, which every thread of the team has read:
  // it has passed a barrier since
  auto refill = [&](int i, uint32_t t, int s) {
    if (nt == 32) __syncwarp();
    if (leader && at_row.ok && i + S < q.count) issue(t + S * q.step, s);
  };
  for (int i = 0; i < q.count; ++i, t += q.step) {
    float r = 1.0f;
    if (HASY && p.gate_tok) r = p.gate_tok[t];
    at_row.wait(p.status);
    const int s = at_row.s;
    const uint32_t at = ring + s * A * slot + mine;
    Pair x[8], y[8], g[8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      get<W, T>(at + v * next, x + v * W / 2);
      if (HASY) get<W, T>(at + slot + v * next, y + v * W / 2);
      if (FULL) get<W, T>(at + 2 * slot + v * next, g + v * W / 2);
    }
    const size_t e = (size_t)t * (uint32_t)p.d + q.begin + q.lane_t * W;
    if (HASY) {
      if (POST) {
        Pair a = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) a = fma2(y[k], y[k], a);
        r *= rsqrtf(fmaf(row_sum(sums, sum2(a)), p.inv_d, p.eps));
        refill(i, t, s);
      }
      const Pair rr = pair(r, r);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        y[k] = mul2(y[k], rr);
        if (FULL) y[k] = mul2(y[k], g[k]);
        x[k] = fma2(y[k], coef[k], mul2(x[k], alpha));
      }
      // rounded here: the next norm reads the stream as it is stored
#pragma unroll
      for (int v = 0; v < NV; ++v)
        put<W>(static_cast<T*>(p.x_out) + e + v * nt * W, (v * nt + q.lane_t) * W < q.cols,
               x + v * W / 2);
    }
    if (PRE) {
      Pair a = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) a = fma2(x[k], x[k], a);
      const float r1 = rsqrtf(fmaf(row_sum(sums, sum2(a)), p.inv_d, p.eps));
      const Pair rr = pair(r1, r1);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = mul2(mul2(x[k], rr), wpre[k]);
#pragma unroll
      for (int v = 0; v < NV; ++v)
        put<W>(static_cast<T*>(p.u) + e + v * nt * W, (v * nt + q.lane_t) * W < q.cols,
               x + v * W / 2);
    }
    if (!POST && !PRE) team_sync(q.team, nt);
    if (!POST) refill(i, t, s);
    at_row.next();
  }
  if (leader) at_row.drain();
  if (p.C > 1) cluster_barrier();  // no CTA leaves while another may write to it
}

template <typename T, bool HASY, bool POST, bool FULL, bool PRE>
int run_fwd(const NormFwd& p0, cudaStream_t st) {
  static NormSetup setup;
  constexpr int stage = kCols * (int)sizeof(T) * (1 + HASY + FULL);
  static_assert(kFwdStages * stage * kNormThreads * kFwdCtas <= kNormSmem, "two CTAs per SM");
  NormFwd p = p0;
  NormPlan q = norm_plan(p.T, p.d, kFwdStages * stage, kFwdCtas);
  const auto kernel = block_norm_fwd<T, HASY, POST, FULL, PRE>;
  const int rc = prepare_norm(kernel, setup, q);
  if (rc != MOE_OK) return rc;
  p.C = q.C;
  p.nt = q.nt;
  return launch_norm(kernel, p, q, st);
}

template <typename T>
int fwd_of(const NormFwd& p, cudaStream_t st) {
  const bool post = p.w_post, full = p.gate_full, pre = p.w_pre;
  if (!p.y) return run_fwd<T, false, false, false, true>(p, st);
  if (post)
    return full ? (pre ? run_fwd<T, true, true, true, true>(p, st)
                       : run_fwd<T, true, true, true, false>(p, st))
                : (pre ? run_fwd<T, true, true, false, true>(p, st)
                       : run_fwd<T, true, true, false, false>(p, st));
  return full ? (pre ? run_fwd<T, true, false, true, true>(p, st)
                     : run_fwd<T, true, false, true, false>(p, st))
              : (pre ? run_fwd<T, true, false, false, true>(p, st)
                     : run_fwd<T, true, false, false, false>(p, st));
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
  p.status = status_word();
  cudaStream_t st = as_stream(stream);
  if (dtype == MOE_F32) return fwd_of<float>(p, st);
  if (dtype == MOE_BF16) return fwd_of<__nv_bfloat16>(p, st);
  return fwd_of<__half>(p, st);
}
