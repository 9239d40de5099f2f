// Scored routing: softmax or sigmoid scores of the router's logits, a bias
// that takes part in the selection only, expert groups, top-k and the combine
// weights, and the gradient of the weights and scores to the logits.
//
//   s_j = sigmoid(z_j)  or  exp(z_j - max z) / sum exp(z - max z), to fp32
//   c_j = s_j + b_j                                            (fp32)
//   a group's score = the sum of its group_top largest c; the top_group best
//   groups are kept (ties to the lower group); top_idx = the k largest c
//   of their experts, ties to the lower expert
//   a_i = scale s_i / sum_{selected} s   or   scale s_i
//
// The selection is a decision on the values s_j + b_j, and a score that is off
// by one rounding can turn it.  So s is formed in double, to a relative error
// below 2^-41, and rounded to fp32 once: it is the correctly rounded score but
// for about one in 10^5, which then is off by one rounding.
#include "common.cuh"

namespace moe {
namespace {

constexpr int kSelWarps = 4;  // tokens of a CTA, one warp each

// 1 / x for x >= 1: the approximate instruction and two Newton steps.
__device__ __forceinline__ double recip(double x) {
  double r;
  asm("rcp.approx.ftz.f64 %0, %1;" : "=d"(r) : "d"(x));
  r = fma(r, fma(-x, r, 1.0), r);
  return fma(r, fma(-x, r, 1.0), r);
}

// exp(x) for |x| <= 150: x = n ln 2 + r with |r| <= ln 2 / 2, the Taylor sum of
// exp(r) to r^10 / 10! (the rest is below 2^-42), times 2^n in the exponent.
// n is rounded by adding 1.5 2^52, which leaves it in the low word.  zero: the
// result is 0 (below 2^-1022) whatever x is.
__device__ __forceinline__ double exp_wide(double x, bool zero = false) {
  constexpr double kRound = 6755399441055744.0;
  const double t = fma(x, 1.4426950408889634, kRound);
  const double r = fma(kRound - t, 0.6931471805599453, x);
  double p = 1.0 / 3628800.0;
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return __hiloint2double(zero ? 0 : __double2hiint(p) + (__double2loint(t) << 20),
                          __double2loint(p));
}

// Order of the selection as an unsigned number: larger values first, a NaN
// below every value.  0 is left for what cannot be selected.
__device__ __forceinline__ uint32_t order_of(float c) {
  const uint32_t b = __float_as_uint(c);
  if (c != c) return 1u;
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  if (o <= 1u) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void cp_async16(void* smem, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(smem))),
               "l"(g)
               : "memory");
}

// A lane's experts: chunks of CH consecutive ones, 32 CH apart, so that a warp
// reads and writes whole 16-byte pieces of a row where N allows it.
template <int PER>
struct Lanes {
  static constexpr int CH = PER < 4 ? PER : 4, Q = PER / CH;
  static __device__ __forceinline__ int expert(int lane, int e) {
    return (e / CH) * 32 * CH + lane * CH + e % CH;
  }
  // wide: the row is 16-byte aligned and N a multiple of 4
  static __device__ __forceinline__ void load(const float* row, int N, int lane, float fill,
                                              bool wide, float* v) {
    if (CH == 4 && wide) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int j = expert(lane, q * CH);
        float4 x = make_float4(fill, fill, fill, fill);
        if (j < N) x = *reinterpret_cast<const float4*>(row + j);
        v[4 * q] = x.x, v[4 * q + 1] = x.y, v[4 * q + 2] = x.z, v[4 * q + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const int j = expert(lane, e);
        v[e] = j < N ? row[j] : fill;
      }
    }
  }
  // from a row in shared memory with room for N up to a multiple of 4; 0 past N
  static __device__ __forceinline__ void load_shared(const float* row, int N, int lane, float* v) {
#pragma unroll
    for (int e = 0; e < PER; e += CH) {
      const int j = expert(lane, e);
      if constexpr (CH == 4) {
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (j < N) x = *reinterpret_cast<const float4*>(row + j);
        v[e] = x.x;
        v[e + 1] = j + 1 < N ? x.y : 0.0f;
        v[e + 2] = j + 2 < N ? x.z : 0.0f;
        v[e + 3] = j + 3 < N ? x.w : 0.0f;
      } else {
#pragma unroll
        for (int i = 0; i < CH; ++i) v[e + i] = j + i < N ? row[j + i] : 0.0f;
      }
    }
  }
  static __device__ __forceinline__ void store(float* row, int N, int lane, const float* v) {
    if (CH == 4 && N % 4 == 0) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int j = expert(lane, q * CH);
        if (j < N)
          *reinterpret_cast<float4*>(row + j) =
              make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const int j = expert(lane, e);
        if (j < N) row[j] = v[e];
      }
    }
  }
};

struct SelectParams {
  int T, N, k, renorm, sigmoid, n_group, top_group, group_top;
  int per;        // experts of a group
  int sub_log;    // log2 of the lanes that read one group
  uint32_t inv;   // j / per = j inv >> 20, exact for j < 1024
  int bias_wide;
  float scale;
  const float* logits;
  const float* bias;
  int32_t* top_idx;
  float* top_w;
  float* scores;
};

// One warp per token.
//
// The k best of a token: with m the k-th largest of the 32 lanes' own largest
// orders, every selected expert has an order of m at least, and few others do
// (some 10 of 256 experts for k = 8, 23 of 896 for k = 16).  These are listed in
// shared memory, one for a lane, and each finds its slot by counting those ahead
// of it.  Where more than 32 qualify (ties, k near 32), the k are taken one
// after another instead.
//
// Bound by the issue of its arithmetic for a few hundred experts: of some 990
// instructions a token (256 experts, 8 groups, top-8: 7.0 of the 10.6 us for 8192
// tokens) the scores in double are a quarter.  Selecting on fp32 scores, with
// exact ones where two lie within their error, was no faster (12.9 us): the checks
// cost what the doubles do.  With many experts all warps are resident at once, a
// token each, and load, compute and store in step: of the 14.5 us for 4096 x 896
// the issue is 6.0 and the fp64 pipe 3.2.  From 24 experts a lane on, the launch
// bound's 72 registers make 32 a lane spill (88 bytes); with fewer warps 896
// experts took 15.5 us.
template <int PER>
__global__ void __launch_bounds__(32 * kSelWarps, PER >= 24 ? 7 : 1)
    route_select(const __grid_constant__ SelectParams p) {
  using L = Lanes<PER>;
  extern __shared__ __align__(16) float sel_mem[];  // per warp: scores, orders [N up to 4]
  // (order, inverted expert) as one number: larger is better
  __shared__ unsigned long long listed[kSelWarps][32];
  pdl_wait();
  pdl_allow_next();
  const int lane = threadIdx.x & 31, wib = threadIdx.x >> 5, N = p.N;
  const int64_t t = (int64_t)blockIdx.x * kSelWarps + wib;
  if (t >= p.T) return;
  const int stride = (N + 3) & ~3;
  float* sc = sel_mem + (size_t)wib * 2 * stride;
  uint32_t* od = reinterpret_cast<uint32_t*>(sc + stride);
  float z[PER];
  L::load(p.logits + t * N, N, lane, -INFINITY, N % 4 == 0, z);
  // scores
  if (p.sigmoid) {
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      // beyond 110 the fp32 score no longer changes
      const double x = (double)fminf(fmaxf(-z[e], -110.0f), 110.0f);
      const float s = (float)recip(1.0 + exp_wide(x));
      z[e] = z[e] != z[e] ? z[e] : s;
    }
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int e = 0; e < PER; ++e) m = max_nan(m, z[e]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const double md = (double)m;
    double x[PER], sum = 0.0;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      // 120 below the largest is 0 in fp32, and a logit of -infinity (or a NaN: the
      // row's factor below) with it
      x[e] = exp_wide((double)z[e] - md, !(z[e] - m >= -120.0f));
      sum += x[e];
    }
    sum = warp_sum(sum);
    // NaN for a row that holds a NaN or +infinity, 0 for one of nothing but -infinity
    const double r = m == -INFINITY ? 0.0 : m < INFINITY ? recip(sum) : __hiloint2double(0x7FF80000, 0);
#pragma unroll
    for (int e = 0; e < PER; ++e) z[e] = (float)(x[e] * r);
  }
  if (p.scores) L::store(p.scores + t * N, N, lane, z);
  // the order of the selection, and the scores for the weights
  uint32_t ord[PER];
  float c[PER];
  if (p.bias) L::load(p.bias, N, lane, 0.0f, p.bias_wide, c);
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const int j = L::expert(lane, e);
    ord[e] = j < N ? order_of(p.bias ? z[e] + c[e] : z[e]) : 0u;
  }
#pragma unroll
  for (int e = 0; e < PER; e += L::CH) {
    const int j = L::expert(lane, e);
    if (j >= N) continue;
    if constexpr (L::CH == 4) {
      *reinterpret_cast<float4*>(sc + j) = make_float4(z[e], z[e + 1], z[e + 2], z[e + 3]);
      *reinterpret_cast<uint4*>(od + j) = make_uint4(ord[e], ord[e + 1], ord[e + 2], ord[e + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < L::CH; ++i)
        if (j + i < N) sc[j + i] = z[e + i], od[j + i] = ord[e + i];
    }
  }
  __syncwarp();
  if (p.n_group > 1) {
    // sub lanes of a group read its experts in turn and keep the two best
    const int G = p.n_group, sub = 1 << p.sub_log, g = lane >> p.sub_log;
    uint32_t b1 = 0u, b2 = 0u;
    if (g < G) {
      const uint32_t* og = od + g * p.per;
#pragma unroll 4
      for (int i = lane & (sub - 1); i < p.per; i += sub) {
        const uint32_t o = og[i];
        b2 = max(b2, min(b1, o));
        b1 = max(b1, o);
      }
    }
    for (int o = sub >> 1; o >= 1; o >>= 1) {
      const uint32_t o1 = __shfl_xor_sync(0xffffffffu, b1, o);
      const uint32_t o2 = __shfl_xor_sync(0xffffffffu, b2, o);
      b2 = max(min(b1, o1), max(b2, o2));
      b1 = max(b1, o1);
    }
    const uint32_t mine =
        order_of(p.group_top == 1 ? value_of(b1) : value_of(b1) + value_of(b2));
    int rank = 0;
#pragma unroll 4
    for (int h = 0; h < G; ++h) {
      const uint32_t o = __shfl_sync(0xffffffffu, mine, h << p.sub_log);
      rank += o > mine || (o == mine && h < g);
    }
    const uint32_t kept = __ballot_sync(0xffffffffu, g < G && rank < p.top_group);
    // bit h << sub_log of kept is group h's (an expert past N has the order 0 anyway)
    if (L::CH == 4 && p.per % 4 == 0) {  // a chunk is of one group
#pragma unroll
      for (int e = 0; e < PER; e += 4) {
        const uint32_t h = L::expert(lane, e) * p.inv >> 20;
        const uint32_t all = (kept >> ((h << p.sub_log) & 31u)) & 1u ? 0xFFFFFFFFu : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) ord[e + i] &= all;
      }
    } else {
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const uint32_t h = L::expert(lane, e) * p.inv >> 20;
        if (!((kept >> ((h << p.sub_log) & 31u)) & 1u)) ord[e] = 0u;
      }
    }
  }
  uint32_t best = 0u;
#pragma unroll
  for (int e = 0; e < PER; ++e) best = max(best, ord[e]);
  uint32_t m = best, least = 0u;
  for (int s = 0; s < p.k; ++s) {  // equal ones go together: that only lowers the bound
    least = __reduce_max_sync(0xffffffffu, m);
    if (m == least) m = 0u;
  }
  if (least == 0u) least = 1u;
  uint32_t in = 0u;
#pragma unroll
  for (int e = 0; e < PER; ++e) in |= (uint32_t)(ord[e] >= least) << e;
  const int own = __popc(in);
  int at = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += v;
  }
  const int count = __shfl_sync(0xffffffffu, at, 31);
  int slot = 32, mine = 0;  // this lane's selected expert and its slot
  if (count <= 32) {
    at -= own;
    while (in) {
      const int j = L::expert(lane, __ffs(in) - 1);
      listed[wib][at++] = (unsigned long long)od[j] << 32 | (uint32_t)~j;
      in &= in - 1;
    }
    __syncwarp();
    const unsigned long long c = lane < count ? listed[wib][lane] : 0u;
    int ahead = 0;
#pragma unroll 4
    for (int i = 0; i < count; ++i) ahead += listed[wib][i] > c;
    mine = (int)~(uint32_t)c;
    if (lane < count) slot = ahead;
  } else {
    int first = 0;  // this lane's best
#pragma unroll
    for (int e = PER - 1; e >= 0; --e)
      if (ord[e] == best) first = e;
    for (int s = 0; s < p.k; ++s) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      const int j = best == top ? L::expert(lane, first) : INT32_MAX;
      const int w = __reduce_min_sync(0xffffffffu, j);
      if (lane == s) mine = w;
      if (j == w) {  // this lane's is taken
        best = 0u;
        int next = 0;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          if (e == first) ord[e] = 0u;
          if (ord[e] > best) best = ord[e], next = e;
        }
        first = next;
      }
    }
    slot = lane;
  }
  const bool taken = slot < p.k;
  float a = taken ? sc[mine] : 0.0f;
  if (p.renorm) {
    const float S = warp_sum(a);
    a = S == 0.0f ? 0.0f : a / S;  // nothing but zero scores: no weight
  }
  if (taken) {
    p.top_idx[t * p.k + slot] = mine;
    p.top_w[t * p.k + slot] = a * p.scale;
  }
}

struct SelectBwdParams {
  int T, N, k, renorm, sigmoid;
  float scale;
  const float* logits;
  const int32_t* top_idx;
  const float* d_top_w;
  const float* d_scores;
  float* dz;
  int* status;
};

// Adds what renormalised weights give to dz of a row whose selected scores sum to
// little: with w_i = s_i / S
//   w_i (da_i - sum da w) (1 - s_i)       softmax: without 1 - s_i, since the slots'
//                                         part of sum g s is 0
// A bias or the groups can select scores near fp32's smallest, where s / S keeps
// few bits and 1 / S overflows; so w comes from the logits z relative to the
// largest selected one.  Where every selected score rounds to 0 in fp32 (150 ln 2
// below 1), the weights are 0.
__device__ __forceinline__ void add_tiny_part(const SelectBwdParams& p, int64_t t, int lane) {
  constexpr float kNoScore = -103.972084f;  // the value below -150 ln 2
  const float* row = p.logits + t * p.N;
  int idx = lane < p.k ? p.top_idx[t * p.k + lane] : -1;
  if (idx >= p.N) idx = -1;
  const float z = idx >= 0 ? row[idx] : -INFINITY;
  const float da = idx >= 0 ? p.d_top_w[t * p.k + lane] * p.scale : 0.0f;
  float top = z;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  float log_top = top;  // of the largest selected score
  if (!p.sigmoid) {
    float m = -INFINITY, sum = 0.0f;
#pragma unroll 1
    for (int j = lane; j < p.N; j += 32) m = fmaxf(m, row[j]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll 1
    for (int j = lane; j < p.N; j += 32) sum += expf(row[j] - m);
    log_top = top - m - logf(warp_sum(sum));
  }
  if (top == -INFINITY || log_top <= kNoScore) return;
  const float x = p.sigmoid ? expf(-fabsf(z)) : 0.0f, q = 1.0f / (1.0f + x);
  if (p.sigmoid) top = fminf(top, 0.0f);
  // s_i over e^top (sigmoid) or over the largest selected score
  float w = p.sigmoid && z >= 0.0f ? q : expf(z - top) * q;
  w /= warp_sum(w);
  const float mean = warp_sum(w * da);
  const float part = w * (da - mean) * (p.sigmoid && z >= 0.0f ? x * q : q);
  float sum = 0.0f;
  int first = 32;
#pragma unroll 1
  for (int r = 0; r < p.k; ++r) {
    const int ir = __shfl_sync(0xffffffffu, idx, r);
    const float pr = __shfl_sync(0xffffffffu, part, r);
    if (ir == idx) {
      sum += pr;
      first = min(first, r);
    }
  }
  if (idx >= 0 && first == lane) p.dz[t * p.N + idx] += sum;
}

// One warp per token.  With g_j = dL/ds_j (d_scores plus what the weights of
// the selected experts give):
//   renorm: dL/ds_i = scale (da_i - sum_l da_l s_l / S) / S;  else scale da_i
//   sigmoid: dz_j = g_j s_j (1 - s_j);  softmax: dz_j = s_j (g_j - sum g s)
// d_scores is copied to shared memory (cp.async) while the scores are formed, so
// that it takes no registers and 28 warps fit an SM (at the price of 8 to 64 bytes
// of spills from 24 experts a lane on).  4096 x 896 with d_scores take 12.7 us, of
// which the bytes are 6.8: the warps, a token each, wait for their loads together.
template <int PER>
__global__ void __launch_bounds__(32 * kSelWarps, PER <= 28 ? 7 : 6)
    route_select_bwd(const __grid_constant__ SelectBwdParams p) {
  using L = Lanes<PER>;
  extern __shared__ __align__(16) float sel_mem[];  // per warp: s, the slots' part of g [N up to 4]
  pdl_wait();
  pdl_allow_next();
  const int lane = threadIdx.x & 31, wib = threadIdx.x >> 5, N = p.N;
  const int64_t t = (int64_t)blockIdx.x * kSelWarps + wib;
  if (t >= p.T) return;
  const int stride = (N + 3) & ~3;
  float* ss = sel_mem + (size_t)wib * 2 * stride;
  float* gs = ss + stride;
  float z[PER];  // becomes s, then the factor s (1 - s) or s
  if (p.d_scores && N % 4 == 0) {
    const float* d = p.d_scores + t * N;
#pragma unroll
    for (int e = 0; e < PER; e += L::CH) {
      const int j = L::expert(lane, e);
      if (L::CH == 4 && j < N) cp_async16(gs + j, d + j);
    }
  }
  L::load(p.logits + t * N, N, lane, -INFINITY, N % 4 == 0, z);
  int idx = lane < p.k ? p.top_idx[t * p.k + lane] : -1;
  float da = lane < p.k ? p.d_top_w[t * p.k + lane] * p.scale : 0.0f;
  if (lane < p.k && (idx < 0 || idx >= N)) {
    record_error(p.status, MOE_ERR_BOUNDS);
    idx = -1;
    da = 0.0f;
  }
  if (!p.sigmoid) {
    float m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int e = 0; e < PER; ++e) m = fmaxf(m, z[e]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      z[e] = z[e] == -INFINITY ? 0.0f : expf(z[e] - m);
      sum += z[e];
    }
    sum = warp_sum(sum);
    const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int e = 0; e < PER; ++e) z[e] *= r;
  }
#pragma unroll
  for (int e = 0; e < PER; e += L::CH) {
    float s[L::CH];
#pragma unroll
    for (int i = 0; i < L::CH; ++i) {
      s[i] = z[e + i];
      if (p.sigmoid) {  // s, and s (1 - s) without cancellation (r's rounding counts twice)
        const float x = expf(-fabsf(s[i])), r = 1.0f / (1.0f + x);
        s[i] = s[i] >= 0.0f ? r : x * r;
        z[e + i] = x * r * r;
      }
    }
    const int j = L::expert(lane, e);
    if (j >= N) continue;
    if constexpr (L::CH == 4) {
      *reinterpret_cast<float4*>(ss + j) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
#pragma unroll
      for (int i = 0; i < L::CH; ++i)
        if (j + i < N) ss[j + i] = s[i];
    }
    if (L::CH < 4 || N % 4 != 0 || !p.d_scores) {
#pragma unroll
      for (int i = 0; i < L::CH; ++i)
        if (j + i < N) gs[j + i] = p.d_scores ? p.d_scores[t * N + j + i] : 0.0f;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  // the selected experts' part; an index that is there twice counts twice
  bool tiny = false;  // of the whole row
  if (p.renorm) {
    const float s = idx >= 0 ? ss[idx] : 0.0f, S = warp_sum(s), ds = warp_sum(da * s);
    // above the bound a subnormal score is 2^-62 of the sum at most, and nothing
    // below 2^62 overflows
    tiny = S < 5.421011e-20f;  // 2^-64
    da = tiny || idx < 0 ? 0.0f : (da - ds / S) / S;
  }
  float sum = 0.0f;
  int first = 32;
#pragma unroll 4
  for (int r = 0; r < p.k; ++r) {
    const int ir = __shfl_sync(0xffffffffu, idx, r);
    const float dr = __shfl_sync(0xffffffffu, da, r);
    if (ir == idx) {
      sum += dr;
      first = min(first, r);
    }
  }
  if (idx >= 0 && first == lane) gs[idx] += sum;
  __syncwarp();
  float g[PER], dot = 0.0f;
  L::load_shared(gs, N, lane, g);
  if (!p.sigmoid) {
#pragma unroll
    for (int e = 0; e < PER; ++e) dot = fmaf(g[e], z[e], dot);
    dot = warp_sum(dot);
  }
#pragma unroll
  for (int e = 0; e < PER; ++e) g[e] = z[e] * (g[e] - dot);
  L::store(p.dz + t * N, N, lane, g);
  if (!tiny) return;
  __syncwarp();  // the row is stored before the selected experts' part is added
  add_tiny_part(p, t, lane);
}

template <template <int> class K, typename P>
int by_width(const P& p, size_t smem, cudaStream_t st) {
  const int chunks = (p.N + 127) / 128;  // of 4 experts a lane
  if (p.N <= 32) return K<1>::launch(p, smem, st);
  if (p.N <= 64) return K<2>::launch(p, smem, st);
  switch (chunks) {
    case 1: return K<4>::launch(p, smem, st);
    case 2: return K<8>::launch(p, smem, st);
    case 3: return K<12>::launch(p, smem, st);
    case 4: return K<16>::launch(p, smem, st);
    case 5: return K<20>::launch(p, smem, st);
    case 6: return K<24>::launch(p, smem, st);
    case 7: return K<28>::launch(p, smem, st);
    default: return K<32>::launch(p, smem, st);
  }
}

template <int PER>
struct Select {
  static int launch(const SelectParams& p, size_t smem, cudaStream_t st) {
    MOE_PREFER_SHARED((route_select<PER>));
    launch_pdl(route_select<PER>, dim3(((unsigned)p.T + kSelWarps - 1) / kSelWarps),
               dim3(32 * kSelWarps), smem, st, p);
    return launch_status();
  }
};
template <int PER>
struct SelectBwd {
  static int launch(const SelectBwdParams& p, size_t smem, cudaStream_t st) {
    MOE_PREFER_SHARED((route_select_bwd<PER>));
    launch_pdl(route_select_bwd<PER>, dim3(((unsigned)p.T + kSelWarps - 1) / kSelWarps),
               dim3(32 * kSelWarps), smem, st, p);
    return launch_status();
  }
};

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool gating_ok(const moe_shape* s, const moe_gating* g) {
  if (!s || !g || s->T < 0 || s->N <= 0 || s->N > 1024 || s->k <= 0 || s->k > 32 || s->k > s->N)
    return false;
  if ((int64_t)s->T * s->k >= (int64_t)1 << 31) return false;
  if (g->score != MOE_SCORE_SOFTMAX && g->score != MOE_SCORE_SIGMOID) return false;
  if (g->n_group < 1 || g->n_group > 32 || s->N % g->n_group != 0) return false;
  const int per = s->N / g->n_group;
  if (g->group_top < 1 || g->group_top > 2 || g->group_top > per) return false;
  return g->top_group >= 1 && g->top_group <= g->n_group && (int64_t)g->top_group * per >= s->k;
}

int launch_select(const moe_shape& s, const moe_gating& g, const float* logits, const float* bias,
                  int32_t* top_idx, float* top_w, float* scores, cudaStream_t st) {
  if (s.T == 0) return MOE_OK;
  // every group kept is no limit
  const int G = g.top_group == g.n_group ? 1 : g.n_group, per = s.N / G;
  int sub_log = 5;
  while (G << sub_log > 32) --sub_log;
  SelectParams p{s.T, s.N, s.k, s.renorm, g.score == MOE_SCORE_SIGMOID, G, g.top_group,
                 g.group_top, per, sub_log, (1u << 20) / per + 1,
                 s.N % 4 == 0 && aligned16(bias), g.scale, logits, bias, top_idx,
                 top_w, scores};
  return by_width<Select>(p, (size_t)kSelWarps * ((s.N + 3) & ~3) * 8, st);
}

}  // namespace
}  // namespace moe

extern "C" int moe_route_select(const moe_shape* shape, const moe_gating* gating,
                                const float* logits, const float* bias, int32_t* top_idx,
                                float* top_w, float* scores, void* stream) {
  using namespace moe;
  if (!gating_ok(shape, gating)) return MOE_ERR_INVALID_ARG;
  if (shape->T > 0 && (!logits || !top_idx || !top_w)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(scores) || !aligned4(bias) || !aligned4(top_idx) ||
      !aligned4(top_w))
    return MOE_ERR_INVALID_ARG;
  return launch_select(*shape, *gating, logits, bias, top_idx, top_w, scores, as_stream(stream));
}

extern "C" int moe_route_select_bwd(const moe_shape* shape, const moe_gating* gating,
                                    const float* logits, const int32_t* top_idx,
                                    const float* d_top_w, const float* d_scores, float* dz,
                                    void* stream) {
  using namespace moe;
  if (!gating_ok(shape, gating)) return MOE_ERR_INVALID_ARG;
  const moe_shape& s = *shape;
  if (s.T > 0 && (!logits || !top_idx || !d_top_w || !dz)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(d_scores) || !aligned16(dz) || !aligned4(top_idx) ||
      !aligned4(d_top_w))
    return MOE_ERR_INVALID_ARG;
  if (s.T == 0) return MOE_OK;
  SelectBwdParams p{s.T, s.N, s.k, s.renorm, gating->score == MOE_SCORE_SIGMOID, gating->scale,
                    logits, top_idx, d_top_w, d_scores, dz, status_word()};
  return by_width<SelectBwd>(p, (size_t)kSelWarps * ((s.N + 3) & ~3) * 8, as_stream(stream));
}

extern "C" size_t moe_route_scored_workspace_bytes(const moe_shape* shape) {
  if (!moe::shape_ok(shape)) return 0;
  return moe::route_ws_bytes(*shape);
}

extern "C" int moe_route_scored(const moe_shape* shape, const moe_gating* gating, const void* u,
                                int32_t u_dtype, const float* w_route, const float* bias,
                                int32_t* top_idx, float* top_w, float* scores, float* logits,
                                void* ws, size_t ws_bytes, void* stream) {
  using namespace moe;
  if (!shape_ok(shape) || !gating_ok(shape, gating) || !valid_act_dtype(u_dtype))
    return MOE_ERR_INVALID_ARG;
  if (shape->T > 0 && (!u || !w_route || !top_idx || !top_w)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(u) || !aligned16(w_route) || !aligned16(logits) || !aligned16(scores) ||
      !aligned4(bias) || !aligned4(top_idx) || !aligned4(top_w))
    return MOE_ERR_INVALID_ARG;
  if (shape->T == 0) return MOE_OK;
  if (!logits && (!ws || ws_bytes < route_ws_bytes(*shape))) return MOE_ERR_WORKSPACE;
  if (!logits && !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  float* z = logits ? logits : static_cast<float*>(ws);
  cudaStream_t st = as_stream(stream);
  const int rc = launch_route_logits(*shape, u, u_dtype, w_route, nullptr, z, st);
  if (rc != MOE_OK) return rc;
  return launch_select(*shape, *gating, z, bias, top_idx, top_w, scores, st);
}
