// The norms around a block of the residual stream, with the block's gate and
// the residual scale, in one pass over the rows:
//   n  = y / sqrt(mean(y^2) + eps) * w_post      (w_post NULL: n = y)
//   x' = res_scale x + out_scale gate n          rounded to the storage type
//   u  = x' / sqrt(mean(x'^2) + eps) * w_pre     of x' as stored
// and its gradients.
//
// Every sum over a row and over the tokens is fp32 in a fixed order.
#include "common.cuh"

namespace moe {
namespace {

constexpr int kNormThreads = 512;   // threads of a CTA, at most
constexpr int kNormMaxD = 16384;    // 4 CTAs of 512 threads x 8 columns

struct NormFwd {
  int T, d, C;             // C: CTAs of a cluster, each with its share of a row's columns
  int nt;                  // threads per row in a CTA (a multiple of 32)
  const void *x, *y, *gate_full;
  const float *w_post, *w_pre, *gate;
  int gate_kind;
  float alpha, beta, eps, inv_d;
  void *x_out, *u;
};

struct NormBwd {
  int T, d, C, nt;
  const void *x_out, *y, *gate_full, *dx_out, *du;
  const float *w_post, *w_pre, *gate;
  int gate_kind, branch;
  float alpha, beta, eps, inv_d;
  void *dx, *dy, *dgate_full;
  float* dgate_tok;
  float *part_post, *part_pre, *part_gate;  // [parts][d], nullable
};

__device__ __forceinline__ void cp16(uint32_t smem, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(g) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T>
constexpr int planes() { return sizeof(T) == 4 ? 2 : 1; }  // 16-byte planes of 8 elements

// A thread's private FIFO in shared memory: each thread copies the 8 columns
// that it will itself use, S - 1 rows ahead, so the copies need no barrier.
// Plane p of stage s holds 16 bytes for each thread of the CTA.
struct Fifo {
  uint32_t base;  // shared address of this thread's slot in plane 0
  char* ptr;
  int plane, stage;  // bytes between planes, between stages
};

template <typename T>
__device__ __forceinline__ void fifo_put(const Fifo& f, int slot, int p, const T* src) {
  const uint32_t a = f.base + slot * f.stage + p * f.plane;
  cp16(a, src);
  if (sizeof(T) == 4) cp16(a + f.plane, reinterpret_cast<const char*>(src) + 16);
}
template <typename T>
__device__ __forceinline__ void fifo_get(const Fifo& f, int slot, int p, float* o) {
  const char* a = f.ptr + slot * f.stage + p * f.plane;
  if (sizeof(T) == 4) {
    const float4 v0 = *reinterpret_cast<const float4*>(a);
    const float4 v1 = *reinterpret_cast<const float4*>(a + f.plane);
    o[0] = v0.x, o[1] = v0.y, o[2] = v0.z, o[3] = v0.w;
    o[4] = v1.x, o[5] = v1.y, o[6] = v1.z, o[7] = v1.w;
  } else {
    load8(reinterpret_cast<const T*>(a), o);
  }
}

// Rounds 8 values to T and stores them; v holds the rounded values after it.
template <typename T>
__device__ __forceinline__ void store8(T* o, float* v) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    __align__(16) T r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = from_f32<T>(v[i]);
    *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(r[i]);
  }
}

__device__ __forceinline__ void gains8(const float* w, int c, bool on, float* o) {
  if (w && on) {
    load8(w + c, o);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = 1.0f;
  }
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}

// Sums of K values over the threads of a row: lanes by a shuffle tree, the
// team's warps likewise from shared memory, then the CTAs of the cluster in
// rank order through distributed shared memory.  Two buffers taken in turn:
// a thread writes a buffer again only after a barrier that every reader of
// its last contents has reached.
struct RowSum {
  float (*warp_part)[16][4];  // [2][16 warps of the CTA][4]
  float (*rank_part)[4][4];   // [2][4 ranks][4]
  int team, nt, warps, C;     // warps: of this team
  int turn;
};

template <int K>
__device__ __forceinline__ void row_sum(RowSum& r, float* v) {
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  const int b = r.turn;
  if (r.warps > 1) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) r.warp_part[b][w][k] = v[k];
    asm volatile("bar.sync %0, %1;" ::"r"(r.team + 1), "r"(r.nt) : "memory");
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = lane < r.warps ? r.warp_part[b][r.team * r.warps + lane][k] : 0.0f;
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
      v[k] = __shfl_sync(0xffffffffu, v[k], 0);
    }
  }
  if (r.C > 1) {
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    if ((int)threadIdx.x < r.C) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        uint32_t a;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(a)
                     : "r"(smem_addr(&r.rank_part[b][rank][k])), "r"(threadIdx.x));
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v[k]) : "memory");
      }
    }
    __syncwarp();
    cluster_barrier();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = 0.0f;
      for (int c = 0; c < r.C; ++c) v[k] += r.rank_part[b][c][k];
    }
  }
  r.turn = b ^ 1;
}

// What a thread of either kernel is: its row team, its 8 columns.
struct Place {
  int team, lane_t;   // team of this CTA, thread in the team
  int c0;             // first column
  bool on;            // whether the columns exist
  int64_t first, step;
};

__device__ __forceinline__ Place place_of(int nt, int C, int d) {
  Place q;
  q.team = threadIdx.x / nt;
  q.lane_t = threadIdx.x - q.team * nt;
  const int teams = blockDim.x / nt;
  const int rank = blockIdx.x % C;
  q.c0 = (rank * nt + q.lane_t) * 8;
  q.on = q.c0 < d;
  q.first = (int64_t)(blockIdx.x / C) * teams + q.team;
  q.step = (int64_t)(gridDim.x / C) * teams;
  return q;
}

template <typename T, int S>
__global__ void __launch_bounds__(kNormThreads, 2) block_norm_fwd(const __grid_constant__ NormFwd p) {
  extern __shared__ __align__(16) char fifo_mem[];
  __shared__ float warp_part[2][16][4];
  __shared__ float rank_part[2][4][4];
  pdl_wait();
  pdl_allow_next();
  const Place q = place_of(p.nt, p.C, p.d);
  RowSum sums{warp_part, rank_part, q.team, p.nt, p.nt / 32, p.C, 0};
  if (p.C > 1) cluster_barrier();  // every CTA of the cluster runs before its memory is written
  constexpr int P = planes<T>();
  const bool has_y = p.y != nullptr, full = p.gate_full != nullptr;
  const int pg = 2 * P;  // planes: x, y, full gate
  Fifo f;
  f.plane = blockDim.x * 16;
  f.stage = (P * (1 + has_y + full)) * f.plane;
  f.ptr = fifo_mem + threadIdx.x * 16;
  f.base = smem_addr(f.ptr);
  const T* x = static_cast<const T*>(p.x) + q.c0;
  const T* y = static_cast<const T*>(p.y) + q.c0;
  const T* g = static_cast<const T*>(p.gate_full) + q.c0;
  auto issue = [&](int64_t row, int slot) {
    if (row < p.T && q.on) {
      const size_t o = (size_t)row * p.d;
      fifo_put<T>(f, slot, 0, x + o);
      if (has_y) fifo_put<T>(f, slot, P, y + o);
      if (full) fifo_put<T>(f, slot, pg, g + o);
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(q.first + s * q.step, s);
  float wpost[8], wpre[8], gch[8];
  gains8(p.w_post, q.c0, q.on, wpost);
  gains8(p.w_pre, q.c0, q.on, wpre);
  gains8(p.gate_kind == MOE_GATE_CHANNEL ? p.gate : nullptr, q.c0, q.on, gch);
  int slot = 0;
  for (int64_t t = q.first; t < p.T; t += q.step) {
    issue(t + (S - 1) * q.step, slot == 0 ? S - 1 : slot - 1);
    const float gt = p.gate_kind == MOE_GATE_TOKEN ? p.gate[t] : 1.0f;
    cp_wait<S - 1>();
    float xv[8], yv[8];
    if (q.on) {
      fifo_get<T>(f, slot, 0, xv);
      if (has_y) fifo_get<T>(f, slot, P, yv);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) xv[i] = yv[i] = 0.0f;
    }
    if (has_y) {
      float r = 1.0f;
      if (p.w_post) {
        float ss[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = fmaf(yv[i], yv[i], ss[0]);
        row_sum<1>(sums, ss);
        r = rsqrtf(fmaf(ss[0], p.inv_d, p.eps));
      }
      float gv[8];
      if (full && q.on) {
        fifo_get<T>(f, slot, pg, gv);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) gv[i] = gch[i] * gt;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        xv[i] = fmaf(p.beta * gv[i], yv[i] * r * wpost[i], p.alpha * xv[i]);
      // rounded here: the next norm reads the stream as it is stored
      if (q.on) store8<T>(static_cast<T*>(p.x_out) + (size_t)t * p.d + q.c0, xv);
    }
    if (p.w_pre) {
      float ss[1] = {0.0f};
      if (q.on)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = fmaf(xv[i], xv[i], ss[0]);
      row_sum<1>(sums, ss);
      const float r = rsqrtf(fmaf(ss[0], p.inv_d, p.eps));
#pragma unroll
      for (int i = 0; i < 8; ++i) xv[i] = xv[i] * r * wpre[i];
      if (q.on) store8<T>(static_cast<T*>(p.u) + (size_t)t * p.d + q.c0, xv);
    }
    slot = slot + 1 == S ? 0 : slot + 1;
  }
}

// Gradients.  With A = sum x'^2, B = sum x' w_pre du, r1 = 1 / sqrt(A/d + eps):
//   dx' = dx_out + r1 (w_pre du - x' r1^2 B / d)         dx = res_scale dx'
//   dw_pre = sum_t du x' r1
// and with b = out_scale dx', yh = y r2, dn = b gate, D = sum yh w_post dn:
//   dy = r2 (w_post dn - yh D / d)   dw_post = sum_t dn yh   dgate = b yh w_post
// The norms' factors are formed again from x' and y, which the row needs anyway.
template <typename T, typename G, int S>
__global__ void __launch_bounds__(kNormThreads, 1) block_norm_bwd(const __grid_constant__ NormBwd p) {
  extern __shared__ __align__(16) char fifo_mem[];
  __shared__ float warp_part[2][16][4];
  __shared__ float rank_part[2][4][4];
  pdl_wait();
  pdl_allow_next();
  const Place q = place_of(p.nt, p.C, p.d);
  RowSum sums{warp_part, rank_part, q.team, p.nt, p.nt / 32, p.C, 0};
  if (p.C > 1) cluster_barrier();
  constexpr int P = planes<T>(), PG = planes<G>();
  const bool pre = p.w_pre != nullptr, post = p.w_post != nullptr;
  const bool has_y = p.y != nullptr, full = p.gate_full != nullptr, has_d = p.dx_out != nullptr;
  const int py = P * pre, pg = py + P * has_y, pd = pg + P * full, pu = pd + PG * has_d;
  Fifo f;
  f.plane = blockDim.x * 16;
  f.stage = (pu + PG * pre) * f.plane;
  f.ptr = fifo_mem + threadIdx.x * 16;
  f.base = smem_addr(f.ptr);
  auto issue = [&](int64_t row, int slot) {
    if (row < p.T && q.on) {
      const size_t o = (size_t)row * p.d + q.c0;
      if (pre) fifo_put<T>(f, slot, 0, static_cast<const T*>(p.x_out) + o);
      if (has_y) fifo_put<T>(f, slot, py, static_cast<const T*>(p.y) + o);
      if (full) fifo_put<T>(f, slot, pg, static_cast<const T*>(p.gate_full) + o);
      if (has_d) fifo_put<G>(f, slot, pd, static_cast<const G*>(p.dx_out) + o);
      if (pre) fifo_put<G>(f, slot, pu, static_cast<const G*>(p.du) + o);
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(q.first + s * q.step, s);
  float wpost[8], wpre[8], gch[8], a_post[8], a_pre[8], a_gate[8];
  gains8(p.w_post, q.c0, q.on, wpost);
  gains8(p.w_pre, q.c0, q.on, wpre);
  gains8(p.gate_kind == MOE_GATE_CHANNEL ? p.gate : nullptr, q.c0, q.on, gch);
#pragma unroll
  for (int i = 0; i < 8; ++i) a_post[i] = a_pre[i] = a_gate[i] = 0.0f;
  int slot = 0;
  for (int64_t t = q.first; t < p.T; t += q.step) {
    issue(t + (S - 1) * q.step, slot == 0 ? S - 1 : slot - 1);
    const float gt = p.gate_kind == MOE_GATE_TOKEN ? p.gate[t] : 1.0f;
    cp_wait<S - 1>();
    float xv[8], yv[8], dv[8], uv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) xv[i] = yv[i] = dv[i] = uv[i] = 0.0f;
    if (q.on) {
      if (pre) {
        fifo_get<T>(f, slot, 0, xv);
        fifo_get<G>(f, slot, pu, uv);
      }
      if (has_y) fifo_get<T>(f, slot, py, yv);
      if (has_d) fifo_get<G>(f, slot, pd, dv);
    }
    float s3[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s3[0] = fmaf(xv[i], xv[i], s3[0]);
      s3[1] = fmaf(xv[i] * wpre[i], uv[i], s3[1]);
      s3[2] = fmaf(yv[i], yv[i], s3[2]);
    }
    if (pre || post) row_sum<3>(sums, s3);
    if (pre) {
      const float r1 = rsqrtf(fmaf(s3[0], p.inv_d, p.eps));
      const float m = s3[1] * p.inv_d * r1 * r1;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a_pre[i] = fmaf(uv[i], xv[i] * r1, a_pre[i]);
        dv[i] = fmaf(r1, fmaf(wpre[i], uv[i], -xv[i] * m), dv[i]);
      }
    }
    float ov[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) ov[i] = p.branch ? p.alpha * dv[i] : dv[i];
    const size_t o = (size_t)t * p.d + q.c0;
    if (q.on) store8<G>(static_cast<G*>(p.dx) + o, ov);
    if (p.branch) {
      const float r2 = post ? rsqrtf(fmaf(s3[2], p.inv_d, p.eps)) : 1.0f;
      float gv[8];
      if (full && q.on) {
        fifo_get<T>(f, slot, pg, gv);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) gv[i] = gch[i] * gt;
      }
      // sum of n b, times the gate where it is one value for the row
      float s1[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dv[i] *= p.beta;       // b
        yv[i] *= r2;           // yh
        const float nb = yv[i] * wpost[i] * dv[i];
        s1[0] = fmaf(nb, p.gate_kind == MOE_GATE_TOKEN ? 1.0f : gv[i], s1[0]);
        ov[i] = nb;            // dgate, before any sum
        a_gate[i] += nb;
        a_post[i] = fmaf(dv[i] * gv[i], yv[i], a_post[i]);
      }
      if (full && q.on) store8<T>(static_cast<T*>(p.dgate_full) + o, ov);
      float m = 0.0f;
      if (post || p.dgate_tok) {
        row_sum<1>(sums, s1);
        if (p.dgate_tok && q.c0 == 0) p.dgate_tok[t] = s1[0];
        m = s1[0] * gt * p.inv_d;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        ov[i] = post ? r2 * fmaf(wpost[i], dv[i] * gv[i], -yv[i] * m) : dv[i] * gv[i];
      if (q.on) store8<T>(static_cast<T*>(p.dy) + o, ov);
    }
    slot = slot + 1 == S ? 0 : slot + 1;
  }
  // The CTA's teams add their columns' sums in team order, through the FIFO's
  // memory once every copy into it has landed.
  cp_wait<0>();
  const int teams = blockDim.x / p.nt;
  float* acc[3] = {p.part_post, p.part_pre, p.part_gate};
  float* mem = reinterpret_cast<float*>(fifo_mem);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (!acc[k]) continue;
    float* a = k == 0 ? a_post : k == 1 ? a_pre : a_gate;
    if (teams > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) mem[i * blockDim.x + threadIdx.x] = a[i];
      __syncthreads();
      if (q.team == 0)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          for (int m = 1; m < teams; ++m) a[i] += mem[i * blockDim.x + m * p.nt + q.lane_t];
    }
    if (q.team == 0 && q.on) {
      float* o = acc[k] + (size_t)(blockIdx.x / p.C) * p.d + q.c0;
      store8<float>(o, a);
    }
  }
}

// dw[c] = sum over the parts, ascending: 32 columns by 8 runs of parts for a
// block, the runs added in order.
struct NormSums {
  int parts, d;
  const float* part[3];
  float* out[3];
};
__global__ void __launch_bounds__(256) block_norm_sums(const __grid_constant__ NormSums p) {
  pdl_wait();
  pdl_allow_next();
  __shared__ float run[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
  const float* src = p.part[blockIdx.y];
  if (!src) return;
  const int per = (p.parts + 7) / 8, lo = r * per, hi = min(p.parts, lo + per);
  float a = 0.0f;
  if (c < p.d)
    for (int i = lo; i < hi; ++i) a += src[(size_t)i * p.d + c];
  run[r][threadIdx.x & 31] = a;
  __syncthreads();
  if (r == 0 && c < p.d) {
#pragma unroll
    for (int i = 1; i < 8; ++i) a += run[i][threadIdx.x];
    p.out[blockIdx.y][c] = a;
  }
}

// ------------------------------------------------------------------- host
struct NormPlan {
  int C, nt, block, grid;
  size_t smem;
};

// bytes: of the FIFO per thread.  ctas: CTAs per SM to launch, at most.
NormPlan norm_plan(int T, int d, int bytes, int ctas) {
  NormPlan q;
  const int chunks = d / 8;
  q.C = (chunks + kNormThreads - 1) / kNormThreads;
  if (q.C == 3) q.C = 4;
  q.nt = ((chunks + q.C - 1) / q.C + 31) / 32 * 32;
  int teams = q.C > 1 ? 1 : kNormThreads / q.nt;
  if (teams > T) teams = T;
  q.block = teams * q.nt;
  q.smem = (size_t)bytes * q.block;
  const int64_t want = (int64_t)((T + teams - 1) / teams) * q.C;
  int64_t most = (int64_t)sm_count() * ctas / q.C * q.C;
  q.grid = (int)(want < most ? want : most);
  return q;
}

constexpr int kBwdParts = 148;  // CTAs (clusters) of the backward, at most

template <typename K, typename P>
int launch_norm(K kernel, const P& p, const NormPlan& q, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)q.grid);
  cfg.blockDim = dim3((unsigned)q.block);
  cfg.dynamicSmemBytes = q.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = q.C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = q.C > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) pdl_launch_error() = e;
  return launch_status();
}

constexpr int kNormSmem = 200 * 1024;  // dynamic shared memory of a CTA, at most

template <typename T, int S>
int run_fwd(const NormFwd& p0, cudaStream_t st) {
  NormFwd p = p0;
  const int bytes = S * 16 * planes<T>() * (1 + (p.y != nullptr) + (p.gate_full != nullptr));
  const NormPlan q = norm_plan(p.T, p.d, bytes, 2);
  p.C = q.C;
  p.nt = q.nt;
  auto kernel = block_norm_fwd<T, S>;
  static std::atomic<bool> configured[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !device_slot(dev)) return MOE_ERR_CUDA;
  if (needs_setup(configured, dev)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    mark_setup(configured, dev);
  }
  MOE_PREFER_SHARED((block_norm_fwd<T, S>));
  return launch_norm(kernel, p, q, st);
}

template <typename T, typename G, int S>
int run_bwd(const NormBwd& p0, const moe_block_norm_grads& g, float* parts, cudaStream_t st) {
  NormBwd p = p0;
  const bool pre = p.w_pre != nullptr;
  const int bytes = S * 16 * (planes<T>() * (pre + (p.y != nullptr) + (p.gate_full != nullptr)) +
                              planes<G>() * ((p.dx_out != nullptr) + pre));
  NormPlan q = norm_plan(p.T, p.d, bytes, 1);
  if (q.grid > kBwdParts) q.grid = kBwdParts / q.C * q.C;
  if (q.smem < (size_t)q.block * 32) q.smem = (size_t)q.block * 32;  // the teams' column sums
  p.C = q.C;
  p.nt = q.nt;
  const int n = q.grid / q.C;
  NormSums s{};
  float** part[3] = {&p.part_post, &p.part_pre, &p.part_gate};
  float* out[3] = {g.dw_post, g.dw_pre, p.gate_kind == MOE_GATE_CHANNEL ? (float*)g.dgate : nullptr};
  for (int k = 0; k < 3; ++k) {
    if (!out[k]) continue;
    // one part: the kernel writes the sums themselves
    *part[k] = n == 1 ? out[k] : parts + (size_t)k * kBwdParts * p.d;
    s.part[k] = *part[k];
    s.out[k] = out[k];
  }
  auto kernel = block_norm_bwd<T, G, S>;
  static std::atomic<bool> configured[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !device_slot(dev)) return MOE_ERR_CUDA;
  if (needs_setup(configured, dev)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    mark_setup(configured, dev);
  }
  MOE_PREFER_SHARED((block_norm_bwd<T, G, S>));
  int rc = launch_norm(kernel, p, q, st);
  if (rc != MOE_OK || n == 1 || (!out[0] && !out[1] && !out[2])) return rc;
  s.parts = n;
  s.d = p.d;
  MOE_PREFER_SHARED((block_norm_sums));
  launch_pdl(block_norm_sums, dim3((p.d + 31) / 32, 3), dim3(256), 0, st, s);
  return launch_status();
}

bool norm_ok(const moe_block_norm* b) {
  if (!b || b->T < 0 || b->d <= 0 || b->d % 8 != 0 || b->d > kNormMaxD) return false;
  return b->gate >= MOE_GATE_NONE && b->gate <= MOE_GATE_FULL && b->eps > 0.0f;
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
  p.gate = b.gate == MOE_GATE_FULL ? nullptr : static_cast<const float*>(gate);
  p.gate_kind = b.gate;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.alpha = b.res_scale;
  p.beta = b.out_scale;
  p.eps = b.eps;
  p.inv_d = 1.0f / (float)b.d;
  p.x_out = x_out;
  p.u = u;
  cudaStream_t st = as_stream(stream);
  if (dtype == MOE_F32) return run_fwd<float, 2>(p, st);
  if (dtype == MOE_BF16) return run_fwd<__nv_bfloat16, 4>(p, st);
  return run_fwd<__half, 4>(p, st);
}

extern "C" size_t moe_block_norm_bwd_workspace_bytes(const moe_block_norm* norm) {
  if (!moe::norm_ok(norm)) return 0;
  return moe::align_up((size_t)3 * moe::kBwdParts * norm->d * 4, 256);
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
  p.gate = b.gate == MOE_GATE_FULL ? nullptr : static_cast<const float*>(gate);
  p.gate_kind = b.gate;
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
  if (dtype == MOE_F32) return run_bwd<float, float, 2>(p, g, parts, st);
  if (dtype == MOE_BF16)
    return grad_dtype == MOE_F32 ? run_bwd<__nv_bfloat16, float, 3>(p, g, parts, st)
                                 : run_bwd<__nv_bfloat16, __nv_bfloat16, 4>(p, g, parts, st);
  return grad_dtype == MOE_F32 ? run_bwd<__half, float, 3>(p, g, parts, st)
                               : run_bwd<__half, __half, 4>(p, g, parts, st);
}
