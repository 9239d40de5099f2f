// Pieces of the block-norm kernels (norm.cu, norm_bwd.cu).
//
// A team of nt threads (a multiple of 32, at most 256) takes a row, 16 columns a
// thread in two chunks of 8, so that the fixed work of a row (its sums'
// shuffles, the barriers, the addresses) is spread over many columns; teams
// walk the rows with a stride.  Each thread copies its own columns of the next
// rows into shared memory with cp.async, S - 1 rows ahead: the copies need no
// barrier, and nothing but the running sums and the gains stays in registers.
// Columns past the row's end are filled with zeros, so only the stores ask for
// them.  Arithmetic is on pairs (one instruction for two fp32 operations).
// Rows above 4096 columns go to a cluster of two or four CTAs that exchange
// their sums through distributed shared memory.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kNormThreads = 256;
constexpr int kNormMaxD = 16384;       // a cluster of 4 CTAs of 256 threads x 16 columns
constexpr int kNormSmem = 200 * 1024;  // dynamic shared memory of an SM that the CTAs take, at most

namespace {

// ---------------------------------------------------------- pairs of fp32
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float a, float b) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 parts(Pair p) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float sum2(Pair p) {
  const float2 v = parts(p);
  return v.x + v.y;
}

// Two values of 16 bits (the low half first) as a pair.
template <typename T>
__device__ __forceinline__ Pair widen(uint32_t w);
template <>
__device__ __forceinline__ Pair widen<__nv_bfloat16>(uint32_t w) {
  return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ Pair widen<__half>(uint32_t w) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pair(v.x, v.y);
}
template <typename T>
__device__ __forceinline__ uint32_t narrow(Pair p);
template <>
__device__ __forceinline__ uint32_t narrow<__nv_bfloat16>(Pair p) {
  const float2 v = parts(p);
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t narrow<__half>(Pair p) {
  const float2 v = parts(p);
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ------------------------------------------------------- the threads' FIFO
// A chunk is 8 columns: 16 bytes of a 16-bit type, two times 16 of fp32.  A
// thread has two chunks of every array, and per stage of the FIFO a slot of 16
// bytes in each plane of blockDim.x slots.
template <typename T>
constexpr int planes() { return 2 * (sizeof(T) == 4 ? 2 : 1); }  // of an array

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes, of which `size` (16 or 0) are read and the others are zeros.
__device__ __forceinline__ void cp16(uint32_t smem, const void* g, uint32_t size) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(g), "r"(size)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// What a thread is: its row team, its two chunks of columns.
struct Place {
  int team, lane_t;     // team of this CTA, thread in the team
  int c[2];             // first column of each chunk; 0 where there is none
  bool on[2];           // whether the columns exist
  uint32_t size[2];     // 16 or 0 (cp16)
  int first, step;      // rows
  int count;            // rows that this team takes
};

__device__ __forceinline__ Place place_of(int nt, int C, int d, int T) {
  Place q;
  q.team = threadIdx.x / nt;
  q.lane_t = threadIdx.x - q.team * nt;
  const int teams = blockDim.x / nt, rank = blockIdx.x % C;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    q.c[v] = ((rank * 2 + v) * nt + q.lane_t) * 8;
    q.on[v] = q.c[v] < d;
    q.size[v] = q.on[v] ? 16 : 0;
    if (!q.on[v]) q.c[v] = 0;
  }
  q.first = (blockIdx.x / C) * teams + q.team;
  q.step = (gridDim.x / C) * teams;
  q.count = q.first < T ? (T - q.first - 1) / q.step + 1 : 0;
  return q;
}

// One array's rows as a thread sees them: the copies walk with their own row.
template <typename T>
struct Stream {
  const T* next;        // the row of the next copy
  uint32_t at;          // its first plane in a stage
  __device__ __forceinline__ void start(const void* p, const Place& q, int d, uint32_t plane) {
    next = static_cast<const T*>(p) + (size_t)q.first * d;
    at = plane;
  }
  // the next row into a stage (its shared address), then one step on
  __device__ __forceinline__ void copy(const Place& q, uint32_t stage, uint32_t step, size_t skip) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const uint32_t a = stage + (at + v * planes<T>() / 2) * step;
      const char* src = reinterpret_cast<const char*>(next + q.c[v]);
      cp16(a, src, q.size[v]);
      if (sizeof(T) == 4) cp16(a + step, src + 16, q.size[v]);
    }
    next += skip;
  }
  // chunk v of a stage
  __device__ __forceinline__ void get(int v, uint32_t stage, uint32_t step, Pair* o) const {
    const uint32_t a = stage + (at + v * planes<T>() / 2) * step;
    const uint4 x = lds16(a);
    if constexpr (sizeof(T) == 4) {
      const uint4 y = lds16(a + step);
      o[0] = pair(__uint_as_float(x.x), __uint_as_float(x.y));
      o[1] = pair(__uint_as_float(x.z), __uint_as_float(x.w));
      o[2] = pair(__uint_as_float(y.x), __uint_as_float(y.y));
      o[3] = pair(__uint_as_float(y.z), __uint_as_float(y.w));
    } else {
      o[0] = widen<T>(x.x);
      o[1] = widen<T>(x.y);
      o[2] = widen<T>(x.z);
      o[3] = widen<T>(x.w);
    }
  }
};

// Rounds a chunk to T and stores it; v holds the rounded values after it.
template <typename T>
__device__ __forceinline__ void store_chunk(T* o, bool on, Pair* v) {
  if constexpr (sizeof(T) == 4) {
    const float2 a = parts(v[0]), b = parts(v[1]), c = parts(v[2]), d = parts(v[3]);
    if (on) {
      reinterpret_cast<float4*>(o)[0] = make_float4(a.x, a.y, b.x, b.y);
      reinterpret_cast<float4*>(o)[1] = make_float4(c.x, c.y, d.x, d.y);
    }
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = narrow<T>(v[i]);
      v[i] = widen<T>(w[i]);
    }
    if (on) *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The products of the gains that are given (NULL: 1), times f.
__device__ __forceinline__ void gains(const Place& q, const float* a, const float* b, float f,
                                      Pair* o) {
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    float w[8], z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = z[i] = 1.0f;
    if (a) load8(a + q.c[v], w);
    if (b) load8(b + q.c[v], z);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[4 * v + i] = pair(w[2 * i] * z[2 * i] * f, w[2 * i + 1] * z[2 * i + 1] * f);
  }
}

__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}

// Sums of K values over the threads of a row: lanes by a shuffle tree, the
// team's warps in order from shared memory, then the CTAs of the cluster in
// rank order through distributed shared memory.  Two buffers taken in turn:
// a thread writes a buffer again only after a barrier that every reader of
// its last contents has reached.
struct SumBuffers {
  float4 warp_part[2][kNormThreads / 32];  // by warp of the CTA
  float4 rank_part[2][4];
};
struct RowSum {
  SumBuffers* m;
  int team, nt, warps, C;     // warps: of this team
  int turn;
};

template <int K>
__device__ __forceinline__ void row_sum(RowSum& r, float* v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  const int b = r.turn;
  if (r.warps > 1) {
    const int w = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0)
      r.m->warp_part[b][w] = make_float4(v[0], K > 1 ? v[1] : 0.0f, K > 2 ? v[2] : 0.0f, 0.0f);
    asm volatile("bar.sync %0, %1;" ::"r"(r.team + 1), "r"(r.nt) : "memory");
    const float4* p = &r.m->warp_part[b][r.team * r.warps];
    float4 a = p[0];
#pragma unroll
    for (int i = 1; i < kNormThreads / 32; ++i) {
      if (i >= r.warps) break;
      a.x += p[i].x;
      if (K > 1) a.y += p[i].y;
      if (K > 2) a.z += p[i].z;
    }
    v[0] = a.x;
    if (K > 1) v[1] = a.y;
    if (K > 2) v[2] = a.z;
  }
  if (r.C > 1) {
    const int rank = blockIdx.x % r.C;
    if ((int)threadIdx.x < r.C) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        uint32_t a;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(a)
                     : "r"(smem_addr(&r.m->rank_part[b][rank]) + 4 * k), "r"(threadIdx.x));
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v[k]) : "memory");
      }
    }
    cluster_barrier();
    float4 a = r.m->rank_part[b][0];
    for (int c = 1; c < r.C; ++c) {
      const float4 z = r.m->rank_part[b][c];
      a.x += z.x, a.y += z.y, a.z += z.z;
    }
    v[0] = a.x;
    if (K > 1) v[1] = a.y;
    if (K > 2) v[2] = a.z;
  }
  r.turn = b ^ 1;
}

// ------------------------------------------------------------------- host
struct NormPlan {
  int C, nt, block, grid;
  size_t smem;
};

// bytes: of the FIFO per thread.  ctas: CTAs of 256 threads per SM.  Few rows
// are spread over the SMs before a CTA gets a second team.
inline NormPlan norm_plan(int T, int d, int bytes, int ctas) {
  NormPlan q;
  const int sms = sm_count(), chunks = d / 8;
  q.C = chunks <= 2 * kNormThreads ? 1 : chunks <= 4 * kNormThreads ? 2 : 4;
  q.nt = ((chunks + 2 * q.C - 1) / (2 * q.C) + 31) / 32 * 32;
  int teams = kNormThreads / q.nt;
  const int spread = (T + sms - 1) / sms;
  if (teams > spread) teams = spread;
  q.block = teams * q.nt;
  q.smem = (size_t)bytes * q.block;
  int per_sm = kNormThreads * ctas / q.block;
  const int fit = (int)(kNormSmem / q.smem);
  if (per_sm > fit) per_sm = fit;
  const int64_t want = (int64_t)((T + teams - 1) / teams) * q.C;
  const int64_t most = (int64_t)sms * per_sm / q.C * q.C;
  q.grid = (int)(want < most ? want : most);
  return q;
}

// Launches a block-norm kernel, with its shared-memory attribute set once per
// device and instantiation.
template <typename P>
int launch_norm(void (*kernel)(P), std::atomic<bool>* configured, const P& p, const NormPlan& q,
                cudaStream_t st) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !device_slot(dev)) return MOE_ERR_CUDA;
  if (needs_setup(configured, dev)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                         (int)cudaSharedmemCarveoutMaxShared);
    mark_setup(configured, dev);
  }
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

inline bool norm_ok(const moe_block_norm* b) {
  if (!b || b->T < 0 || b->d <= 0 || b->d % 8 != 0 || b->d > kNormMaxD) return false;
  return b->gate >= MOE_GATE_NONE && b->gate <= MOE_GATE_FULL && b->eps > 0.0f;
}

}  // namespace
}  // namespace moe
