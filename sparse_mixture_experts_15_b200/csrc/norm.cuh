// Pieces of the block-norm kernels (norm.cu, norm_bwd.cu).
//
// A team of nt threads (a multiple of 32, at most 256) takes a row, 16 columns a
// thread, so that the fixed work of a row (its sums' shuffles, the barriers, the
// addresses) is spread over many columns; teams walk the rows with a stride.
// One thread of a team starts bulk copies of the next rows into a ring in
// shared memory, so that the loads in flight cost no registers and no
// instructions of the other threads.  (Copies by every thread, cp.async, reached
// the same bandwidth alone, but not next to the row's arithmetic: 136 us against
// 106 for the gradients of 8192 x 4096 bf16 with fp32 stream gradients.)
// Arithmetic is on pairs (one instruction for two fp32 operations).  Rows
// above 4096 columns go to a cluster of two or four CTAs that exchange their sums
// through distributed shared memory.
#pragma once

#include "common.cuh"
#include "pairs.cuh"
#include "tc_primitives.cuh"

namespace moe {

constexpr int kNormThreads = 256;
constexpr int kNormMaxD = 16384;       // a cluster of 4 CTAs of 256 threads x 16 columns
constexpr int kNormSmem = 200 * 1024;  // dynamic shared memory of an SM that the CTAs take, at most

namespace {

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

// ------------------------------------------------------------ the rows' ring
// A thread's columns are chunks of W, nt W apart: W = 8 where every array has
// 16-bit elements (16 bytes a thread), 4 where one has fp32, so that the
// threads' reads of either width are of consecutive bytes.
constexpr int kCols = 16;  // columns a thread
template <typename T, typename G>
constexpr int chunk_width() { return sizeof(T) == 2 && sizeof(G) == 2 ? 8 : 4; }

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// What a thread is: its row team and its columns.
struct Place {
  int team, lane_t;        // team of this CTA, thread in the team
  int begin, cols;         // the columns of this CTA: first one, how many
  uint32_t first, step;    // rows
  int count;               // rows that this team takes
};

__device__ __forceinline__ Place place_of(int nt, int C, int d, int T) {
  Place q;
  q.team = threadIdx.x / nt;
  q.lane_t = threadIdx.x - q.team * nt;
  const int teams = blockDim.x / nt, rank = blockIdx.x % C;
  q.begin = rank * nt * kCols;
  q.cols = min(nt * kCols, d - q.begin);
  if (q.cols < 0) q.cols = 0;
  q.first = (blockIdx.x / C) * teams + q.team;
  q.step = (gridDim.x / C) * teams;
  q.count = q.first < (uint32_t)T ? (T - q.first - 1) / q.step + 1 : 0;
  return q;
}

// A chunk of W columns from shared memory.
template <int W, typename T>
__device__ __forceinline__ void get(uint32_t a, Pair* o) {
  static_assert(W * sizeof(T) == 16 || W * sizeof(T) == 8, "16 or 8 bytes a thread");
  if constexpr (sizeof(T) == 4) {
    asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(o[0]), "=l"(o[1]) : "r"(a) : "memory");
  } else if constexpr (W == 8) {
    uint32_t w[4];
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(a)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = widen<T>(w[i]);
  } else {
    uint32_t w[2];
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
    o[0] = widen<T>(w[0]);
    o[1] = widen<T>(w[1]);
  }
}

// Rounds a chunk to T and stores it; v holds the rounded values after it.
template <int W, typename T>
__device__ __forceinline__ void put(T* o, bool on, Pair* v) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const float2 a = parts(v[2 * i]), b = parts(v[2 * i + 1]);
      if (on) reinterpret_cast<float4*>(o)[i] = make_float4(a.x, a.y, b.x, b.y);
    }
  } else {
    uint32_t w[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      w[i] = narrow<T>(v[i]);
      v[i] = widen<T>(w[i]);
    }
    if constexpr (W == 8) {
      if (on) *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      if (on) *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
    }
  }
}

// The products of the gains that are given (NULL: 1), times f.
template <int W>
__device__ __forceinline__ void gains(const Place& q, int nt, const float* a, const float* b,
                                      float f, Pair* o) {
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) {
    const int c = ((2 * i / W) * nt + q.lane_t) * W + 2 * i % W;
    float2 w = make_float2(1.0f, 1.0f), z = w;
    if (a && c < q.cols) w = *reinterpret_cast<const float2*>(a + q.begin + c);
    if (b && c < q.cols) z = *reinterpret_cast<const float2*>(b + q.begin + c);
    o[i] = pair(w.x * z.x * f, w.y * z.y * f);
  }
}

// Each team has a ring of S stages of its rows' arrays, filled by bulk copies
// that its first thread starts; a stage's barrier completes when they landed.
// Columns that the row does not have stay the zeros they are set to here.
constexpr long long kRowWait = 4000000000LL;  // cycles (~2 s)
constexpr int kMaxTeams = kNormThreads / 32;

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// A team's place in its ring.  A wait that runs out records an error once; the
// team then goes on without waiting and without new copies (every thread still
// reaches every barrier), and its first thread waits once more, again with a
// limit, for the copies that may be in flight before it leaves.
struct Ring {
  uint32_t bar;       // the stages' barriers
  int stages, s;      // s: the current stage
  uint32_t phase;
  bool ok;
  int failed_s;
  uint32_t failed_phase;
  __device__ __forceinline__ void wait(int* status) {
    if (ok && !tc::mbar_wait(bar + 8 * s, phase, nullptr, kRowWait)) {
      record_error(status, MOE_ERR_TIMEOUT);
      ok = false;
      failed_s = s;
      failed_phase = phase;
    }
  }
  __device__ __forceinline__ void next() {
    if (++s == stages) s = 0, phase ^= 1u;
  }
  __device__ __forceinline__ void drain() {
    if (ok) return;
    for (int k = 0; k < stages; ++k) {
      tc::mbar_wait(bar + 8 * failed_s, failed_phase, nullptr, kRowWait / 8);
      if (++failed_s == stages) failed_s = 0, failed_phase ^= 1u;
    }
  }
};

// Zeros in columns [cols, nt kCols) of an array's slot of element size `size`
// (the row's bytes are a multiple of 16), by the team.
__device__ __forceinline__ void zero_tail(const Place& q, int nt, uint32_t slot, int size) {
  for (int b = q.cols * size + q.lane_t * 16; b < nt * kCols * size; b += nt * 16)
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(slot + b), "r"(0) : "memory");
}

__device__ __forceinline__ void team_sync(int team, int nt) {
  if (nt == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(nt) : "memory");
}

__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}

// The exchange of a cluster's sums: a CTA's values go to every CTA of the
// cluster by stores that count on the receiver's barrier, two barriers in turn.
// (A cluster barrier instead orders the row's stores to global memory first,
// which takes longer than the sums.)
// A barrier's next use can't begin early: a CTA sends use k + 2 after it has all
// of use k + 1, and this CTA's part of that is sent after all its threads are
// past use k.  A wait that runs out records an error, once, and later ones do
// not wait; the kernel's closing cluster barrier keeps every receiver alive.
struct Exchange {
  uint32_t bar;  // of the two barriers
  bool ok;
  int* status;
  __device__ __forceinline__ void init() {
    if (threadIdx.x == 0) {
      tc::mbar_init(bar, 1);
      tc::mbar_init(bar + 8, 1);
      tc::fence_barrier_init();
    }
  }
  // bytes: that come in for this use, the CTA's own among them; one thread
  __device__ __forceinline__ void expect(int turn, uint32_t bytes) {
    tc::mbar_arrive_expect_tx(bar + 8 * turn, bytes);
  }
  // v to the CTA `to`, where slot is in this one
  __device__ __forceinline__ void send(int turn, const float* slot, int to, float v) {
    uint32_t a, b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(slot)), "r"(to));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(bar + 8 * turn), "r"(to));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(a),
                 "r"(__float_as_uint(v)), "r"(b)
                 : "memory");
  }
  __device__ __forceinline__ void wait(int turn, uint32_t phase) {
    if (!ok) return;
    const long long t0 = clock64();
    uint32_t done = 0;
    while (true) {
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(done)
          : "r"(bar + 8 * turn), "r"(phase)
          : "memory");
      if (done) return;
      if (clock64() - t0 > kRowWait) break;
    }
    record_error(status, MOE_ERR_TIMEOUT);
    ok = false;
  }
};

// ------------------------------------------------------------------- host
struct NormPlan {
  int C, nt, block, grid;
  size_t smem;
};

// bytes: of the ring per thread.  ctas: CTAs of 256 threads per SM.  Few rows
// are spread over the SMs before a CTA gets a second team.
inline NormPlan norm_plan(int T, int d, int bytes, int ctas) {
  NormPlan q;
  const int sms = sm_count(), chunks = d / 8;
  // (three CTAs, where they fill an SM's threads better, are slower: 4096 bf16 rows
  // of 6144, both norms, 56.0 us, two 48.5; of 12288 95.0 where four take 113.6,
  // but the gradients 257 and 186)
  q.C = chunks <= 2 * kNormThreads ? 1 : chunks <= 4 * kNormThreads ? 2 : 4;
  q.nt = ((chunks + 2 * q.C - 1) / (2 * q.C) + 31) / 32 * 32;
  int teams = kNormThreads / q.nt;
  const int spread = (int)(((uint32_t)T + sms - 1) / sms);  // T is at most 2^31 - 1
  if (teams > spread) teams = spread;
  q.block = teams * q.nt;
  q.smem = (size_t)bytes * q.block;
  int per_sm = kNormThreads * ctas / q.block;
  const int fit = (int)(kNormSmem / q.smem);
  if (per_sm > fit) per_sm = fit;
  const int64_t want = ((int64_t)T + teams - 1) / teams * q.C;
  const int64_t most = (int64_t)sms * per_sm / q.C * q.C;
  q.grid = (int)(want < most ? want : most);
  return q;
}

// What an instantiation keeps per device: whether its attributes are set, and the
// last plan's clusters that can run at once (block << 40 | C << 32 | clusters).
struct NormSetup {
  std::atomic<bool> configured[kMaxDevices];
  std::atomic<uint64_t> resident[kMaxDevices];
};

inline void norm_config(const NormPlan& q, cudaStream_t st, cudaLaunchConfig_t* cfg,
                        cudaLaunchAttribute* attr) {
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = dim3((unsigned)q.grid);
  cfg->blockDim = dim3((unsigned)q.block);
  cfg->dynamicSmemBytes = q.smem;
  cfg->stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = q.C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = q.C > 1 ? 2 : 1;
}

// Sets a kernel's attributes, once, and takes from the plan's grid the clusters
// that would not run at once with the others: a cluster's CTAs share a GPC, whose
// SMs they may not divide evenly, and the rows are dealt out beforehand, so a
// cluster left over would take as long again as all the others.  (4096 bf16 rows
// of 16384, both norms: 118 us, the whole grid 207, and 323 with cluster barriers
// for the sums.  CTAs of 512 threads, whose rows of 8192 need no cluster, took
// 56.8 us for those, two of 256 57.4, and the gradients 123 and 107.)
template <typename P>
int prepare_norm(void (*kernel)(P), NormSetup& set, NormPlan& q) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !device_slot(dev)) return MOE_ERR_CUDA;
  if (needs_setup(set.configured, dev)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                         (int)cudaSharedmemCarveoutMaxShared);
    mark_setup(set.configured, dev);
  }
  if (q.C == 1) return MOE_OK;
  const uint64_t key = ((uint64_t)q.block << 8 | (uint64_t)q.C) << 32;
  uint64_t known = set.resident[dev].load(std::memory_order_relaxed);
  if ((known & ~0xFFFFFFFFull) != key) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    norm_config(q, nullptr, &cfg, attr);
    cfg.gridDim = dim3((unsigned)(16 * sm_count() / q.C * q.C));
    cfg.attrs = attr + 1;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      return MOE_ERR_CUDA;
    }
    known = key | (uint64_t)n;
    set.resident[dev].store(known, std::memory_order_relaxed);
  }
  const int64_t most = (int64_t)(known & 0xFFFFFFFFull) * q.C;
  if (q.grid > most) q.grid = (int)most;
  return MOE_OK;
}

template <typename P>
int launch_norm(void (*kernel)(P), const P& p, const NormPlan& q, cudaStream_t st) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  norm_config(q, st, &cfg, attr);
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
