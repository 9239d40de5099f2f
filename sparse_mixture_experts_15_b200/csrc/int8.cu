// Products of 8-bit integer codes with a scale per token and per channel, and
// the experts built from them.
//
//   x[r][c] ~ s_x[r] q_x[r][c],  s_x = amax(row) fp32(1/127),  q = rint(x / s_x)
//   (the scale is the product, which is what torch makes of a device tensor divided
//   by the number 127; a division differs in the last bit of one row in 22)
//   y[r][j] = s_x[r] s_w[e][j] sum_c q_x[r][c] q_w[e][j][c]     r a row of expert e
//
// The sum is an s32 sum of exact products (kind::i8 of the tensor cores), so
// it does not depend on any order; the only roundings are the conversion of
// the sum to fp32, the two scalings and the output's type.
#include "common.cuh"
#include "pairs.cuh"
#include "tc_primitives.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------- quantiser
// Sixteen elements of a row as they are stored: 2 (16-bit) or 4 (fp32) times
// 16 bytes.
template <typename T>
struct Raw {
  static constexpr int N = sizeof(T) == 4 ? 4 : 2;
  uint4 w[N];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  // The largest magnitude as the bits of its fp32 value, at least m.  Magnitudes
  // are compared as bit patterns, where a NaN's is above infinity's.
  __device__ __forceinline__ uint32_t largest(uint32_t m) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        m = max(m, max(w[i].x & 0x7FFFFFFFu, w[i].y & 0x7FFFFFFFu));
        m = max(m, max(w[i].z & 0x7FFFFFFFu, w[i].w & 0x7FFFFFFFu));
      }
      return m;
    } else {
      uint32_t h = 0;  // two 16-bit maxima
#pragma unroll
      for (int i = 0; i < N; ++i) {
        h = __vmaxu2(h, __vmaxu2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu));
        h = __vmaxu2(h, __vmaxu2(w[i].z & 0x7FFF7FFFu, w[i].w & 0x7FFF7FFFu));
      }
      const uint16_t t = (uint16_t)max(h & 0xFFFFu, h >> 16);
      return max(m, __float_as_uint(to_f32(*reinterpret_cast<const T*>(&t))));
    }
  }
  __device__ __forceinline__ void values(float* v) const {
#pragma unroll
    for (int i = 0; i < 16; i += 8)
      load8(reinterpret_cast<const T*>(w) + i, v + i);
  }
};

// Four elements to codes, rint of the rounded quotient x / s.  The product
// by 1 / s is within 2^-15 of that quotient (three roundings of half a step at
// most, 2^-24 of values up to 127.5), so only a product within 2^-14 of a tie
// needs the division.  Rounding is by
// adding 1.5 2^23, which leaves the whole number in the low byte; within a row of
// a normal scale no quotient rounds above 127.  `slow`: s is subnormal, infinite
// or NaN; codes are then held within +-127, and a NaN (an infinity or a NaN over
// the scale) is 0.
__device__ __forceinline__ uint32_t codes4(const float* x, float s, float inv, bool slow) {
  constexpr float kRound = 12582912.0f;
  uint32_t q[4];
  float off = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const Pair v = mul2(pair(x[i], x[i + 1]), pair(inv, inv)), r = add2(v, pair(kRound, kRound));
    const float2 w = parts(r);
    q[i] = __float_as_uint(w.x);
    q[i + 1] = __float_as_uint(w.y);
    const float2 d = parts(fma2(add2(r, pair(-kRound, -kRound)), pair(-1.0f, -1.0f), v));
    off = fmaxf(off, fmaxf(fabsf(d.x), fabsf(d.y)));
  }
  if (slow || off > 0.5f - 1.0f / 16384) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = (uint32_t)min(max(__float2int_rn(__fdiv_rn(x[i], s)), -127), 127);
  }
  return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
}
__device__ __forceinline__ uint4 codes16(const float* x, float s, float inv, bool slow) {
  return make_uint4(codes4(x, s, inv, slow), codes4(x + 4, s, inv, slow),
                    codes4(x + 8, s, inv, slow), codes4(x + 12, s, inv, slow));
}

// A team of nt threads (a multiple of 32) takes a row, 16 V elements a thread, held
// as stored between the row's largest magnitude and the codes, with the next
// row's loads in flight: one pass over the bytes (16384 x 4096 bf16 41 us, of which
// the bytes are 31; fp32 62 and 51).  A row with an infinity or a NaN keeps it in
// its scale.  V = 0: rows too long for that, read twice by a CTA (1024 x 32768
// bf16 31 us, the bytes once 15).
constexpr int kQuantThreads = 256;

template <typename T, int V>
__global__ void __launch_bounds__(kQuantThreads)
    quant_rows_i8(const T* __restrict__ x, int64_t rows, const int32_t* __restrict__ rows_dev,
                  int cols, int nt, int8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ uint32_t largest[2][kQuantThreads / 32];
  pdl_wait();
  pdl_allow_next();
  if (rows_dev) rows = min(rows, (int64_t)max(*rows_dev, 0));
  const int team = threadIdx.x / nt, lane_t = threadIdx.x - team * nt, teams = blockDim.x / nt;
  constexpr int H = V > 0 ? V : 1;
  Raw<T> now[H], next[H];
  const int64_t step = (int64_t)gridDim.x * teams;
  int64_t r = (int64_t)blockIdx.x * teams + team;
  const T* src = x + r * cols + lane_t * 16;  // the next row to fetch
  auto fetch = [&](int64_t row, Raw<T>* o) {
#pragma unroll
    for (int k = 0; k < H; ++k) {
      if (row < rows && (k * nt + lane_t) * 16 < cols) o[k].load(src + k * nt * 16);
      else o[k].zero();
    }
    src += step * cols;
  };
  if (V > 0) fetch(r, next);
  int turn = 0;
  for (; r < rows; r += step) {
    uint32_t m = 0;
    if constexpr (V > 0) {
#pragma unroll
      for (int k = 0; k < H; ++k) now[k] = next[k];
      fetch(r + step, next);
#pragma unroll
      for (int k = 0; k < H; ++k) m = now[k].largest(m);
    } else {
      for (int c = lane_t * 16; c < cols; c += nt * 16) {
        now[0].load(x + r * cols + c);
        m = now[0].largest(m);
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (nt > 32) {
      const int w0 = team * (nt / 32);
      if ((threadIdx.x & 31) == 0) largest[turn][threadIdx.x >> 5] = m;
      asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(nt) : "memory");
      const int lane = threadIdx.x & 31;
      m = __reduce_max_sync(0xffffffffu, lane < nt / 32 ? largest[turn][w0 + lane] : 0u);
      turn ^= 1;  // written again only after the next row's barrier
    }
    const float s = m ? __fmul_rn(__uint_as_float(m), 1.0f / 127.0f) : 1.0f, inv = 1.0f / s;
    const bool slow = !(s >= 1.1754944e-38f && s < INFINITY);
    float v[16];
    if constexpr (V > 0) {
#pragma unroll
      for (int k = 0; k < H; ++k) {
        const int c = (k * nt + lane_t) * 16;
        now[k].values(v);
        if (c < cols) *reinterpret_cast<uint4*>(codes + r * cols + c) = codes16(v, s, inv, slow);
      }
    } else {
      for (int c = lane_t * 16; c < cols; c += nt * 16) {
        now[0].load(x + r * cols + c);
        now[0].values(v);
        *reinterpret_cast<uint4*>(codes + r * cols + c) = codes16(v, s, inv, slow);
      }
    }
    if (lane_t == 0) scales[r] = s;
  }
}

int quantize(int64_t rows, const int32_t* rows_dev, int cols, const void* x, int32_t x_dtype,
             int8_t* codes, float* scales, cudaStream_t st) {
  if (rows == 0) return MOE_OK;
  const int pieces = cols / 16;
  const int V = pieces <= kQuantThreads ? 1 : pieces <= 2 * kQuantThreads ? 2
                : pieces <= 4 * kQuantThreads ? 4 : 0;
  const int per = V ? (pieces + V - 1) / V : kQuantThreads;
  const int nt = (per + 31) / 32 * 32, sms = sm_count();
  int teams = kQuantThreads / nt;
  if (teams > (rows + sms - 1) / sms) teams = (int)((rows + sms - 1) / sms);
  int64_t grid = (rows + teams - 1) / teams;
  if (grid > (int64_t)sms * 16) grid = (int64_t)sms * 16;
#define MOE_QUANT(T, V)                                                                       \
  do {                                                                                        \
    MOE_PREFER_SHARED((quant_rows_i8<T, V>));                                                 \
    launch_pdl(quant_rows_i8<T, V>, dim3((unsigned)grid), dim3((unsigned)(teams * nt)), 0,    \
               st, static_cast<const T*>(x), rows, rows_dev, cols, nt, codes, scales);        \
  } while (0)
#define MOE_QUANT_V(T)           \
  do {                           \
    if (V == 1) MOE_QUANT(T, 1); \
    else if (V == 2) MOE_QUANT(T, 2); \
    else if (V == 4) MOE_QUANT(T, 4); \
    else MOE_QUANT(T, 0);        \
  } while (0)
  if (x_dtype == MOE_F32) MOE_QUANT_V(float);
  else if (x_dtype == MOE_BF16) MOE_QUANT_V(__nv_bfloat16);
  else MOE_QUANT_V(__half);
#undef MOE_QUANT_V
#undef MOE_QUANT
  return launch_status();
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// 128 * 128 bounds a product of codes (a code may be -128): the s32 sum of K
// of them stays in range.
constexpr int kMaxK = 131056;

bool gemm_sizes_ok(int32_t rows, int32_t G, int32_t K, int32_t n) {
  return rows >= 0 && G >= 1 && G <= 1024 && K >= 16 && K % 16 == 0 && K <= kMaxK && n >= 1 &&
         (int64_t)G * n < ((int64_t)1 << 31);
}

// -------------------------------------------------------------- few rows
// The product for at most 2 rows in all, bound by the weights' bytes: each warp
// streams whole weight rows, 16 bytes a lane, four channels at once, and forms
// four products an instruction (dp4a) with the token rows, which the CTA holds in
// shared memory; a channel's sum is one integer reduction of the warp.  The
// channels of the groups that have rows are dealt to the CTAs (one per SM) and
// their warps in equal shares.  With one group a CTA knows its share at once and
// starts its fetch to L2 before it waits for the previous kernel (a fetch to L2
// holds nothing that could grow stale).  Rows x 4096 -> 14336 in us, here and with
// the tensor cores: 1 row 11.7 and 14.4, 2 rows 11.9 and 14.4 (4 rows: 15.0 and 14.8).
constexpr int kFewRows = 2, kFewThreads = 1024, kFewSmem = 200 * 1024;

struct FewParams {
  int rows, G, K, n;
  const int8_t *x, *w;
  const float *x_scale, *w_scale;
  const int32_t* offsets;
  void* y;
  int* status;
};

__device__ __forceinline__ uint4 stream16(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ int dot16(uint4 a, uint4 b, int c) {
  c = __dp4a((int)a.x, (int)b.x, c);
  c = __dp4a((int)a.y, (int)b.y, c);
  c = __dp4a((int)a.z, (int)b.z, c);
  return __dp4a((int)a.w, (int)b.w, c);
}

// Channels ch .. ch + nch - 1 (nch <= 4) of one group for its R rows, in xs [R][K].
template <int R, typename TY>
__device__ __forceinline__ void few_dots(const FewParams& p, int g, int ch, int nch, int row0,
                                         const int8_t* xs) {
  const int lane = threadIdx.x & 31;
  const int8_t* w[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) w[c] = p.w + ((size_t)g * p.n + ch + min(c, nch - 1)) * p.K;
  int acc[4][R];
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int r = 0; r < R; ++r) acc[c][r] = 0;
  for (int k = lane * 16; k < p.K; k += 512) {
    uint4 v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = c < nch ? stream16(w[c] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint4 x = *reinterpret_cast<const uint4*>(xs + (size_t)r * p.K + k);
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c][r] = dot16(v[c], x, acc[c][r]);
    }
  }
  __syncwarp();
  int mine = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int s = __reduce_add_sync(0xffffffffu, acc[c][r]);
      if (lane == c * R + r) mine = s;
    }
  const int c = lane / R, r = lane % R;
  if (c < nch)
    static_cast<TY*>(p.y)[(size_t)(row0 + r) * p.n + ch + c] = from_f32<TY>(
        __int2float_rn(mine) * p.w_scale[(size_t)g * p.n + ch + c] * p.x_scale[row0 + r]);
}

template <typename TY>
__global__ void __launch_bounds__(kFewThreads, 1) i8_few_rows(const __grid_constant__ FewParams p) {
  extern __shared__ __align__(16) int8_t xs[];  // [rows of a group][K]
  __shared__ int grp[kFewRows], beg[kFewRows], cnt[kFewRows], groups;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (p.G == 1) {
    const int64_t lo = (int64_t)p.n * blockIdx.x / gridDim.x;
    const int64_t hi = (int64_t)p.n * (blockIdx.x + 1) / gridDim.x;
    for (int64_t c = lo + tid; c < hi; c += kFewThreads) tc::l2_prefetch(p.w + c * p.K, p.K);
  }
  pdl_wait();
  pdl_allow_next();
  if (warp == 0) {  // the groups that have rows: at most p.rows of them, in order
    int found = 0;
    for (int base = 0; base < p.G; base += 32) {
      const int g = base + lane;
      int b = 0, c = 0;
      if (g < p.G) {
        b = p.offsets ? p.offsets[g] : 0;
        c = (p.offsets ? p.offsets[g + 1] : p.rows) - b;
        if (c < 0 || b < 0 || b > p.rows || c > p.rows - b) {  // rows outside the buffers
          record_error(p.status, MOE_ERR_BOUNDS);
          c = 0;
        }
      }
      const uint32_t some = __ballot_sync(0xffffffffu, c > 0);
      const int at = found + __popc(some & ((1u << lane) - 1));
      // offsets that run back and forth could name more groups than there are rows
      if (c > 0 && at < kFewRows) grp[at] = g, beg[at] = b, cnt[at] = c;
      found += __popc(some);
    }
    if (lane == 0) {
      if (found > kFewRows) record_error(p.status, MOE_ERR_BOUNDS);
      groups = min(found, kFewRows);
    }
  }
  __syncthreads();
  const int64_t all = (int64_t)groups * p.n;
  int64_t at = all * blockIdx.x / gridDim.x;
  const int64_t end = all * (blockIdx.x + 1) / gridDim.x;
  while (at < end) {
    const int a = (int)(at / p.n), ch0 = (int)(at - (int64_t)a * p.n);
    const int seg = (int)min((int64_t)(p.n - ch0), end - at);
    const int rows = cnt[a], row0 = beg[a];
    __syncthreads();  // the last segment's rows are no longer read
    for (int i = tid; i < rows * (p.K / 16); i += kFewThreads)
      reinterpret_cast<uint4*>(xs)[i] =
          reinterpret_cast<const uint4*>(p.x + (size_t)row0 * p.K)[i];
    __syncthreads();
    constexpr int W = kFewThreads / 32;
    const int lo = ch0 + (int)((int64_t)seg * warp / W);
    const int hi = ch0 + (int)((int64_t)seg * (warp + 1) / W);
    for (int ch = lo; ch < hi; ch += 4) {
      const int nch = min(4, hi - ch);
      if (rows == 1) few_dots<1, TY>(p, grp[a], ch, nch, row0, xs);
      else few_dots<2, TY>(p, grp[a], ch, nch, row0, xs);
    }
    at += seg;
  }
}

// Shared memory of i8_few_rows, or 0 where it does not fit.
size_t few_smem(int rows, int K) {
  if (rows > kFewRows) return 0;
  const size_t b = (size_t)rows * K;
  return b <= kFewSmem ? b : 0;
}

template <typename TY>
int launch_few(const FewParams& p, size_t smem, cudaStream_t st) {
  static std::atomic<bool> configured[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !device_slot(dev)) return MOE_ERR_CUDA;
  if (needs_setup(configured, dev)) {
    if (cudaFuncSetAttribute(i8_few_rows<TY>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kFewSmem) != cudaSuccess)
      return MOE_ERR_CUDA;
    mark_setup(configured, dev);
  }
  MOE_PREFER_SHARED((i8_few_rows<TY>));
  launch_pdl(i8_few_rows<TY>, dim3((unsigned)sm_count()), dim3(kFewThreads), smem, st, p);
  return launch_status();
}

}  // namespace
}  // namespace moe

extern "C" int moe_quantize_i8_rows(int64_t rows, int32_t cols, const void* x, int32_t x_dtype,
                                    int8_t* codes, float* scales, void* stream) {
  using namespace moe;
  if (rows < 0 || cols <= 0 || cols % 16 != 0) return MOE_ERR_INVALID_ARG;
  if (!valid_act_dtype(x_dtype)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned4(scales))
    return MOE_ERR_INVALID_ARG;
  return quantize(rows, nullptr, cols, x, x_dtype, codes, scales, as_stream(stream));
}

extern "C" size_t moe_grouped_gemm_i8_workspace_bytes(int32_t rows, int32_t G, int32_t K,
                                                      int32_t n) {
  (void)rows, (void)G, (void)K, (void)n;
  return 0;
}

extern "C" int moe_grouped_gemm_i8(int32_t rows, int32_t G, int32_t K, int32_t n, const int8_t* x,
                                   const float* x_scale, const int32_t* offsets, const int8_t* w,
                                   const float* w_scale, void* y, int32_t y_dtype, void* ws,
                                   size_t ws_bytes, void* stream) {
  using namespace moe;
  if (!gemm_sizes_ok(rows, G, K, n) || (!offsets && G != 1)) return MOE_ERR_INVALID_ARG;
  if (!valid_act_dtype(y_dtype)) return MOE_ERR_UNSUPPORTED;
  if (!w || !w_scale || !aligned16(w) || !aligned4(w_scale) || !aligned4(offsets))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!x || !x_scale || !y || !aligned16(x) || !aligned4(x_scale) || !aligned16(y))
    return MOE_ERR_INVALID_ARG;
  (void)ws, (void)ws_bytes;
  cudaStream_t st = as_stream(stream);
  if (const size_t smem = few_smem(rows, K)) {
    const FewParams p{rows, G, K, n, x, w, x_scale, w_scale, offsets, y, status_word()};
    return y_dtype == MOE_F32    ? launch_few<float>(p, smem, st)
           : y_dtype == MOE_BF16 ? launch_few<__nv_bfloat16>(p, smem, st)
                                 : launch_few<__half>(p, smem, st);
  }
  TcF8 ops{{w_scale, nullptr}, x_scale, OPS_I8};
  TcSeg seg{w, (int64_t)G * n, K, 0, x, rows, K, 0};
  const int mode = y_dtype == MOE_F32 ? MODE_STORE_F32
                   : y_dtype == MOE_BF16 ? MODE_STORE_BF16 : MODE_STORE_F16;
  return tc_store(offsets, rows, G, n, &seg, 1, y, mode, n, st, &ops);
}

// H bf16 [T*k][h], its codes [T*k][h] and their row scales [T*k]
static size_t ffn_i8_carve(const moe_shape& s, void* ws, void** H, int8_t** codes, float** scale) {
  moe::Carver c(ws);
  const size_t R = (size_t)s.T * s.k;
  *H = c.take<uint16_t>(R * s.h);
  *codes = c.take<int8_t>(R * s.h);
  *scale = c.take<float>(R);
  return c.used();
}

extern "C" size_t moe_expert_ffn_i8_workspace_bytes(const moe_shape* shape) {
  if (!moe::shape_ok(shape) || shape->h <= 0) return 0;
  void* H;
  int8_t* codes;
  float* scale;
  return ffn_i8_carve(*shape, nullptr, &H, &codes, &scale);
}

extern "C" int moe_expert_ffn_i8(const moe_shape* shape, int32_t width, const int8_t* x_rows,
                                 const float* x_scale, const int32_t* offsets,
                                 const int8_t* w_gate, const int8_t* w_up, const int8_t* w_down,
                                 const moe_i8_scales* scales, const moe_act* act, float* y_rows,
                                 void* ws, size_t ws_bytes, void* stream) {
  using namespace moe;
  if (!shape_ok(shape) || !act || !scales || !offsets || !w_gate || !w_up || !w_down)
    return MOE_ERR_INVALID_ARG;
  const moe_shape& s = *shape;
  if (width <= 0 || width % 128 != 0 || s.h <= 0 || s.h % 128 != 0 || width > kMaxK || s.h > kMaxK)
    return MOE_ERR_UNSUPPORTED;
  if ((int64_t)s.N * s.h >= (int64_t)1 << 31 || (int64_t)s.N * width >= (int64_t)1 << 31)
    return MOE_ERR_UNSUPPORTED;
  if (act->kind != MOE_ACT_SWIGLU &&
      !(act->kind == MOE_ACT_SITU_GLU && act->beta_gate > 0.0f && act->beta_up > 0.0f))
    return MOE_ERR_INVALID_ARG;
  if (!scales->gate_scale || !scales->up_scale || !scales->down_scale) return MOE_ERR_INVALID_ARG;
  if (s.T > 0 && (!x_rows || !x_scale || !y_rows)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x_rows) || !aligned16(w_gate) || !aligned16(w_up) || !aligned16(w_down) ||
      !aligned16(y_rows) || !aligned16(ws))
    return MOE_ERR_INVALID_ARG;
  void* H;
  int8_t* codes;
  float* scale;
  const size_t need = ffn_i8_carve(s, ws, &H, &codes, &scale);
  if (s.T == 0) return MOE_OK;
  if (!ws || ws_bytes < need) return MOE_ERR_WORKSPACE;
  const int64_t R = (int64_t)s.T * s.k;
  cudaStream_t st = as_stream(stream);
  TcF8 gu{{scales->gate_scale, scales->up_scale}, x_scale, OPS_I8};
  int rc = tc_gateup(offsets, (int)R, s.N, x_rows, R, width, w_gate, w_up, s.h, *act, H, s.h, 0,
                     st, &gu);
  // H has one scale per row, known only once the row is whole, so it is stored
  // between the products: as bf16, whose rounding (2^-9 of a value) is below
  // the 8-bit code's (2^-8 of the row's largest) wherever the code is large
  if (rc == MOE_OK) rc = quantize(R, offsets + s.N, s.h, H, MOE_BF16, codes, scale, st);
  if (rc != MOE_OK) return rc;
  TcF8 dn{{scales->down_scale, nullptr}, scale, OPS_I8};
  TcSeg seg{w_down, (int64_t)s.N * width, s.h, 0, codes, R, s.h, 0};
  return tc_store(offsets, (int)R, s.N, width, &seg, 1, y_rows, MODE_STORE_F32, width, st, &dn);
}
