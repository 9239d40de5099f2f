// Products of 8-bit integer codes with a scale per token and per channel, and
// the experts built from them.
//
//   x[r][c] ~ s_x[r] q_x[r][c],  s_x = amax(row) / 127,  q = rint(x / s_x)
//   y[r][j] = s_x[r] s_w[e][j] sum_c q_x[r][c] q_w[e][j][c]     r a row of expert e
//
// The sum is an s32 sum of exact products (kind::i8 of the tensor cores), so
// it does not depend on any order; the only roundings are the conversion of
// the sum to fp32, the two scalings and the output's type.
#include "common.cuh"

namespace moe {
namespace {

// Four whole numbers to four bytes, v[0] lowest, held within +-127; a NaN (an
// infinity or a NaN over the row's scale) is 0.
__device__ __forceinline__ uint32_t pack_i8(const float* v) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= (uint32_t)(uint8_t)(int8_t)min(max(__float2int_rn(v[i]), -127), 127) << (8 * i);
  return w;
}

// Sixteen elements of a row to codes.  rint of the rounded quotient x / s: the
// product by 1 / s is within 2^-16 of that quotient (three roundings of at most
// 127.5), so only a product within 2^-12 of a tie needs the division.  `slow`:
// s is subnormal, infinite or NaN.
__device__ __forceinline__ uint4 codes16(const float* x, float s, float inv, bool slow) {
  float q[16];
  bool near = slow;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float v = x[i] * inv;
    q[i] = rintf(v);
    near |= fabsf(v - q[i]) > 0.5f - 1.0f / 4096;
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = __fdiv_rn(x[i], s);
  }
  return make_uint4(pack_i8(q), pack_i8(q + 4), pack_i8(q + 8), pack_i8(q + 12));
}

// A team of nt threads (a multiple of 32) takes a row, 16 V elements a thread, held
// in registers between the row's largest magnitude and the codes: one pass over
// the bytes, which bound it.  The magnitude is taken on the bit patterns (a NaN's are
// above infinity's), so a row with an infinity or a NaN keeps it in its scale.
// V = 0: rows too long for that, read twice by a CTA.
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
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * teams + team; r < rows; r += (int64_t)gridDim.x * teams) {
    const T* xr = x + r * cols;
    float v[V > 0 ? V : 1][16];
    uint32_t m = 0;
    if constexpr (V > 0) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = (k * nt + lane_t) * 16;
        if (c < cols) {
          load8(xr + c, v[k]);
          load8(xr + c + 8, v[k] + 8);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[k][i] = 0.0f;
        }
      }
#pragma unroll
      for (int k = 0; k < V; ++k)
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[k][i]) & 0x7FFFFFFFu);
    } else {
      for (int c = lane_t * 16; c < cols; c += nt * 16) {
        load8(xr + c, v[0]);
        load8(xr + c + 8, v[0] + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[0][i]) & 0x7FFFFFFFu);
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (nt > 32) {
      const int w0 = team * (nt / 32);
      if ((threadIdx.x & 31) == 0) largest[turn][threadIdx.x >> 5] = m;
      asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(nt) : "memory");
      for (int w = 0; w < nt / 32; ++w) m = max(m, largest[turn][w0 + w]);
      turn ^= 1;  // written again only after the next row's barrier
    }
    const float s = m ? __fdiv_rn(__uint_as_float(m), 127.0f) : 1.0f, inv = 1.0f / s;
    const bool slow = !(s >= 1.1754944e-38f && s < INFINITY);
    if constexpr (V > 0) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = (k * nt + lane_t) * 16;
        if (c < cols)
          *reinterpret_cast<uint4*>(codes + r * cols + c) = codes16(v[k], s, inv, slow);
      }
    } else {
      for (int c = lane_t * 16; c < cols; c += nt * 16) {
        load8(xr + c, v[0]);
        load8(xr + c + 8, v[0] + 8);
        *reinterpret_cast<uint4*>(codes + r * cols + c) = codes16(v[0], s, inv, slow);
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

// 127 * 128 bounds a product of codes (a code may be -128): the s32 sum of K
// of them stays in range.
constexpr int kMaxK = 131056;

bool gemm_sizes_ok(int32_t rows, int32_t G, int32_t K, int32_t n) {
  return rows >= 0 && G >= 1 && G <= 1024 && K >= 16 && K % 16 == 0 && K <= kMaxK && n >= 1 &&
         (int64_t)G * n < ((int64_t)1 << 31);
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
  TcF8 ops{{w_scale, nullptr}, x_scale, OPS_I8};
  TcSeg seg{w, (int64_t)G * n, K, 0, x, rows, K, 0};
  const int mode = y_dtype == MOE_F32 ? MODE_STORE_F32
                   : y_dtype == MOE_BF16 ? MODE_STORE_BF16 : MODE_STORE_F16;
  return tc_store(offsets, rows, G, n, &seg, 1, y, mode, n, as_stream(stream), &ops);
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
