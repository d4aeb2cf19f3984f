// e4m3 codes with one fp32 scale per block of 128 columns, on gfx950: the
// operands of the 8-bit block-scaled products.
//
//   s = max(amax(block) / 448, 2^-126),  code = e4m3(y / s)
//
// 448 is the largest e4m3 value, so every block uses the whole range; the
// floor keeps 1 / s finite and gives an all-zero block zero codes.  amax is
// taken on the bits of |y| as unsigned integers, where a NaN is larger than
// everything: a block that holds a NaN or an infinity gets that as its scale
// and dequantises to NaN throughout, it does not pass for a number.  Everything
// is fp32 until the one rounding to e4m3.
//
// Blocks are 1 x 128 (activations) or 128 x 128 (weights); y is x itself,
// silu(gate) * up of rows [gate | up], or the residual sum's RMS norm.
//
// Rows are cut into units of 512 columns, one wavefront pass each: a lane has 8
// consecutive columns, 16 lanes share a block, and a unit's four scales are one
// 16-byte piece of the scale row (scale rows are padded to 4 columns).
#include "common.hpp"

namespace mi {
namespace {

constexpr float F8Q_MAX = 448.f;
constexpr float F8Q_MIN_SCALE = 1.17549435e-38f;  // 2^-126

template <typename T>
struct Vec8 {  // 8 consecutive elements of a 16-bit type
  u32x4 v;
  __device__ void load(const T* p) { v = gld<u32x4>(p); }
  __device__ void zero() { v = u32x4{0, 0, 0, 0}; }
  __device__ float get(int i) const {
    const uint32_t w = v[i >> 1];
    if constexpr (std::is_same<T, __bf16>::value)
      return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
    else
      return static_cast<float>(
          __builtin_bit_cast(_Float16, static_cast<uint16_t>((i & 1) ? (w >> 16) : (w & 0xffff))));
  }
};
template <>
struct Vec8<float> {
  f32x4 a, b;
  __device__ void load(const float* p) {
    a = gld<f32x4>(p);
    b = gld<f32x4>(p + 4);
  }
  __device__ void zero() { a = b = f32x4{0.f, 0.f, 0.f, 0.f}; }
  __device__ float get(int i) const { return i < 4 ? a[i] : b[i - 4]; }
};

// 8 floats rounded once to T
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* y) {
  if constexpr (sizeof(T) == 4) {
    gst<f32x4>(p, f32x4{y[0], y[1], y[2], y[3]});
    gst<f32x4>(p + 4, f32x4{y[4], y[5], y[6], y[7]});
  } else {
    typedef T t8 __attribute__((ext_vector_type(8)));
    typedef float f8 __attribute__((ext_vector_type(8)));
    const f8 v = {y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]};
    gst<t8>(p, __builtin_convertvector(v, t8));
  }
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t amax8(const float* y) {
  uint32_t m = abs_bits(y[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max(m, abs_bits(y[i]));
  return m;
}

// silu(g) = g E' / (1 + E) with E = exp(-|g|) in [0, 1] and E' = 1 or, below zero, E:
// nothing overflows.  E = 2^t e^r with t = fl(-|g| log2 e) and the rest r = -|g| - t ln 2
// from the fma and ln 2's own rest; |r| < 2^-16, so e^r is 1 + r.  Without r the result
// would be off by |g| half steps at a negative gate (65 at -85).  2^24 E is what is
// computed, as v_exp gives zero for a subnormal result; the 24 is rounded into t before
// r is taken (t + 24 - 24 is exact for what is left), so nothing may be contracted
// here.  Past -150 E is zero, and an infinite gate below zero gives NaN.
// 1 / (1 + E) is v_rcp and one Newton step.  At most 7 roundings, 9 with up and the
// scale's division.  65536 x 2048 of bf16 rows [gate | up], VALU and memory close to
// each other: 127 us; a bare exp and full divisions 128, expf and full divisions 13% more.
__device__ __forceinline__ float silu(float g) {
#pragma clang fp contract(off)
  constexpr float L = 1.44269502f, LN2 = 0.693147182f, REST = -1.90465430e-9f, UP = 0x1p-24f;
  const float v = __builtin_amdgcn_fmed3f(-fabsf(g), -150.f, 0.f);
  const float t = v * L + 24.f, u = 24.f - t;
  const float r = __builtin_fmaf(u, REST, __builtin_fmaf(u, LN2, v));
  const float p = __builtin_amdgcn_exp2f(t);
  const float e = __builtin_fmaf(p, r, p);
  const float d = __builtin_fmaf(e, UP, 1.f), q = __builtin_amdgcn_rcpf(d);
  return (g >= 0.f ? g : g * e * UP) * __builtin_fmaf(__builtin_fmaf(-d, q, 1.f), q, q);
}

// The quotient a / b from inv, 1 / b to a step: one correction by the exact remainder,
// which then rounds as a division does (3 operations where a division has 11; 448 was
// tried with every mantissa of a)
__device__ __forceinline__ float quotient(float a, float b, float inv) {
  const float q = a * inv;
  return __builtin_fmaf(__builtin_fmaf(q, -b, a), inv, q);
}

// the scale of a block from its amax bits; a NaN stays a NaN, an infinity itself
__device__ __forceinline__ float block_scale(uint32_t m) {
  const float a = __uint_as_float(m);
  const float s = m < 0x7f800000u ? quotient(a, F8Q_MAX, 1.f / F8Q_MAX) : a;
  return s < F8Q_MIN_SCALE ? F8Q_MIN_SCALE : s;
}

// The codes of y / s.  Without the quotients' correction a value within two roundings of
// a tie between two codes may take the wrong one (8 x 2000 x 4112 of fp32: 2.1e-5 of the
// codes' rms against 2.3e-6).
__device__ __forceinline__ u32x2 codes8(const float* y, float s) {
  const float rcp = __builtin_amdgcn_rcpf(s);  // good to a step, and a Newton step on it
  float inv = __builtin_fmaf(__builtin_fmaf(-s, rcp, 1.f), rcp, rcp);
  // an infinite scale has no remainder: numbers get code 0, infinities NaN
  const bool inf = s == __builtin_inff();
  if (inf) inv = 0.f;
  const float d = inf ? 0.f : s;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = quotient(y[i], d, inv);
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return u32x2{static_cast<uint32_t>(lo), static_cast<uint32_t>(hi)};
}

// Quantises this lane's 8 values at column `col` (a multiple of 8) of a row of
// k columns; all 64 lanes of a unit call it, with zeros past k.
__device__ __forceinline__ void quantise_unit(const float* y, int col, int k, uint8_t* codes_row,
                                              float* scales_row) {
  uint32_t m = amax8(y);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o, 64)));
  const float s = block_scale(m);
  if (col < k) gst<u32x2>(codes_row + col, codes8(y, s));
  // padding columns of the scale row are zero
  if ((col & 127) == 0) gst<float>(scales_row + (col >> 7), col < k ? s : 0.f);
}

// 1 x 128 blocks: a wavefront per unit.  Bound by memory: x is read once with
// 16-byte loads (fp32: two), and a block's amax takes 4 exchanges among its 16
// lanes, no LDS and no barrier.  65536 x 2048 of bf16 [gate | up]: 675 MB in
// 127 to 131 us by card, 5.2 TB/s, the rate of a large copy.
template <typename T, bool GLU>
__global__ __launch_bounds__(256) void f8_rows_kernel(const T* __restrict__ x, int64_t units,
                                                      int k, int upr, uint8_t* __restrict__ codes,
                                                      float* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int64_t nw = static_cast<int64_t>(gridDim.x) * 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + wave; u < units; u += nw) {
    const int64_t row = u / upr;
    const int col = static_cast<int>(u - row * upr) * 512 + lane * 8;
    Vec8<T> a, b;
    if (col < k) {
      const T* px = x + row * (GLU ? 2 * static_cast<int64_t>(k) : k) + col;
      a.load(px);
      if constexpr (GLU) b.load(px + k);
    } else {
      a.zero();
      if constexpr (GLU) b.zero();
    }
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = a.get(i);
      if constexpr (GLU) y[i] = silu(y[i]) * b.get(i);
    }
    quantise_unit(y, col, k, codes + row * k, scales + row * (4 * upr));
  }
}

// One 128 x 128 block per workgroup: thread (tid / 16, tid % 16) has 8 columns
// of 8 rows, 16 rows apart, in registers between the reduction and the codes, so
// x is read once.  Bound by memory: 8 x 2000 x 4112 of fp32, 329 MB in 64.5 us,
// 5.1 TB/s, the rate of a large copy.
template <typename T>
__global__ __launch_bounds__(256) void f8_blocks_kernel(const T* __restrict__ x, int64_t blocks,
                                                        int rows, int k, int sc, int nb, int kb,
                                                        uint8_t* __restrict__ codes,
                                                        float* __restrict__ scales) {
  __shared__ uint32_t s_max[4];
  // workgroup ids go to the 8 XCDs in turn: each XCD gets a contiguous run of
  // blocks, so that its L2 joins the lines two neighbours write parts of
  const int64_t total = blocks / 8 * 8, per_xcd = total / 8;
  const int64_t id = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
  if (id >= blocks) return;
  const int64_t blk = id < total ? (id & 7) * per_xcd + (id >> 3) : id;
  const int cb = static_cast<int>(blk % kb);
  const int64_t rest = blk / kb;
  const int rb = static_cast<int>(rest % nb);
  const int64_t batch = rest / nb;
  const int col = cb * 128 + (threadIdx.x & 15) * 8;
  const int row0 = rb * 128 + (threadIdx.x >> 4);
  const int64_t base = batch * rows * static_cast<int64_t>(k);
  Vec8<T> v[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + 16 * i;
    if (row < rows && col < k) v[i].load(x + base + static_cast<int64_t>(row) * k + col);
    else v[i].zero();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int c = 0; c < 8; ++c) m = max(m, abs_bits(v[i].get(c)));
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o, 64)));
  if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
  const float s = block_scale(m);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + 16 * i;
    if (row >= rows || col >= k) continue;
    float y[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) y[c] = v[i].get(c);
    gst<u32x2>(codes + base + static_cast<int64_t>(row) * k + col, codes8(y, s));
  }
  if (threadIdx.x == 0) {
    float* srow = scales + (batch * nb + rb) * sc;
    gst<float>(srow + cb, s);
    if (cb == kb - 1)
      for (int c = kb; c < sc; ++c) gst<float>(srow + c, 0.f);
  }
}

// h = x (+ r), y = h / sqrt(mean(h^2) + eps) * w, one workgroup per row.  h
// stays in fp32 for the norm and is rounded once for the stored stream.  NC > 0:
// the row's NC units per wavefront are kept in registers between the sum of
// squares and the output; NC == 0: any length, x and r are read again (before
// this thread overwrites its own part of the stream, which may be r itself).
// One workgroup per row also where rows are few: the row's sum is then one barrier
// away (one token of 4096: 3.2 us, the latency of a launch and two dependent passes
// over the registers).  Many rows are bound by memory: 8192 x 7168 of bf16 with
// both streams and y itself, 530 MB in 104 us, 5.1 TB/s, the rate of a large copy.
// A row of up to 8192 values stays in registers; longer ones are read twice, the
// second time mostly from L2.
template <typename T, int NC>
__global__ __launch_bounds__(256) void rmsnorm_f8_kernel(const T* x, const T* r,
                                                         const void* __restrict__ w, bool w_f32,
                                                         int t, int h, int upr, float eps, T* res_out,
                                                         T* norm_out, uint8_t* __restrict__ codes,
                                                         float* __restrict__ scales) {
  __shared__ float s_sum[4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
  if (row >= t) return;
  x += row * h;
  if (r != nullptr) r += row * h;
  auto load_h = [&](int col, float* y) {
    Vec8<T> a, b;
    a.zero();
    b.zero();
    if (col < h) {
      a.load(x + col);
      if (r != nullptr) b.load(r + col);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = a.get(i) + b.get(i);
  };
  float keep[NC > 0 ? NC : 1][8];
  float ss = 0.f;
  const int nc = NC > 0 ? NC : (upr + 3) / 4;
#pragma unroll NC > 0 ? NC : 1
  for (int c = 0; c < nc; ++c) {
    float* y = keep[NC > 0 ? c : 0];
    load_h((c * 4 + wave) * 512 + lane * 8, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(y[i], y[i], ss);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) ss += __shfl_xor(ss, o, 64);
  if (lane == 0) s_sum[wave] = ss;
  __syncthreads();
  ss = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
  const float rstd = __fdiv_rn(1.f, __fsqrt_rn(ss / static_cast<float>(h) + eps));
  codes += row * h;
  scales += row * (4 * upr);
#pragma unroll NC > 0 ? NC : 1
  for (int c = 0; c < nc; ++c) {
    const int unit = c * 4 + wave, col = unit * 512 + lane * 8;
    if (unit >= upr) break;
    float* y = keep[NC > 0 ? c : 0];
    if constexpr (NC == 0) load_h(col, y);
    float wv[8];
    if (w_f32) {
      Vec8<float> t;
      t.zero();
      if (col < h) t.load(static_cast<const float*>(w) + col);
#pragma unroll
      for (int i = 0; i < 8; ++i) wv[i] = t.get(i);
    } else {
      Vec8<T> t;
      t.zero();
      if (col < h) t.load(static_cast<const T*>(w) + col);
#pragma unroll
      for (int i = 0; i < 8; ++i) wv[i] = t.get(i);
    }
    if (res_out != nullptr && col < h) store8<T>(res_out + row * h + col, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = y[i] * rstd * wv[i];
    if (norm_out != nullptr && col < h) store8<T>(norm_out + row * h + col, y);
    quantise_unit(y, col, h, codes, scales);
  }
}

// A workgroup each: a launch has fewer than 2^32 threads per dimension
dim3 f8q_grid(int64_t n) {
  constexpr int64_t X = 1 << 20;
  return n <= X ? dim3(static_cast<unsigned>(n))
                : dim3(static_cast<unsigned>(X), static_cast<unsigned>((n + X - 1) / X));
}

int64_t f8_units(int64_t k) { return (k + 511) / 512; }

template <typename T>
mi_status launch_quantize(const void* x, int64_t batch, int64_t rows, int64_t k, int block_rows,
                          bool glu, uint8_t* codes, float* scales, hipStream_t s) {
  const T* xp = static_cast<const T*>(x);
  const int upr = static_cast<int>(f8_units(k)), ki = static_cast<int>(k);
  if (block_rows == 1) {
    const int64_t units = batch * rows * upr;
    int64_t blocks = (units + 3) / 4;
    if (blocks > 8192) blocks = 8192;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (glu)
      hipLaunchKernelGGL((f8_rows_kernel<T, true>), grid, dim3(256), 0, s, xp, units, ki, upr,
                         codes, scales);
    else
      hipLaunchKernelGGL((f8_rows_kernel<T, false>), grid, dim3(256), 0, s, xp, units, ki, upr,
                         codes, scales);
  } else {
    const int64_t nb = (rows + 127) / 128, kb = (k + 127) / 128;
    hipLaunchKernelGGL((f8_blocks_kernel<T>), f8q_grid(batch * nb * kb), dim3(256), 0, s, xp,
                       batch * nb * kb, static_cast<int>(rows), ki, 4 * upr,
                       static_cast<int>(nb), static_cast<int>(kb), codes, scales);
  }
  return launch_status("fp8_quantize");
}

template <typename T>
mi_status launch_norm(const void* x, const void* r, const void* w, bool w_f32, int64_t t,
                      int64_t h, float eps, void* res_out, void* norm_out, uint8_t* codes,
                      float* scales, hipStream_t s) {
  const int upr = static_cast<int>(f8_units(h));
#define MI_NORM_LAUNCH(NC_)                                                                     \
  hipLaunchKernelGGL((rmsnorm_f8_kernel<T, NC_>), f8q_grid(t), dim3(256), 0, s,                 \
                     static_cast<const T*>(x), static_cast<const T*>(r), w, w_f32,              \
                     static_cast<int>(t), static_cast<int>(h), upr, eps, static_cast<T*>(res_out), \
                     static_cast<T*>(norm_out), codes, scales)
  if (upr <= 4) MI_NORM_LAUNCH(1);
  else if (upr <= 8) MI_NORM_LAUNCH(2);
  else if (upr <= 16) MI_NORM_LAUNCH(4);
  else MI_NORM_LAUNCH(0);
#undef MI_NORM_LAUNCH
  return launch_status("add_rmsnorm_fp8");
}

}  // namespace
}  // namespace mi

extern "C" int64_t mi_fp8_scale_cols(int64_t k) { return k < 1 ? 0 : 4 * mi::f8_units(k); }

extern "C" mi_status mi_fp8_quantize(const void* x, int64_t batch, int64_t rows, int64_t k,
                                     mi_dtype dtype, int64_t block_rows, int swiglu,
                                     uint8_t* codes, float* scales, void* stream) {
  using namespace mi;
  clear_error();
  MI_REQUIRE(dtype == MI_BF16 || dtype == MI_F16 || dtype == MI_F32,
             "fp8_quantize: x must be bf16, fp16 or fp32");
  MI_REQUIRE(block_rows == 1 || block_rows == 128,
             "fp8_quantize: block_rows must be 1 or 128 (got %lld)", (long long)block_rows);
  MI_REQUIRE(!swiglu || block_rows == 1, "fp8_quantize: swiglu needs block_rows == 1");
  MI_REQUIRE(k >= 16 && k % 16 == 0 && k < (1LL << 30),
             "fp8_quantize: K %% 16 == 0 required (got K=%lld)", (long long)k);
  MI_REQUIRE(batch >= 0 && rows >= 0 && rows < (1LL << 31) - 128 && batch < (1LL << 31) &&
                 batch * rows <= (1LL << 62) / (4 * k),
             "fp8_quantize: batch or rows out of range");
  if (batch == 0 || rows == 0) return MI_OK;
  MI_REQUIRE(x != nullptr && codes != nullptr && scales != nullptr, "fp8_quantize: null pointer");
  MI_REQUIRE(aligned16(x) && aligned16(codes) && aligned16(scales),
             "fp8_quantize: x, codes and scales must be 16-byte aligned");
  MI_REQUIRE(block_rows == 1 || batch * ((rows + 127) / 128) * ((k + 127) / 128) < (1LL << 31),
             "fp8_quantize: too many blocks");
  const int64_t values = batch * rows * k;
  const int64_t xb = values * (dtype == MI_F32 ? 4 : 2) * (swiglu ? 2 : 1);
  const int64_t sb = batch * ((rows + block_rows - 1) / block_rows) * mi_fp8_scale_cols(k) * 4;
  MI_REQUIRE(!overlap(codes, values, x, xb) && !overlap(scales, sb, x, xb) &&
                 !overlap(codes, values, scales, sb),
             "fp8_quantize: codes and scales may not overlap x or each other");
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int br = static_cast<int>(block_rows);
  if (dtype == MI_BF16)
    return launch_quantize<__bf16>(x, batch, rows, k, br, swiglu != 0, codes, scales, s);
  if (dtype == MI_F16)
    return launch_quantize<_Float16>(x, batch, rows, k, br, swiglu != 0, codes, scales, s);
  return launch_quantize<float>(x, batch, rows, k, br, swiglu != 0, codes, scales, s);
}

extern "C" mi_status mi_add_rmsnorm_fp8(const void* x, const void* residual, const void* weight,
                                        mi_dtype dtype, mi_dtype weight_dtype,
                                        int64_t num_tokens, int64_t hidden_size, float eps,
                                        void* residual_out, void* norm_out, uint8_t* codes,
                                        float* scales, void* stream) {
  using namespace mi;
  clear_error();
  MI_REQUIRE(dtype == MI_BF16 || dtype == MI_F16 || dtype == MI_F32,
             "add_rmsnorm_fp8: x must be bf16, fp16 or fp32");
  MI_REQUIRE(weight_dtype == dtype || weight_dtype == MI_F32,
             "add_rmsnorm_fp8: weight must be of x's type or fp32");
  MI_REQUIRE(hidden_size >= 16 && hidden_size % 16 == 0 && hidden_size < (1LL << 30),
             "add_rmsnorm_fp8: hidden_size %% 16 == 0 required (got %lld)",
             (long long)hidden_size);
  MI_REQUIRE(num_tokens >= 0 && num_tokens < (1LL << 31),
             "add_rmsnorm_fp8: num_tokens out of range (%lld)", (long long)num_tokens);
  MI_REQUIRE(eps >= 0.f, "add_rmsnorm_fp8: eps must be >= 0");
  MI_REQUIRE((residual == nullptr) == (residual_out == nullptr) || num_tokens == 0,
             "add_rmsnorm_fp8: residual and residual_out go together");
  if (num_tokens == 0) return MI_OK;
  MI_REQUIRE(x != nullptr && weight != nullptr && codes != nullptr && scales != nullptr,
             "add_rmsnorm_fp8: null pointer");
  MI_REQUIRE(aligned16(x) && aligned16(residual) && aligned16(weight) && aligned16(residual_out) &&
                 aligned16(norm_out) && aligned16(codes) && aligned16(scales),
             "add_rmsnorm_fp8: every tensor must be 16-byte aligned");
  // a stream written where another row is still to be read would race
  const int64_t n = num_tokens * hidden_size, bytes = n * (dtype == MI_F32 ? 4 : 2);
  MI_REQUIRE(residual_out == residual || !overlap(residual_out, bytes, residual, bytes),
             "add_rmsnorm_fp8: residual_out may be residual itself, not overlap it otherwise");
  MI_REQUIRE(residual_out == x || !overlap(residual_out, bytes, x, bytes),
             "add_rmsnorm_fp8: residual_out may be x itself, not overlap it otherwise");
  MI_REQUIRE(!overlap(norm_out, bytes, x, bytes) && !overlap(norm_out, bytes, residual, bytes) &&
                 !overlap(norm_out, bytes, residual_out, bytes),
             "add_rmsnorm_fp8: norm_out may not overlap x, residual or residual_out");
  const int64_t sb = num_tokens * mi_fp8_scale_cols(hidden_size) * 4;
  const int64_t wb = hidden_size * (weight_dtype == MI_F32 ? 4 : 2);
  MI_REQUIRE(!overlap(residual_out, bytes, weight, wb) && !overlap(norm_out, bytes, weight, wb) &&
                 !overlap(codes, n, weight, wb) && !overlap(scales, sb, weight, wb),
             "add_rmsnorm_fp8: no output may overlap weight");
  for (const void* const other : {x, residual, static_cast<const void*>(residual_out),
                                  static_cast<const void*>(norm_out)})
    MI_REQUIRE(!overlap(codes, n, other, bytes) && !overlap(scales, sb, other, bytes),
               "add_rmsnorm_fp8: codes and scales may not overlap another tensor");
  MI_REQUIRE(!overlap(codes, n, scales, sb),
             "add_rmsnorm_fp8: codes and scales may not overlap another tensor");
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool wf = weight_dtype == MI_F32;
  if (dtype == MI_BF16)
    return launch_norm<__bf16>(x, residual, weight, wf, num_tokens, hidden_size, eps, residual_out,
                               norm_out, codes, scales, s);
  if (dtype == MI_F16)
    return launch_norm<_Float16>(x, residual, weight, wf, num_tokens, hidden_size, eps,
                                 residual_out, norm_out, codes, scales, s);
  return launch_norm<float>(x, residual, weight, wf, num_tokens, hidden_size, eps, residual_out,
                            norm_out, codes, scales, s);
}
