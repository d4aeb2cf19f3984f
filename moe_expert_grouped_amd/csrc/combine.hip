// The way back from expert order to token order, and its gradients, on gfx950.
//
//   out[t]        = sum_j w[t, j] rows[perm[t, j]]              (moe_combine_rows)
//   grad_rows[p]  = w[t, j] go[t],   p = perm[t, j]             (its gradient)
//   grad_w[t, j]  = sum_h rows[p, h] go[t, h]
//
// Without weights the first line is the gradient of the copy to expert order.
// A slot whose row is outside [0, num_rows) contributes nothing and gets a
// zero weight gradient.  Sums are fp32, over the slots in their order, so the
// result does not depend on the schedule; one rounding.
//
// All three are bound by memory: top_k rows read (and written) per token, 2
// operations a value.  A large copy reaches 5.1 TB/s on the same card.
#include "common.hpp"

namespace mi {
namespace {

// the 16-byte piece of a row: 8 values of a 16-bit type, 4 of fp32
template <typename T>
struct Piece {
  static constexpr int N = 16 / sizeof(T);
  u32x4 v;
  __device__ float get(int i) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(v[i]);
    } else {
      const uint32_t w = v[i >> 1];
      if constexpr (std::is_same<T, __bf16>::value)
        return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
      else
        return static_cast<float>(__builtin_bit_cast(
            _Float16, static_cast<uint16_t>((i & 1) ? (w >> 16) : (w & 0xffff))));
    }
  }
};

// N floats (4 or 8) loaded from, or rounded once to, T at p
template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float* y) {
  constexpr int B = N * sizeof(T);
  if constexpr (B == 8) {
    typedef T t4 __attribute__((ext_vector_type(4)));
    const t4 v = gld<t4>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = static_cast<float>(v[i]);
  } else {
#pragma unroll
    for (int c = 0; c < B / 16; ++c) {
      Piece<T> q{gld<u32x4>(p + c * Piece<T>::N)};
#pragma unroll
      for (int i = 0; i < Piece<T>::N; ++i) y[c * Piece<T>::N + i] = q.get(i);
    }
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float* y) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int c = 0; c < N / 4; ++c)
      gst<f32x4>(p + 4 * c, f32x4{y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]});
  } else {
    typedef T tn __attribute__((ext_vector_type(N)));
    typedef float fn __attribute__((ext_vector_type(N)));
    fn v;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = y[i];
    gst<tn>(p, __builtin_convertvector(v, tn));
  }
}

// A unit is 64 pieces of one token's output row, one wavefront each, so that few
// tokens still spread over the chip (16 tokens, top 8, H 7168: 224 units, 3.7 us):
// the unit's pieces of the token's rows are loaded CU_SLOTS at a time, all in
// flight together, before the first is used.  8192 tokens, top 8, H 4096 bf16,
// 5% of the slots without a row: 578 MB in 113 us, 5.1 TB/s.
constexpr int CU_SLOTS = 8;

template <typename T, typename OutT>
__global__ __launch_bounds__(256) void combine_kernel(const T* __restrict__ rows, int64_t num_rows,
                                                      int h, const int32_t* __restrict__ perm,
                                                      const float* __restrict__ weights,
                                                      int64_t units, int upr, int top_k,
                                                      OutT* __restrict__ out) {
  constexpr int N = Piece<T>::N;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t nw = static_cast<int64_t>(gridDim.x) * 4;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + wave; u < units; u += nw) {
    const int64_t t = u / upr;
    const int col = (static_cast<int>(u - t * upr) * 64 + lane) * N;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < top_k; j0 += CU_SLOTS) {
      Piece<T> d[CU_SLOTS];
      float w[CU_SLOTS];
      bool on[CU_SLOTS];
#pragma unroll
      for (int j = 0; j < CU_SLOTS; ++j) {
        const int64_t x = t * top_k + min(j0 + j, top_k - 1);
        const int p = perm[x];
        on[j] = j0 + j < top_k && p >= 0 && p < num_rows;
        w[j] = weights != nullptr ? weights[x] : 1.f;
        if (on[j] && col < h) d[j].v = gld<u32x4>(rows + static_cast<int64_t>(p) * h + col);
        else d[j].v = u32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int j = 0; j < CU_SLOTS; ++j) {
        // an absent slot's weight is not looked at, it may be anything
        if (on[j]) {
#pragma unroll
          for (int i = 0; i < N; ++i) acc[i] = __builtin_fmaf(w[j], d[j].get(i), acc[i]);
        }
      }
    }
    if (col < h) store_n<OutT, N>(out + t * h + col, acc);
  }
}

// One wavefront per slot: w * go[t] to the slot's row, and the dot product of
// the row with go[t].  With the inverse permutation a row's one writer is the slot
// that the inverse names, if that slot points at the row; else wavefront p writes
// zeros to row p.  So every row is written once, whatever the two arrays hold
// (slots taken out of one of them, two slots with one row): the order of the
// wavefronts does not matter and no row is left as it was.  The inverse costs a
// second, dependent 4-byte read a slot, which the rows' loads do not wait for.
template <typename T, typename GoT>
__global__ __launch_bounds__(256) void combine_backward_kernel(
    const GoT* __restrict__ go, const T* __restrict__ rows, int64_t num_rows, int h,
    const int32_t* __restrict__ perm, const int32_t* __restrict__ inverse,
    const float* __restrict__ weights, int64_t slots, int top_k, T* __restrict__ grad_rows,
    float* __restrict__ grad_w) {
  constexpr int N = Piece<T>::N;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t nw = static_cast<int64_t>(gridDim.x) * 4;
  const int64_t units = inverse != nullptr && num_rows > slots ? num_rows : slots;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + wave; u < units; u += nw) {
    if (u < slots) {
      const int p = perm[u];
      float dot = 0.f;
      if (p >= 0 && p < num_rows) {
        const float w = weights[u];
        const GoT* g = go + u / top_k * h;
        const T* src = rows + static_cast<int64_t>(p) * h;
        T* dst = grad_rows + static_cast<int64_t>(p) * h;
        const bool writer = inverse == nullptr || inverse[p] == u;
        for (int col = lane * N; col < h; col += 64 * N) {
          float y[N];
          load_n<GoT, N>(g + col, y);
          if (grad_w != nullptr) {
            float d[N];
            load_n<T, N>(src + col, d);
#pragma unroll
            for (int i = 0; i < N; ++i) dot = __builtin_fmaf(d[i], y[i], dot);
          }
#pragma unroll
          for (int i = 0; i < N; ++i) y[i] *= w;
          if (writer) store_n<T, N>(dst + col, y);
        }
      }
      if (grad_w != nullptr) {
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) dot += __shfl_xor(dot, o, 64);
        if (lane == 0) gst<float>(grad_w + u, dot);
      }
    }
    bool empty = false;
    if (inverse != nullptr && u < num_rows) {
      const int s = inverse[u];
      empty = s < 0 || s >= slots || perm[s] != u;
    }
    if (empty) {
      const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int col = lane * N; col < h; col += 64 * N)
        store_n<T, N>(grad_rows + u * h + col, z);
    }
  }
}

int64_t size_of(mi_dtype d) { return d == MI_F32 ? 4 : 2; }
bool known(mi_dtype d) { return d == MI_BF16 || d == MI_F16 || d == MI_F32; }
// grid of 4-wavefront workgroups over `units`; the wavefronts stride over the rest
dim3 grid_of(int64_t units) {
  const int64_t b = (units + 3) / 4;
  return dim3(static_cast<unsigned>(b > 16384 ? 16384 : b));
}

}  // namespace
}  // namespace mi

// calls F<T, U>(...) for the two element types
#define MI_BY_TYPE(D, T, ...)                                     \
  if (D == MI_BF16) { using T = __bf16; __VA_ARGS__ }             \
  else if (D == MI_F16) { using T = _Float16; __VA_ARGS__ }       \
  else { using T = float; __VA_ARGS__ }

extern "C" mi_status mi_moe_combine_rows(const void* rows, mi_dtype rows_dtype, int64_t num_rows,
                                         int64_t hidden_size, const int32_t* perm,
                                         const float* weights, int64_t num_tokens, int64_t top_k,
                                         void* out, mi_dtype out_dtype, void* stream) {
  using namespace mi;
  clear_error();
  MI_REQUIRE(known(rows_dtype) && known(out_dtype),
             "moe_combine_rows: rows and out must be bf16, fp16 or fp32");
  MI_REQUIRE(hidden_size > 0 && hidden_size % 8 == 0 && hidden_size < (1LL << 30),
             "moe_combine_rows: hidden_size %% 8 == 0 required (got %lld)",
             (long long)hidden_size);
  MI_REQUIRE(num_tokens >= 0 && top_k >= 1 && num_tokens <= ((1LL << 31) - 1) / top_k,
             "moe_combine_rows: num_tokens * top_k must be in [0, 2^31)");
  MI_REQUIRE(num_rows >= 0, "moe_combine_rows: num_rows must be >= 0");
  if (num_tokens == 0) return MI_OK;
  MI_REQUIRE(perm != nullptr && out != nullptr && (rows != nullptr || num_rows == 0),
             "moe_combine_rows: null pointer");
  MI_REQUIRE(aligned16(rows) && aligned16(out), "moe_combine_rows: rows and out must be 16-byte aligned");
  MI_REQUIRE(num_rows < (1LL << 31), "moe_combine_rows: num_rows out of range");
  const int64_t slots = num_tokens * top_k, ob = num_tokens * hidden_size * size_of(out_dtype);
  MI_REQUIRE(!overlap(out, ob, rows, num_rows * hidden_size * size_of(rows_dtype)) &&
                 !overlap(out, ob, perm, slots * 4) && !overlap(out, ob, weights, slots * 4),
             "moe_combine_rows: out may not overlap an input");
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int h = static_cast<int>(hidden_size);
  const int upr = (h + (rows_dtype == MI_F32 ? 255 : 511)) / (rows_dtype == MI_F32 ? 256 : 512);
  const int64_t units = num_tokens * upr;
  MI_BY_TYPE(rows_dtype, T, MI_BY_TYPE(out_dtype, O, {
    hipLaunchKernelGGL((combine_kernel<T, O>), grid_of(units), dim3(256), 0, s,
                       static_cast<const T*>(rows), num_rows, h, perm, weights, units, upr,
                       static_cast<int>(top_k), static_cast<O*>(out));
  }))
  return launch_status("moe_combine_rows");
}

extern "C" mi_status mi_moe_combine_rows_backward(
    const void* grad_out, mi_dtype grad_dtype, const void* rows, mi_dtype rows_dtype,
    int64_t num_rows, int64_t hidden_size, const int32_t* perm, const int32_t* inverse,
    const float* weights, int64_t num_tokens, int64_t top_k, void* grad_rows, float* grad_weights,
    void* stream) {
  using namespace mi;
  clear_error();
  MI_REQUIRE(known(rows_dtype) && known(grad_dtype),
             "moe_combine_rows_backward: grad_out and rows must be bf16, fp16 or fp32");
  MI_REQUIRE(hidden_size > 0 && hidden_size % 8 == 0 && hidden_size < (1LL << 30),
             "moe_combine_rows_backward: hidden_size %% 8 == 0 required (got %lld)",
             (long long)hidden_size);
  MI_REQUIRE(num_tokens >= 0 && top_k >= 1 && num_tokens <= ((1LL << 31) - 1) / top_k,
             "moe_combine_rows_backward: num_tokens * top_k must be in [0, 2^31)");
  MI_REQUIRE(num_rows >= 0 && num_rows < (1LL << 31),
             "moe_combine_rows_backward: num_rows out of range");
  if (num_tokens == 0 && (inverse == nullptr || num_rows == 0)) return MI_OK;
  MI_REQUIRE(num_tokens == 0 || (perm != nullptr && weights != nullptr && grad_out != nullptr),
             "moe_combine_rows_backward: grad_out, weights or the permutation is null");
  MI_REQUIRE(num_rows == 0 || grad_rows != nullptr, "moe_combine_rows_backward: grad_rows is null");
  MI_REQUIRE(grad_weights == nullptr || rows != nullptr || num_rows == 0 || num_tokens == 0,
             "moe_combine_rows_backward: grad_weights needs rows");
  MI_REQUIRE(aligned16(grad_out) && aligned16(rows) && aligned16(grad_rows),
             "moe_combine_rows_backward: grad_out, rows and grad_rows must be 16-byte aligned");
  const int64_t slots = num_tokens * top_k;
  const int64_t rb = num_rows * hidden_size * size_of(rows_dtype);
  const int64_t gb = num_tokens * hidden_size * size_of(grad_dtype);
  auto apart = [&](const void* o, int64_t n) {  // from every input
    return !overlap(o, n, grad_out, gb) && !overlap(o, n, rows, rb) &&
           !overlap(o, n, perm, slots * 4) && !overlap(o, n, inverse, num_rows * 4) &&
           !overlap(o, n, weights, slots * 4);
  };
  MI_REQUIRE(apart(grad_rows, rb) && apart(grad_weights, slots * 4) &&
                 !overlap(grad_rows, rb, grad_weights, slots * 4),
             "moe_combine_rows_backward: grad_rows and grad_weights may not overlap an input or "
             "each other");
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t units = inverse != nullptr && num_rows > slots ? num_rows : slots;
  MI_BY_TYPE(rows_dtype, T, MI_BY_TYPE(grad_dtype, G, {
    hipLaunchKernelGGL((combine_backward_kernel<T, G>), grid_of(units), dim3(256), 0, s,
                       static_cast<const G*>(grad_out), static_cast<const T*>(rows), num_rows,
                       static_cast<int>(hidden_size), perm, inverse, weights, slots,
                       static_cast<int>(top_k), static_cast<T*>(grad_rows), grad_weights);
  }))
  return launch_status("moe_combine_rows_backward");
}
