// The router of a MoE layer on gfx950: the top_k experts of a token, the balance
// loss of a batch and the gradient of the logits through both.
//
//   p[t]     = softmax(logits[t])                                    fp32
//   route:     ids[t] = the top_k largest logits, ties to the lowest index,
//              w[t, j] = p[t, ids[t, j]]  (/ their sum over j, if renormalised)
//   balance:   counts[e] = choices of e,  f = counts / sum counts,
//              P[e] = mean of p[:, e],    loss = coef * E * sum_e f[e] P[e],
//              slopes[e] = d loss / d p[t, e] = coef * E * f[e] / tokens
//   backward:  grad = p * (q - sum_e p q),  q = grad_loss * slopes
//                                             + grad_w scattered to the ids;
//              renormalised weights add w[j] (grad_w[j] - sum_i grad_w[i] w[i]) at
//              ids[j] instead.
//
// A token's row lies in a group of G lanes, VPL values a lane, in pieces of 16
// bytes (piece i * G + g is lane g's): a row is read once and every sum, maximum
// and choice is a butterfly over G lanes that serves 64 / G tokens at once.
//
// A logit of -inf is an expert that cannot be chosen: its p is 0; where a row has
// fewer than top_k others, the rest of its ids is -1 with weight 0, and a row of
// -inf only has p = 0.  NaN is above every number, as in a sort.  Tokens that
// token_mask takes out (padding) have ids -1, weights 0, gradients 0, and count
// nowhere; their logits are not looked at.
#include "common.hpp"

namespace mi {
namespace {

constexpr int RT_MAX_EXPERTS = 1024;
constexpr int RT_MAX_TOPK = 64;

// ---------------------------------------------------------------------------
// over the G lanes of a row
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ uint32_t rt_dpp(uint32_t v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, true);
}

// op over the lanes of every aligned group of G, the result in all of them
template <int G, typename F>
__device__ __forceinline__ uint32_t rt_all(uint32_t v, F op) {
  v = op(v, rt_dpp<0xb1>(v));                         // quad_perm 1, 0, 3, 2
  v = op(v, rt_dpp<0x4e>(v));                         // quad_perm 2, 3, 0, 1
  v = op(v, rt_dpp<0x141>(v));                        // row_half_mirror: the other quad
  if constexpr (G >= 16) v = op(v, rt_dpp<0x140>(v)); // row_mirror: the other eight
  if constexpr (G >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op(r[0], r[1]);
  }
  if constexpr (G >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = op(r[0], r[1]);
  }
  return v;
}
template <int G>
__device__ __forceinline__ float rt_sum(float v) {
  return __uint_as_float(rt_all<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int G>
__device__ __forceinline__ float rt_max(float v) {  // NaN is passed over
  return __uint_as_float(rt_all<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int G>
__device__ __forceinline__ uint32_t rt_umax(uint32_t v) {
  return rt_all<G>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// exp(d) for d <= 0 with the argument's rest carried: d * log2(e) rounded is off by
// half a step of the product, which at d = -60 would be 45 steps of the result
__device__ __forceinline__ float rt_exp(float d) {
  constexpr float L = 1.44269504088896340736f, L_LO = 1.9259629911266175e-8f;
  const float t = d * L;
  const float rest = __builtin_fmaf(d, L_LO, __builtin_fmaf(d, L, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  // rest is inf - inf where t is -inf: e is 0 there
  return t < -150.f ? 0.f : __builtin_fmaf(e, rest * 0.69314718055994530942f, e);
}

// ---------------------------------------------------------------------------
// a row
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ float rt_f32(T v) {
  return static_cast<float>(v);
}

// Columns of lane g: piece i covers (i * G + g) * VEC ..
template <typename T, int G, int VPL>
struct RtRow {
  static constexpr int VEC = 16 / sizeof(T), NV = VPL / VEC;
  static_assert(NV * VEC == VPL, "row");
  float z[VPL];
  T raw[VPL];  // as they are stored
  __device__ __forceinline__ static int col(int g, int v) {
    return ((v / VEC) * G + g) * VEC + v % VEC;
  }
  // columns past E are -inf
  __device__ __forceinline__ void load(const T* row, int g, int E, bool vec) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col(g, i * VEC);
      T part[VEC] = {};
      if (vec) {
        if (c < E) {
          const u32x4 q = gld<u32x4>(row + c);
          __builtin_memcpy(part, &q, 16);
        }
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (c + j < E) part[j] = gld<T>(row + c + j);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        raw[i * VEC + j] = part[j];
        z[i * VEC + j] = c + j < E ? rt_f32(part[j]) : -__builtin_inff();
      }
    }
  }
  // exp(z - max) into p; returns their sum and the maximum (all columns -inf: zeros).
  // A NaN makes the sum NaN, and with it every weight of the row.
  __device__ __forceinline__ float exps(float (&p)[VPL], float& top) const {
    float m = z[0];
#pragma unroll
    for (int v = 1; v < VPL; ++v) m = fmaxf(m, z[v]);
    m = rt_max<G>(m);
    top = m;
    const bool none = m == -__builtin_inff();
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      p[v] = none && z[v] == z[v] ? 0.f : z[v] == -__builtin_inff() ? 0.f : rt_exp(z[v] - m);
      s += p[v];
    }
    return rt_sum<G>(s);
  }
};

// p / sum, rounded once as a division is, from the sum's reciprocal (0 for a sum of 0): the
// product's error is exact and corrects it (32768 tokens of 256 experts in bf16, balance and
// gradient: 38.7 us, the product alone 38.2)
__device__ __forceinline__ float rt_over(float p, float sum, float inv) {
  const float q = p * inv;
  return __builtin_fmaf(__builtin_fmaf(-sum, q, p), inv, q);
}

// order of a logit: larger is larger, -0 is 0, -inf is 0 (never chosen), NaN the largest
__device__ __forceinline__ uint32_t rt_order(float z) {
  if (z != z) return 0xffffffffu;
  if (z == -__builtin_inff()) return 0u;
  const uint32_t b = __float_as_uint(z + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float rt_logit(uint32_t order) {
  return __uint_as_float(order & 0x80000000u ? order & 0x7fffffffu : ~order);
}

// A candidate: its order and its column, such that the largest key is the largest logit of
// the lowest column.  bf16 and fp16 have both in 32 bits (their order is 16 bits, once the
// fp16 is taken as it is stored); fp32 takes two words.
template <typename T>
struct RtKey {
  uint32_t k;
  __device__ __forceinline__ static RtKey make(T raw, float z, int col) {
    const uint32_t b = __builtin_bit_cast(uint16_t, raw);
    uint32_t o = b & 0x8000u ? ~b & 0xffffu : b | 0x8000u;
    if (z == 0.f) o = 0x8000u;
    if (z != z) o = 0xffffu;
    return {z == -__builtin_inff() ? 0u : o << 16 | (0xffffu - col)};
  }
  __device__ __forceinline__ bool any() const { return k != 0u; }
  __device__ __forceinline__ int col() const { return 0xffff - (k & 0xffffu); }
  __device__ __forceinline__ float logit() const {
    const uint32_t o = k >> 16;
    if (o == 0xffffu) return __builtin_nanf("");
    return static_cast<float>(__builtin_bit_cast(T, static_cast<uint16_t>(o & 0x8000u ? o & 0x7fffu : ~o)));
  }
  // a and b in falling order
  __device__ __forceinline__ static void sort(RtKey& a, RtKey& b) {
    const uint32_t hi = max(a.k, b.k), lo = min(a.k, b.k);
    a.k = hi;
    b.k = lo;
  }
  template <int G>
  __device__ __forceinline__ static RtKey best(RtKey head) { return {rt_umax<G>(head.k)}; }
  __device__ __forceinline__ bool is(const RtKey& o) const { return k == o.k; }
  __device__ __forceinline__ static RtKey none() { return {0u}; }
};
template <>
struct RtKey<float> {
  uint32_t o, c;  // order, ~column
  __device__ __forceinline__ static RtKey make(float, float z, int col) {
    return {rt_order(z), ~static_cast<uint32_t>(col)};
  }
  __device__ __forceinline__ bool any() const { return o != 0u; }
  __device__ __forceinline__ int col() const { return static_cast<int>(~c); }
  __device__ __forceinline__ float logit() const { return o == 0xffffffffu ? __builtin_nanf("") : rt_logit(o); }
  __device__ __forceinline__ static void sort(RtKey& a, RtKey& b) {
    const bool swap = (static_cast<uint64_t>(b.o) << 32 | b.c) > (static_cast<uint64_t>(a.o) << 32 | a.c);
    const RtKey x = a;
    a.o = swap ? b.o : a.o;
    a.c = swap ? b.c : a.c;
    b.o = swap ? x.o : b.o;
    b.c = swap ? x.c : b.c;
  }
  template <int G>
  __device__ __forceinline__ static RtKey best(RtKey head) {
    const uint32_t o = rt_umax<G>(head.o);
    return {o, rt_umax<G>(head.o == o ? head.c : 0u)};
  }
  __device__ __forceinline__ bool is(const RtKey& x) const { return o == x.o && c == x.c; }
  __device__ __forceinline__ static RtKey none() { return {0u, 0u}; }
};

// falling order by an odd-even merge network
template <int N, typename K>
__device__ __forceinline__ void rt_sort(K (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) K::sort(k[i + j], k[i + j + q]);
}

struct RtRoute {
  const void* logits;
  const uint8_t* mask;
  float* weights;
  int32_t* ids;
  int T, E, k;
  bool renorm, vec;
};

// ---------------------------------------------------------------------------
// top_k.  A lane sorts its own values; then k times the largest of the lanes' heads is
// taken and its lane moves on.  Keys are unique, so no choice depends on the layout.
// Lane j keeps choice j and computes its weight from the logit that the key holds.
// Bound by the VALU (the row's exponentials among it, which renormalised weights do not need):
// 32768 tokens, 128 experts, top 8, bf16: 8.3 us (10.5 MB), 13.3 with the
// values left unsorted and three butterflies a choice.
// ---------------------------------------------------------------------------
template <typename T, int G, int VPL>
__global__ __launch_bounds__(256) void rt_route_kernel(RtRoute a) {
  using Row = RtRow<T, G, VPL>;
  using Key = RtKey<T>;
  const int g = threadIdx.x & (G - 1);
  const int64_t per = static_cast<int64_t>(gridDim.x) * (256 / G);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (256 / G) + threadIdx.x / G; t < a.T; t += per) {
    const uint8_t real = a.mask == nullptr ? 1 : gld<uint8_t>(a.mask + t);
    Row row;
    row.load(static_cast<const T*>(a.logits) + t * a.E, g, a.E, a.vec);
    if (real == 0) {
      if (g < a.k) {
        gst<float>(a.weights + t * a.k + g, 0.f);
        gst<int32_t>(a.ids + t * a.k + g, -1);
      }
      continue;
    }
    float p[VPL], top;
    const float sum = row.exps(p, top);
    Key key[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c = Row::col(g, v);
      key[v] = c < a.E ? Key::make(row.raw[v], row.z[v], c) : Key::none();
    }
    rt_sort(key);
    Key mine = Key::none();
    for (int j = 0; j < a.k; ++j) {
      const Key best = Key::template best<G>(key[0]);
      if (j == g) mine = best;
      const bool gone = key[0].is(best);
#pragma unroll
      for (int v = 0; v + 1 < VPL; ++v)
        if (gone) key[v] = key[v + 1];
      if (gone) key[VPL - 1] = Key::none();
    }
    const bool has = g < a.k && mine.any();
    const float w = has ? rt_exp(mine.logit() - top) : 0.f;
    const float by = a.renorm ? rt_sum<G>(w) : sum;
    if (g < a.k) {
      gst<float>(a.weights + t * a.k + g, has ? w / by : 0.f);
      gst<int32_t>(a.ids + t * a.k + g, has ? mine.col() : -1);
    }
  }
}

// ---------------------------------------------------------------------------
// balance.  A lane's columns are the same for every row it takes, so the sums of p
// stay in its registers over all of a workgroup's rows; then they are added in a
// fixed order, over the workgroup in LDS and over the workgroups by a second
// launch, whose workgroups have 64 experts each and leave the loss's terms to the last
// of them to end.  One workgroup does it all for a small batch.  No atomic adds floats.  Bound by
// latency, of a few rows' loads for every wavefront, then of the second launch's: 16411 tokens
// of 256 experts in fp32: 9.7 and 7.9 us (17 MB); 512 tokens of 64 in one launch 10.4.
// ---------------------------------------------------------------------------
struct RtBalance {
  const void* logits;
  const int32_t* ids;
  const uint8_t* mask;
  const int32_t* given;  // counts of more than these tokens, or null
  float* part_p;         // [blocks, E]
  int32_t* part_c;       // [blocks, E + 2]: choices, tokens, sum of the choices
  float* terms;          // [ceil(E / 64)] of the loss
  int32_t* ended;        // workgroups of the second launch that have ended
  float* loss;
  int32_t* counts;
  float* slopes;
  int T, E, k, blocks;
  float coef;
  bool vec;
};

constexpr int RT_BT = 1024;  // threads of a balance workgroup

__device__ __forceinline__ double rt_block_sum(double v, double* s) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((tid & 63) == 0) s[tid >> 6] = v;
  __syncthreads();
  double all = 0.;
  for (int w = 0; w < RT_BT / 64; ++w) all += s[w];
  return all;
}

// sums of p and counts of all tokens, thread e's of expert e, and the number of tokens
__device__ __forceinline__ void rt_finish(const RtBalance& a, float p, int c, int tokens,
                                          double* s) {
  const int e = threadIdx.x;
  const bool in = e < a.E;
  const int by = in ? (a.given != nullptr ? gld<int32_t>(a.given + e) : c) : 0;
  const double choices = rt_block_sum(static_cast<double>(by), s);
  const double unit = tokens > 0 && choices > 0.
                          ? static_cast<double>(a.coef) * a.E / choices / tokens : 0.;
  const double slope = unit * by;
  const double loss = rt_block_sum(in ? slope * p : 0., s);
  if (in) {
    gst<int32_t>(a.counts + e, c);
    gst<float>(a.slopes + e, static_cast<float>(slope));
  }
  if (e == 0) gst<float>(a.loss, static_cast<float>(loss));
}

template <typename T, int G, int VPL>
__global__ __launch_bounds__(RT_BT) void rt_balance_kernel(RtBalance a) {
  using Row = RtRow<T, G, VPL>;
  constexpr int ROWS = RT_BT / G;
  __shared__ float s_p[16][RT_MAX_EXPERTS];  // a wavefront's sums
  __shared__ int s_c[RT_MAX_EXPERTS + 1];
  __shared__ double s_d[RT_BT / 64];
  const int tid = threadIdx.x, g = tid & (G - 1), lane = tid & 63, wave = tid >> 6;
  if (tid < a.E) s_c[tid] = 0;
  if (tid == 0) s_c[RT_MAX_EXPERTS] = 0;
  __syncthreads();
  float acc[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) acc[v] = 0.f;
  int tokens = 0;
  const int64_t per = static_cast<int64_t>(a.blocks) * ROWS;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * ROWS + tid / G; t < a.T; t += per) {
    const uint8_t real = a.mask == nullptr ? 1 : gld<uint8_t>(a.mask + t);
    Row row;
    row.load(static_cast<const T*>(a.logits) + t * a.E, g, a.E, a.vec);
    const int first = g < a.k ? gld<int32_t>(a.ids + t * a.k + g) : -1;
    if (real == 0) continue;
    ++tokens;
    float p[VPL], top;
    const float sum = row.exps(p, top);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int v = 0; v < VPL; ++v) acc[v] += rt_over(p[v], sum, inv);
    for (int j = g; j < a.k; j += G) {
      const int id = j == g ? first : gld<int32_t>(a.ids + t * a.k + j);
      if (id >= 0 && id < a.E) atomicAdd(&s_c[id], 1);
    }
  }
  if (g == 0 && tokens) atomicAdd(&s_c[RT_MAX_EXPERTS], tokens);
  // the 64 / G rows of a wavefront, then the wavefronts
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    float x = acc[v];
#pragma unroll
    for (int o = 32; o >= G; o >>= 1) x += __shfl_xor(x, o, 64);
    const int c = Row::col(g, v);
    if (lane < G && c < a.E) s_p[wave][c] = x;
  }
  __syncthreads();
  float p = 0.f;
  int c = 0;
  if (tid < a.E) {
    for (int w = 0; w < RT_BT / 64; ++w) p += s_p[w][tid];
    c = s_c[tid];
  }
  const int all = s_c[RT_MAX_EXPERTS];
  if (a.blocks == 1) {
    rt_finish(a, p, c, all, s_d);
    return;
  }
  int32_t* const part = a.part_c + static_cast<int64_t>(blockIdx.x) * (a.E + 2);
  if (tid < a.E) {
    gst<float>(a.part_p + static_cast<int64_t>(blockIdx.x) * a.E + tid, p);
    gst<int32_t>(part + tid, c);
  }
  const double choices = rt_block_sum(static_cast<double>(c), s_d);
  if (tid == 0) {
    gst<int32_t>(part + a.E, all);
    gst<int32_t>(part + a.E + 1, static_cast<int32_t>(choices));
    if (blockIdx.x == 0) gst<int32_t>(a.ended, 0);
  }
}

// 64 experts a workgroup, a wavefront every sixteenth of the first launch's workgroups.
// The totals are whole numbers: the first wavefront adds them itself.
constexpr int RT_BLOCKS = 256;  // of the first launch, at most
__global__ __launch_bounds__(RT_BT) void rt_balance_finish_kernel(RtBalance a) {
  __shared__ float s_p[RT_BT];
  __shared__ int s_c[RT_BT];
  constexpr int W = RT_BT / 64, PER = RT_BLOCKS / W;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = blockIdx.x * 64 + lane;
  const bool in = e < a.E;
  int64_t tokens = 0, choices = 0;
  if (wave == 0) {
#pragma unroll
    for (int i = 0; i < RT_BLOCKS / 64; ++i) {
      const int b = i * 64 + lane;
      if (b < a.blocks) {
        const int32_t* const part = a.part_c + static_cast<int64_t>(b) * (a.E + 2) + a.E;
        tokens += gld<int32_t>(part);
        choices += gld<int32_t>(part + 1);
      }
    }
    if (a.given != nullptr) {
      choices = 0;
      for (int i = lane; i < a.E; i += 64) choices += gld<int32_t>(a.given + i);
    }
  }
  float p = 0.f, ps[PER];
  int c = 0, cs[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = wave + W * i;
    const bool here = in && b < a.blocks;
    ps[i] = here ? gld<float>(a.part_p + static_cast<int64_t>(b) * a.E + e) : 0.f;
    cs[i] = here ? gld<int32_t>(a.part_c + static_cast<int64_t>(b) * (a.E + 2) + e) : 0;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    p += ps[i];
    c += cs[i];
  }
  s_p[tid] = p;
  s_c[tid] = c;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    tokens += __shfl_xor(tokens, o, 64);
    choices += __shfl_xor(choices, o, 64);
  }
#pragma unroll
  for (int w = 1; w < W; ++w) {
    p += s_p[w * 64 + lane];
    c += s_c[w * 64 + lane];
  }
  double term = 0.;
  if (in) {
    const int by = a.given != nullptr ? gld<int32_t>(a.given + e) : c;
    const double slope = tokens > 0 && choices > 0
                             ? static_cast<double>(a.coef) * a.E / static_cast<double>(choices) /
                                   static_cast<double>(tokens) * by : 0.;
    gst<int32_t>(a.counts + e, c);
    gst<float>(a.slopes + e, static_cast<float>(slope));
    term = slope * p;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) term += __shfl_xor(term, o, 64);
  if (lane != 0) return;
  if (gridDim.x == 1) {
    gst<float>(a.loss, static_cast<float>(term));
    return;
  }
  __hip_atomic_store(a.terms + blockIdx.x, static_cast<float>(term), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __threadfence();
  if (atomicAdd(a.ended, 1) == static_cast<int>(gridDim.x) - 1) {
    __threadfence();
    double loss = 0.;
    for (int b = 0; b < static_cast<int>(gridDim.x); ++b)
      loss += __hip_atomic_load(a.terms + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    gst<float>(a.loss, static_cast<float>(loss));
  }
}

// ---------------------------------------------------------------------------
// backward.  A row is read and written once: 16411 tokens of 256 experts in fp32, of the
// loss: 12.7 us (34 MB: 2.6 TB/s, the grid's start and end among it); through the weights of
// 6 choices as well, 16384 tokens of 64: 6.3 us.
// ---------------------------------------------------------------------------
struct RtBackward {
  const void* logits;
  const int32_t* ids;
  const float* weights;
  const float* grad_w;     // null: nothing through the weights
  const float* slopes;     // null: nothing through the loss
  const float* grad_loss;
  const uint8_t* mask;
  void* out;
  int T, E, k;
  bool renorm, vec;
};

template <typename T, int G, int VPL, bool THROUGH, typename OutT>
__global__ __launch_bounds__(256) void rt_backward_kernel(RtBackward a) {
  using Row = RtRow<T, G, VPL>;
  constexpr int VEC = Row::VEC;
  const int g = threadIdx.x & (G - 1);
  float b[VPL];
  const float gl = a.slopes != nullptr ? gld<float>(a.grad_loss) : 0.f;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = Row::col(g, v);
    b[v] = a.slopes != nullptr && c < a.E ? gl * gld<float>(a.slopes + c) : 0.f;
  }
  const int64_t per = static_cast<int64_t>(gridDim.x) * (256 / G);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (256 / G) + threadIdx.x / G; t < a.T; t += per) {
    float d[VPL];
    // all loads of the row before anything waits; lane j has slot j of the first G
    const uint8_t real = a.mask == nullptr ? 1 : gld<uint8_t>(a.mask + t);
    Row row;
    row.load(static_cast<const T*>(a.logits) + t * a.E, g, a.E, a.vec);
    int id = -1;
    float gw = 0.f, w = 0.f;
    auto slot = [&](int j) {
      id = -1;
      gw = w = 0.f;
      if (j < a.k) {
        id = gld<int32_t>(a.ids + t * a.k + j);
        gw = gld<float>(a.grad_w + t * a.k + j);
        if (a.renorm) w = gld<float>(a.weights + t * a.k + j);
        if (id < 0 || id >= a.E) {
          id = -1;
          gw = w = 0.f;
        }
      }
    };
    if constexpr (THROUGH) slot(g);
    if (real == 0) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) d[v] = 0.f;
    } else {
      float p[VPL], q[VPL], top;
      const float sum = row.exps(p, top);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        p[v] = rt_over(p[v], sum, inv);
        q[v] = b[v];
        d[v] = 0.f;
      }
      if constexpr (THROUGH) {
        float mean = gw * w;  // sum_j grad_w[j] w[j]
        for (int j0 = G; j0 < a.k && a.renorm; j0 += G) {
          slot(j0 + g);
          mean = __builtin_fmaf(gw, w, mean);
        }
        mean = a.renorm ? rt_sum<G>(mean) : 0.f;
        for (int j0 = 0; j0 < a.k; j0 += G) {
          if (a.k > G) slot(j0 + g);
          const float val = a.renorm ? w * (gw - mean) : gw;
          for (int j = 0; j < min(a.k - j0, G); ++j) {
            const int at = __shfl(id, j, G);
            const float x = __shfl(val, j, G);
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
              const float y = Row::col(g, v) == at ? x : 0.f;
              if (a.renorm) d[v] += y; else q[v] += y;
            }
          }
        }
      }
      float c = 0.f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) c = __builtin_fmaf(p[v], q[v], c);
      c = rt_sum<G>(c);
#pragma unroll
      for (int v = 0; v < VPL; ++v) d[v] = __builtin_fmaf(p[v], q[v] - c, d[v]);
    }
    OutT* const out = static_cast<OutT*>(a.out) + t * a.E;
#pragma unroll
    for (int i = 0; i < VPL / VEC; ++i) {
      const int c = Row::col(g, i * VEC);
      OutT part[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) part[j] = static_cast<OutT>(d[i * VEC + j]);
      if (a.vec) {
        if (c < a.E) {
#pragma unroll
          for (int h = 0; h < static_cast<int>(VEC * sizeof(OutT)) / 16; ++h) {
            u32x4 raw;
            __builtin_memcpy(&raw, reinterpret_cast<const char*>(part) + 16 * h, 16);
            gst<u32x4>(reinterpret_cast<char*>(out + c) + 16 * h, raw);
          }
          if constexpr (VEC * sizeof(OutT) == 8) {
            u32x2 raw;
            __builtin_memcpy(&raw, part, 8);
            gst<u32x2>(out + c, raw);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (c + j < a.E) gst<OutT>(out + c + j, part[j]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------
// Lanes of a row and values of a lane: 8 values while 16 lanes are enough, then 16;
// a lane for each of the top_k at least.
// WIDE: 8 values while 64 lanes are enough, for kernels that wait for memory (balance and
// its gradient, 16411 tokens of 256 experts in fp32: 12 and 15 us with 16 values).
template <bool WIDE = false, typename F>
mi_status rt_shape(int E, int k, F f) {
  const int need = k > 32 ? 64 : k > 16 ? 32 : k > 8 ? 16 : 8;
#define RT_TRY(G_, VPL_)                   \
  if (need <= G_ && E <= G_ * VPL_)        \
    return f(std::integral_constant<int, G_>{}, std::integral_constant<int, VPL_>{});
  RT_TRY(8, 8)
  RT_TRY(16, 8)
  if constexpr (WIDE) {
    RT_TRY(32, 8)
    RT_TRY(64, 8)
  }
  RT_TRY(16, 16)
  RT_TRY(32, 16)
  RT_TRY(64, 16)
#undef RT_TRY
  set_error("router: no shape");
  return MI_EINVAL;
}
template <typename F>
mi_status rt_type(mi_dtype dt, F f) {
  if (dt == MI_BF16) return f(__bf16{});
  if (dt == MI_F16) return f(_Float16{});
  return f(float{});
}

bool rt_vec(const void* p, int64_t E, mi_dtype dt) {
  const int es = dt == MI_F32 ? 4 : 2;
  return aligned16(p) && E % (16 / es) == 0;
}

unsigned rt_blocks(int64_t T, int rows) {
  const int64_t b = (T + rows - 1) / rows;
  return static_cast<unsigned>(b < 4096 ? b : 4096);
}

// One workgroup, and one launch, while its rows go in four rounds at most (as many lanes a row as
// rt_shape gives it); else up to 256 of 64 rows at least.  us in a graph, one workgroup and two
// launches: 64 experts, 256 tokens (two rounds) 7.9 and 8.9, 512 tokens 10.5 and 8.9, where the
// second launch costs the host more than that, 1024 tokens 16.1 and 9.1; 256 experts, 128 tokens
// (four) 10.3 and 11.5, 256 tokens 16.2 and 11.3; 8 experts, 512 tokens (four) 9.7 and 8.6, 4096
// tokens 42 and 9.2.
int rt_balance_blocks(int64_t T, int64_t E) {
  const int64_t lanes = E <= 64 ? 8 : E <= 128 ? 16 : E <= 256 ? 32 : 64;
  if (T <= 4 * (RT_BT / lanes)) return 1;
  const int64_t b = (T + 63) / 64;
  return static_cast<int>(b < RT_BLOCKS ? b : RT_BLOCKS);
}

mi_status rt_sizes(const char* what, int64_t T, int64_t E, int64_t k, mi_dtype dt) {
  MI_REQUIRE(T >= 0 && T < (1LL << 31) / (k > 0 ? k : 1), "%s: num_tokens * top_k must be in [0, 2^31)",
             what);
  MI_REQUIRE(E >= 1 && E <= RT_MAX_EXPERTS, "%s: num_experts must be in [1, %d] (got %lld)", what,
             RT_MAX_EXPERTS, (long long)E);
  MI_REQUIRE(dt == MI_BF16 || dt == MI_F16 || dt == MI_F32,
             "%s: the logits must be bf16, fp16 or fp32", what);
  return MI_OK;
}
mi_status rt_topk(const char* what, int64_t E, int64_t k) {
  MI_REQUIRE(k >= 1 && k <= E && k <= RT_MAX_TOPK,
             "%s: top_k must be in [1, min(num_experts, %d)] (got %lld)", what, RT_MAX_TOPK,
             (long long)k);
  return MI_OK;
}

}  // namespace
}  // namespace mi

extern "C" mi_status mi_moe_route_topk(const void* logits, mi_dtype logits_dtype,
                                       int64_t num_tokens, int64_t num_experts, int64_t top_k,
                                       int renormalize, const uint8_t* token_mask,
                                       float* topk_weights, int32_t* topk_ids, void* stream) {
  using namespace mi;
  clear_error();
  const char* what = "moe_route_topk";
  mi_status st = rt_topk(what, num_experts, top_k);
  if (st == MI_OK) st = rt_sizes(what, num_tokens, num_experts, top_k, logits_dtype);
  if (st != MI_OK || num_tokens == 0) return st;
  MI_REQUIRE(logits != nullptr && topk_weights != nullptr && topk_ids != nullptr,
             "%s: logits, topk_weights or topk_ids is null", what);
  const int64_t in = num_tokens * num_experts * (logits_dtype == MI_F32 ? 4 : 2);
  const int64_t out = num_tokens * top_k * 4;
  MI_REQUIRE(!overlap(topk_weights, out, logits, in) && !overlap(topk_ids, out, logits, in) &&
                 !overlap(topk_ids, out, topk_weights, out) &&
                 !overlap(topk_ids, out, token_mask, num_tokens) &&
                 !overlap(topk_weights, out, token_mask, num_tokens),
             "%s: an output may not overlap another tensor", what);
  RtRoute a{logits, token_mask, topk_weights, topk_ids, static_cast<int>(num_tokens),
            static_cast<int>(num_experts), static_cast<int>(top_k), renormalize != 0,
            rt_vec(logits, num_experts, logits_dtype)};
  return rt_type(logits_dtype, [&](auto type) {
    return rt_shape(a.E, a.k, [&](auto g, auto vpl) {
      constexpr int G = decltype(g)::value, VPL = decltype(vpl)::value;
      hipLaunchKernelGGL((rt_route_kernel<decltype(type), G, VPL>),
                         dim3(rt_blocks(a.T, 256 / G)), dim3(256), 0,
                         static_cast<hipStream_t>(stream), a);
      return launch_status("moe_route_topk");
    });
  });
}

extern "C" size_t mi_moe_balance_loss_workspace_size(int64_t num_tokens, int64_t num_experts) {
  if (num_tokens < 0 || num_experts < 1 || num_experts > mi::RT_MAX_EXPERTS) return 0;
  const size_t b = static_cast<size_t>(mi::rt_balance_blocks(num_tokens, num_experts));
  return (b * (2 * static_cast<size_t>(num_experts) + 2) + (num_experts + 63) / 64 + 1) * 4;
}

extern "C" mi_status mi_moe_balance_loss(const void* logits, mi_dtype logits_dtype,
                                         int64_t num_tokens, int64_t num_experts,
                                         const int32_t* topk_ids, int64_t top_k,
                                         const uint8_t* token_mask, const int32_t* given_counts,
                                         float coef, float* loss, int32_t* counts, float* slopes,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  using namespace mi;
  clear_error();
  const char* what = "moe_balance_loss";
  MI_REQUIRE(top_k >= 1 && top_k < (1LL << 31), "%s: top_k must be at least 1 (got %lld)", what,
             (long long)top_k);
  const mi_status st = rt_sizes(what, num_tokens, num_experts, top_k, logits_dtype);
  if (st != MI_OK) return st;
  MI_REQUIRE(loss != nullptr && counts != nullptr && slopes != nullptr,
             "%s: loss, counts or slopes is null", what);
  MI_REQUIRE(num_tokens == 0 || (logits != nullptr && topk_ids != nullptr),
             "%s: logits or topk_ids is null", what);
  const size_t need = mi_moe_balance_loss_workspace_size(num_tokens, num_experts);
  MI_REQUIRE(workspace != nullptr && workspace_bytes >= need &&
                 (reinterpret_cast<uintptr_t>(workspace) & 3) == 0,
             "%s: the workspace needs %zu bytes, aligned to 4 (got %zu)", what, need,
             workspace_bytes);
  const int64_t in = num_tokens * num_experts * (logits_dtype == MI_F32 ? 4 : 2);
  const int64_t eb = num_experts * 4;
  const struct { const void* p; int64_t n; } outs[4] = {
      {loss, 4}, {counts, eb}, {slopes, eb}, {workspace, static_cast<int64_t>(need)}};
  for (int i = 0; i < 4; ++i) {
    MI_REQUIRE(!overlap(outs[i].p, outs[i].n, logits, in) &&
                   !overlap(outs[i].p, outs[i].n, topk_ids, num_tokens * top_k * 4) &&
                   !overlap(outs[i].p, outs[i].n, token_mask, num_tokens) &&
                   !overlap(outs[i].p, outs[i].n, given_counts, eb),
               "%s: an output or the workspace may not overlap an input", what);
    for (int j = 0; j < i; ++j)
      MI_REQUIRE(!overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n),
                 "%s: the outputs and the workspace may not overlap each other", what);
  }
  const int blocks = rt_balance_blocks(num_tokens, num_experts);
  RtBalance a{};
  a.logits = logits;
  a.ids = topk_ids;
  a.mask = token_mask;
  a.given = given_counts;
  a.part_p = static_cast<float*>(workspace);
  a.part_c = reinterpret_cast<int32_t*>(a.part_p + static_cast<size_t>(blocks) * num_experts);
  a.terms = reinterpret_cast<float*>(a.part_c + static_cast<size_t>(blocks) * (num_experts + 2));
  a.ended = reinterpret_cast<int32_t*>(a.terms + (num_experts + 63) / 64);
  a.loss = loss;
  a.counts = counts;
  a.slopes = slopes;
  a.T = static_cast<int>(num_tokens);
  a.E = static_cast<int>(num_experts);
  a.k = static_cast<int>(top_k);
  a.blocks = blocks;
  a.coef = coef;
  a.vec = rt_vec(logits, num_experts, logits_dtype);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return rt_type(logits_dtype, [&](auto type) {
    return rt_shape<true>(a.E, 1, [&](auto g, auto vpl) {
      constexpr int G = decltype(g)::value, VPL = decltype(vpl)::value;
      hipLaunchKernelGGL((rt_balance_kernel<decltype(type), G, VPL>), dim3(blocks), dim3(RT_BT),
                         0, s, a);
      const mi_status one = launch_status("moe_balance_loss");
      if (one != MI_OK || blocks == 1) return one;
      hipLaunchKernelGGL(rt_balance_finish_kernel, dim3((a.E + 63) / 64), dim3(RT_BT), 0, s, a);
      return launch_status("moe_balance_loss (finish)");
    });
  });
}

extern "C" mi_status mi_moe_route_backward(const void* logits, mi_dtype logits_dtype,
                                           int64_t num_tokens, int64_t num_experts,
                                           const int32_t* topk_ids, const float* topk_weights,
                                           const float* grad_weights, int64_t top_k,
                                           int renormalize, const float* slopes,
                                           const float* grad_loss, const uint8_t* token_mask,
                                           void* grad_logits, mi_dtype grad_dtype, void* stream) {
  using namespace mi;
  clear_error();
  const char* what = "moe_route_backward";
  const bool through = grad_weights != nullptr;
  MI_REQUIRE(through || slopes != nullptr, "%s: grad_weights or slopes is needed", what);
  MI_REQUIRE((slopes == nullptr) == (grad_loss == nullptr),
             "%s: slopes and grad_loss are given together", what);
  MI_REQUIRE(!through || (top_k >= 1 && top_k < (1LL << 31)),
             "%s: top_k must be at least 1 (got %lld)", what, (long long)top_k);
  const mi_status st = rt_sizes(what, num_tokens, num_experts, through ? top_k : 1, logits_dtype);
  if (st != MI_OK) return st;
  MI_REQUIRE(grad_dtype == MI_BF16 || grad_dtype == MI_F16 || grad_dtype == MI_F32,
             "%s: grad_logits must be bf16, fp16 or fp32", what);
  if (num_tokens == 0) return MI_OK;
  MI_REQUIRE(logits != nullptr && grad_logits != nullptr, "%s: logits or grad_logits is null", what);
  MI_REQUIRE(!through || (topk_ids != nullptr && (!renormalize || topk_weights != nullptr)),
             "%s: grad_weights needs topk_ids, and topk_weights if they are renormalised", what);
  const int64_t n = num_tokens * num_experts, in = n * (logits_dtype == MI_F32 ? 4 : 2);
  const int64_t ob = n * (grad_dtype == MI_F32 ? 4 : 2), pick = num_tokens * top_k * 4;
  // a row is read whole before it is written, so the gradient may take the logits' place
  MI_REQUIRE((grad_logits == logits && ob == in) || !overlap(grad_logits, ob, logits, in),
             "%s: grad_logits may be logits itself, but not overlap it otherwise", what);
  MI_REQUIRE(!(through && (overlap(grad_logits, ob, topk_ids, pick) ||
                           overlap(grad_logits, ob, topk_weights, pick) ||
                           overlap(grad_logits, ob, grad_weights, pick))) &&
                 !overlap(grad_logits, ob, slopes, num_experts * 4) &&
                 !overlap(grad_logits, ob, grad_loss, 4) &&
                 !overlap(grad_logits, ob, token_mask, num_tokens),
             "%s: grad_logits may not overlap another input", what);
  RtBackward a{logits, topk_ids, topk_weights, grad_weights, slopes, grad_loss, token_mask,
               grad_logits, static_cast<int>(num_tokens), static_cast<int>(num_experts),
               static_cast<int>(through ? top_k : 0), renormalize != 0,
               rt_vec(logits, num_experts, logits_dtype) && aligned16(grad_logits)};
  return rt_type(logits_dtype, [&](auto type) {
    return rt_type(grad_dtype, [&](auto otype) {
      return rt_shape<true>(a.E, 1, [&](auto g, auto vpl) {
        constexpr int G = decltype(g)::value, VPL = decltype(vpl)::value;
        const dim3 grid(rt_blocks(a.T, 256 / G));
        hipStream_t s = static_cast<hipStream_t>(stream);
        if (through)
          hipLaunchKernelGGL((rt_backward_kernel<decltype(type), G, VPL, true, decltype(otype)>), grid, dim3(256), 0, s, a);
        else
          hipLaunchKernelGGL((rt_backward_kernel<decltype(type), G, VPL, false, decltype(otype)>), grid, dim3(256), 0, s, a);
        return launch_status("moe_route_backward");
      });
    });
  });
}
