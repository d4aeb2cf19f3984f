// A shared projection with the low-rank adapters of many requests beside it, and
// the gradients, on gfx950.  With l = ids[t] the adapter of row t (none where it
// lies outside [0, L)):
//
//   v[t]   = x[t] A[l]^T                                   [R], fp32
//   out[t] = x[t] w^T + bias + s[l] v[t] B[l]^T            [N], rounded once
//   u[t]   = go[t] B[l]                                    [R], fp32
//   gx[t]  = go[t] w + s[l] u[t] A[l]                      [K], rounded once
//   gA[l]  = s[l] sum_{t of l} u[t]^T x[t]                 [R, K]
//   gB[l]  = s[l] sum_{t of l} go[t]^T v[t]                [N, R]
//
// Steps, each a launch on the caller's stream:
//   plan    (one launch or two) sorts the rows by adapter (stable), cuts every adapter's
//           rows into items of 32 and its items into chunks
//   shrink  v (or u) of an item; kept as three bf16 pieces whose sum has 24 bits,
//           so that the second product runs on bf16 MFMAs without a rounding of v
//   mm      the dense product over rows in sorted order, the adapters' part added
//           to the same accumulators before the one rounding
//   grads   gA and gB of a chunk of an adapter's rows, from the pieces; partial sums
//           where an adapter has several chunks
//   reduce  those partial sums in order
#include "common.hpp"

namespace mi {
namespace {

typedef __attribute__((address_space(3))) void* lds_void_ptr;
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_ptr;
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int LM_MAX_ADAPTERS = 1024;
constexpr int LM_MAX_RANK = 256;
constexpr int LM_ITEM = 32;            // rows of an item
constexpr int LM_BK = 64;              // 128 bytes of a row of x: one step
constexpr uint32_t LM_OUT = 0x80000000u;  // past every descriptor's range

__device__ __forceinline__ lds_void_ptr lm_lds(void* p) { return (lds_void_ptr)(p); }

// the sorted rows and what is cut from them
struct LmPlan {
  int* rank;        // [T] of a row among its chunk's rows of its adapter
  int* counts;      // [chunks, L + 1] of adapters' rows
  i32x2* order;     // [T] {row, adapter}; rows without one last, adapter L
  int* item_id;     // adapter of every item
  int* slot_row;    // [LM_ITEM * items] row of every slot of an item, -1: none
  i32x4* chunks;     // {adapter, first item, items, place of its partial sums or -1}
  i32x4* spans;      // [L] {first chunk, chunks, first partial place or -1, 0}
  int* totals;      // items of adapters, chunks, items with those of rows without one
  uint16_t* zeros;  // 16 bytes of zeros
};

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
constexpr int PL_T = 1024, PL_W = PL_T / 64, PL_S = PL_W + 1;

// exclusive sums over the workgroup of two values at once, all of them in `total`
struct PlPair { uint64_t a, b; };
__device__ __forceinline__ PlPair pl_scan(PlPair v, PlPair* s, PlPair* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto upto = [&](PlPair x, int width) {
#pragma unroll 1
    for (int o = 1; o < width; o <<= 1) {
      const uint64_t a = __shfl_up(x.a, o, 64), b = __shfl_up(x.b, o, 64);
      if (lane >= o) {
        x.a += a;
        x.b += b;
      }
    }
    return x;
  };
  const PlPair incl = upto(v, 64);
  if (lane == 63) s[wave] = incl;
  __syncthreads();
  const PlPair all = upto(lane < PL_W ? s[lane] : PlPair{0, 0}, PL_W);
  *total = {__shfl(all.a, PL_W - 1, 64), __shfl(all.b, PL_W - 1, 64)};
  const uint64_t a = __shfl(all.a, wave - 1, 64), b = __shfl(all.b, wave - 1, 64);
  return {incl.a - v.a + (wave ? a : 0), incl.b - v.b + (wave ? b : 0)};
}

// lanes of the wavefront that hold the same value
__device__ __forceinline__ uint64_t pl_peers(int v, int bits) {
  uint64_t peers = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool bit = (v >> b) & 1;
    const uint64_t bal = __ballot(bit);
    peers &= bit ? bal : ~bal;
  }
  return peers;
}

// Up to PL_ONE rows one workgroup does it all; beyond, two launches of a workgroup per
// chunk of rows (1024, or a 64th of them).  count: the chunk's rows of every adapter, and
// each row's rank among its wavefront's; a wavefront's rows go in order.  place: every
// workgroup adds the chunks' counts itself, which gives all places; the first writes the
// lists.  (us, one workgroup and two launches: 1111 rows 5.9 and 9.3, 8192 rows 13.4 and 10.5.)
constexpr int PL_ONE = 4096;

// Counts of the rows [r0, r1) of a wavefront, 64 at a time, into its column of s_cnt; f
// gets every row's id and its rank among the wavefront's rows of that adapter.
template <typename F>
__device__ __forceinline__ void pl_count(const int32_t* ids, int r0, int r1, int L, int* s_cnt, F f) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto id_at = [&](int row) {
    const int id = row < r1 ? gld<int32_t>(ids + row) : L;
    return id < 0 || id > L ? L : id;
  };
  int id = id_at(r0 + lane);
#pragma unroll 1
  for (int i = threadIdx.x; i < (L + 1) * PL_S; i += PL_T) s_cnt[i] = 0;
  __syncthreads();
  const int bits = 32 - __builtin_clz(L);  // ids 0 .. L
  int* const cnt = s_cnt + wave;           // of adapter l at l * PL_S
#pragma unroll 1
  for (int at = r0; at < r1; at += 64) {
    const int row = at + lane, next = id_at(row + 64);
    // the lanes that hold the same id; a run's rows all do
    const uint64_t live = __ballot(row < r1);
    uint64_t peers = __ballot(id == __builtin_amdgcn_readfirstlane(id)) & live;
    if (peers != live) peers = pl_peers(id, bits) & live;
    const uint64_t below = peers & ((1ull << lane) - 1);
    if (row < r1) {
      const int before = cnt[id * PL_S];
      f(row, id, before + __popcll(below));
      if (below == 0) cnt[id * PL_S] = before + __popcll(peers);
    }
    // LDS operations of one wavefront complete in order
    __builtin_amdgcn_wave_barrier();
    id = next;
  }
  __syncthreads();
  // the wavefronts' counts become the counts before them; the sum behind them
  for (int l = threadIdx.x; l <= L; l += PL_T) {
    int run = 0;
#pragma unroll
    for (int w = 0; w < PL_W; ++w) {
      const int c = s_cnt[l * PL_S + w];
      s_cnt[l * PL_S + w] = run;
      run += c;
    }
    s_cnt[l * PL_S + PL_W] = run;
  }
  __syncthreads();
}

__global__ __launch_bounds__(PL_T) void lm_count_kernel(const int32_t* __restrict__ ids, int T,
                                                        int L, int chunk, LmPlan p) {
  __shared__ int s_cnt[(LM_MAX_ADAPTERS + 1) * PL_S];
  const int per = chunk / PL_W, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int r0 = min(static_cast<int>(blockIdx.x) * chunk + wave * per, T), r1 = min(r0 + per, T);
  pl_count(ids, r0, r1, L, s_cnt, [&](int row, int, int rank) { gst<int>(p.rank + row, rank); });
  for (int l = threadIdx.x; l <= L; l += PL_T)
    gst<int>(p.counts + static_cast<int64_t>(blockIdx.x) * (L + 1) + l, s_cnt[l * PL_S + PL_W]);
#pragma unroll 2
  for (int row = r0 + lane; row < r1; row += 64) {
    const int id = gld<int32_t>(ids + row), l = id < 0 || id > L ? L : id;
    const int add = s_cnt[l * PL_S + wave];
    if (add) gst<int>(p.rank + row, gld<int>(p.rank + row) + add);
  }
}

template <bool ONE>
__global__ __launch_bounds__(PL_T) void lm_place_kernel(const int32_t* __restrict__ ids, int T,
                                                        int L, int chunk, int chunk_items,
                                                        LmPlan p) {
  __shared__ int s_cnt[ONE ? (LM_MAX_ADAPTERS + 1) * PL_S : 1];
  __shared__ int s_base[LM_MAX_ADAPTERS + 1];  // place of this chunk's first row
  __shared__ int s_seg[LM_MAX_ADAPTERS + 1], s_item0[LM_MAX_ADAPTERS + 2];
  __shared__ PlPair s_scan[PL_W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int blocks = ONE ? 1 : gridDim.x, block = ONE ? 0 : blockIdx.x;
  const bool lists = block == 0;
  const int per = ((T + PL_W - 1) / PL_W + 63) & ~63;  // ONE: rows of a wavefront
  const int w0 = min(wave * per, T), w1 = min(w0 + per, T);
  int rank_of[PL_ONE / PL_T], id_of[PL_ONE / PL_T];
  if constexpr (ONE)
    pl_count(ids, w0, w1, L, s_cnt, [&](int row, int id, int rank) {
#pragma unroll
      for (int i = 0; i < PL_ONE / PL_T; ++i)
        if (row == w0 + 64 * i + lane) {
          rank_of[i] = rank;
          id_of[i] = id;
        }
    });
  // thread l: adapter l
  int rows = 0, mine = 0;
  if (tid < L) {
    if constexpr (ONE) {
      rows = s_cnt[tid * PL_S + PL_W];
    } else {
#pragma unroll 4
      for (int c = 0; c < blocks; ++c) {
        const int v = gld<int>(p.counts + static_cast<int64_t>(c) * (L + 1) + tid);
        rows += v;
        mine += c < block ? v : 0;
      }
    }
  }
  const int items = (rows + LM_ITEM - 1) / LM_ITEM;
  const int chunks = tid < L ? max((items + chunk_items - 1) / chunk_items, 1) : 0;
  PlPair all;
  const PlPair before =
      pl_scan({static_cast<uint64_t>(rows) | static_cast<uint64_t>(items) << 32,
               static_cast<uint64_t>(chunks) | static_cast<uint64_t>(chunks > 1 ? chunks : 0) << 32},
              s_scan, &all);
  const int seg = static_cast<int>(before.a), item0 = static_cast<int>(before.a >> 32);
  const int chunk0 = static_cast<int>(before.b), part0 = static_cast<int>(before.b >> 32);
  // the rows without an adapter follow, in items of their own
  const int in = static_cast<int>(all.a), real = static_cast<int>(all.a >> 32);
  const int more = (T - in + LM_ITEM - 1) / LM_ITEM;
  if (tid < L) {
    s_base[tid] = seg + mine;
    s_seg[tid] = seg;
    s_item0[tid] = item0;
    if (lists) {
#pragma unroll 1
      for (int c = 0; c < chunks; ++c)
        gst<i32x4>(p.chunks + chunk0 + c,
                   i32x4{tid, item0 + c * chunk_items, min(items - c * chunk_items, chunk_items),
                         chunks > 1 ? part0 + c : -1});
      gst<i32x4>(p.spans + tid, i32x4{chunk0, chunks, chunks > 1 ? part0 : -1, 0});
#pragma unroll 1
      for (int i = rows; i < items * LM_ITEM; ++i) gst<int>(p.slot_row + item0 * LM_ITEM + i, -1);
    }
  }
  if (tid == PL_T - 1) {
    int run = in;
#pragma unroll 4
    for (int c = 0; c < block; ++c) run += gld<int>(p.counts + static_cast<int64_t>(c) * (L + 1) + L);
    s_base[L] = run;
    s_seg[L] = in;
    s_item0[L] = real;
    s_item0[L + 1] = real + more;
    if (lists) {
      gst<i32x4>(p.totals, i32x4{real, static_cast<int>(all.b), real + more, 0});
      gst<u32x4>(p.zeros, u32x4{0, 0, 0, 0});
#pragma unroll 1
      for (int i = T - in; i < more * LM_ITEM; ++i) gst<int>(p.slot_row + real * LM_ITEM + i, -1);
    }
  }
  __syncthreads();
  auto put = [&](int row, int id, int rank_in) {
    const int pos = s_base[id] + rank_in, rank = pos - s_seg[id];
    const int item = s_item0[id] + rank / LM_ITEM;
    // all so where the ids did not change between the passes
    if (rank < 0 || pos >= T || item >= s_item0[id + 1]) return;
    gst<i32x2>(p.order + pos, i32x2{row, id});
    gst<int>(p.slot_row + item * LM_ITEM + rank % LM_ITEM, row);
    if (rank % LM_ITEM == 0) gst<int>(p.item_id + item, id);
  };
  if constexpr (ONE) {
#pragma unroll
    for (int i = 0; i < PL_ONE / PL_T; ++i) {
      const int row = w0 + 64 * i + lane;
      if (row < w1) put(row, id_of[i], rank_of[i] + s_cnt[id_of[i] * PL_S + wave]);
    }
  } else {
    const int r1 = min((block + 1) * chunk, T);
#pragma unroll 4
    for (int row = block * chunk + tid; row < r1; row += PL_T) {
      const int id = gld<int32_t>(ids + row);
      put(row, id < 0 || id > L ? L : id, gld<int>(p.rank + row));
    }
  }
}

// ---------------------------------------------------------------------------
// numbers
// ---------------------------------------------------------------------------
template <bool F16>
__device__ __forceinline__ f32x4 lm_mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <bool F16>
__device__ __forceinline__ float lm_half(uint16_t h) {
  return F16 ? static_cast<float>(__builtin_bit_cast(_Float16, h)) : bf16_bits_to_f32(h);
}

// bf16 pieces of v: each the rounding of what the ones before leave, 24 bits together.  A finite
// v past the largest bf16 has that one as its first.  An infinity or NaN is the last piece,
// behind 1 with its sign: the products with the first two stay finite.
struct LmPieces { uint16_t p[3]; };
__device__ __forceinline__ LmPieces lm_pieces(float v) {
  const uint32_t bits = __float_as_uint(v);
  const bool odd = (bits & 0x7f800000u) == 0x7f800000u;
  LmPieces o;
  float rest = odd ? __builtin_copysignf(1.f, v) : v;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    uint16_t h = __builtin_bit_cast(uint16_t, static_cast<__bf16>(rest));
    if (i == 0 && (h & 0x7f80) == 0x7f80) --h;
    o.p[i] = h;
    rest -= bf16_bits_to_f32(h);
  }
  if (odd) o.p[2] = static_cast<uint16_t>(bits >> 16 | (bits & 0xffffu ? 1u : 0u));
  return o;
}

// A sum over pieces takes an infinity or NaN of its other factor once, with the first piece and
// on its own: the later pieces are 0 or of the other sign, and would make NaN of an infinity.
// In the sum itself 1 with its sign stands in its place.
//
// The largest magnitudes of bf16 values, two a word and each doubled, and whether one of
// them is not finite
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 lm_top(u32x4 q, u16x2 top) {
#pragma unroll
  for (int i = 0; i < 4; ++i) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, q[i] << 1));
  return top;
}
__device__ __forceinline__ bool lm_odd(u16x2 top) { return max(top.x, top.y) >= 0xff00; }
// the values that are not finite (else 0), and those that are (else 1 with the sign)
struct LmOdd { u32x4 odd, rest; };
__device__ __forceinline__ LmOdd lm_part(u32x4 q) {
  LmOdd o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t hit = ((q[i] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
    const uint32_t low = hit - (hit >> 15);  // all bits but the sign
    o.odd[i] = q[i] & (hit | low);
    o.rest[i] = (q[i] & ~low) | (0x3f803f80u & low);
  }
  return o;
}

// eight fp16 values as two bf16 pieces, exact: fp16 has 11 bits, and no exponent that
// bf16 lacks (not finite: second piece 0)
__device__ __forceinline__ void lm_split(u32x4 h, u32x4& hi, u32x4& lo) {
  const f16x8 f = __builtin_bit_cast(f16x8, h);
  bf16x8 a, b;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = static_cast<float>(f[i]);
    a[i] = static_cast<__bf16>(v);
    const float rest = v - static_cast<float>(a[i]);
    b[i] = static_cast<__bf16>(rest == rest ? rest : 0.f);
  }
  hi = __builtin_bit_cast(u32x4, a);
  lo = __builtin_bit_cast(u32x4, b);
}

// eight values of one column, down the rows: two transposed reads of four rows
__device__ __forceinline__ u32x4 lm_column(const uint8_t* first, const uint8_t* second) {
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(first));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(second));
  const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
  return u32x4{x[0], x[1], y[0], y[1]};
}

// chunk c (16 bytes) of LDS row R sits at slot c ^ lm_swz(R)
__device__ __forceinline__ int lm_swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// ---------------------------------------------------------------------------
// shrink: one item's rows times its adapter's matrix.
//   BT == false: bank [L, R, C], v[t, r] = sum_c x[t, c] bank[l, r, c]
//   BT == true:  bank [L, C, R], v[t, r] = sum_c x[t, c] bank[l, c, r]
// A workgroup has the item's rows and 16 NB ranks; its wavefronts take steps of 64 columns
// in turn, and their sums are added in order in LDS.  Bound by the reads of x, once, beside the
// bank's from the L2: 8192 rows of 4096 columns, rank 16: 21 us (67 MB: 3.3 TB/s), transposed, with
// the pieces of both orders, 27; 16 adapters of rank 64 24 us.
// ---------------------------------------------------------------------------
struct LmShrink {
  const void* x;          // [T, C]
  const void* bank;
  const float* scale;     // [L] or null
  const float* act;       // [T, R]: split into pieces_t2 beside pieces_t
  LmPlan plan;
  float* out;             // [T, R] unscaled, or null
  uint16_t* pieces;       // [T, 3 RP] scaled, or null
  uint16_t* pieces_t;     // [3 RP, slots] scaled, or null
  uint16_t* pieces_t2;    // the same of act
  int T, C, L, R, RP, slots;
};

// Loads go straight into LDS, a line of 128 bytes of each row at a time, and from there
// into MFMA operands; a wavefront has its own stages, ST steps of them in flight, and no
// barrier.  (Loads straight into operand registers touch half a line of 16 rows an
// instruction: 8192 rows, 4096 columns, rank 16: 28 us against 20, rank 64: 34 against 23.)
template <int NB>
struct LmShape {
  static constexpr int W = NB <= 2 ? 8 : 4;                  // wavefronts
  static constexpr int ST = NB == 2 ? 2 : 3;                 // stages
  static constexpr int X = LM_ITEM * 128, BYTES = X + NB * 2048;  // of a wavefront's stage
};

template <bool F16, bool BT, int NB>
__device__ __forceinline__ void lm_shrink(const LmShrink& a, uint8_t* s0, uint8_t* s1, uint8_t* s2, f32x4* red) {
  using Shape = LmShape<NB>;
  constexpr int FM = LM_ITEM / 16, W = Shape::W, ST = Shape::ST, NX = LM_ITEM / 8, CPR = 2 * NB, NI = NX + CPR;
  const int item = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
  const int* const slots = a.plan.slot_row + item * LM_ITEM;
  const int R = a.R, rank0 = blockIdx.y * 16 * NB;
  // all that the plan says of the item at once (past the last item it is not used)
  const i32x4 totals = gld<i32x4>(a.plan.totals);
  const int l = __builtin_amdgcn_readfirstlane(gld<int>(a.plan.item_id + item));
  const int r = lane & 15, g = lane >> 4, lr = lane >> 3;
  int row_of[NX];
#pragma unroll
  for (int i = 0; i < NX; ++i) row_of[i] = gld<int>(slots + 8 * i + lr);
  if (item >= totals.z) return;
  if (item >= totals.x) {  // rows without an adapter: zeros for activations
    if (a.out != nullptr)
      for (int q = tid; q < LM_ITEM * NB * 4; q += 64 * W) {
        const int t = gld<int>(slots + q / (NB * 4)), rk = rank0 + q % (NB * 4) * 4;
        if (t >= 0 && rk < R) gst<f32x4>(a.out + static_cast<int64_t>(t) * R + rk, f32x4{0.f, 0.f, 0.f, 0.f});
      }
    return;
  }
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int C = a.C, KT = (C + LM_BK - 1) / LM_BK;
  const __amdgpu_buffer_rsrc_t xr =
      buf_rsrc(a.x, static_cast<uint32_t>(a.T) * static_cast<uint32_t>(C) * 2u);
  const __amdgpu_buffer_rsrc_t br =
      buf_rsrc(static_cast<const uint16_t*>(a.bank) + static_cast<int64_t>(l) * R * C,
               static_cast<uint32_t>(R) * static_cast<uint32_t>(C) * 2u);
  // instruction i of x: rows 8 i .. 8 i + 7, lane (row, slot) the chunk that the slot holds
  uint32_t vx[NX], vb[CPR];
  uint32_t cx[2];  // byte of a row's step that this lane's chunk starts at, even and odd i
#pragma unroll
  for (int i = 0; i < 2; ++i) cx[i] = ((lane & 7) ^ lr ^ i) * 16;
#pragma unroll
  for (int i = 0; i < NX; ++i)
    vx[i] = row_of[i] >= 0 ? static_cast<uint32_t>(row_of[i]) * C * 2 + cx[i & 1] : LM_OUT;
#pragma unroll
  for (int i = 0; i < CPR; ++i) {
    if constexpr (BT) {  // 64 rows of CPR chunks
      const int at = i * 64 + lane, rk = rank0 + at % CPR * 8;
      vb[i] = rk < R ? (static_cast<uint32_t>(at / CPR) * R + rk) * 2 : LM_OUT;
    } else {
      const int rk = rank0 + 8 * i + lr;
      vb[i] = rk < R ? static_cast<uint32_t>(rk) * C * 2 + cx[i & 1] : LM_OUT;
    }
  }
  auto load = [&](uint8_t* st, int kt) {  // a step past the last loads zeros
    const int kb = min(kt, KT - 1);
    const uint32_t so = __builtin_amdgcn_readfirstlane(kb * (LM_BK * 2));
    uint32_t drop[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) drop[i] = kt < KT && so + cx[i] < static_cast<uint32_t>(C) * 2 ? 0u : LM_OUT;
#pragma unroll
    for (int i = 0; i < NX; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, lm_lds(st + i * 1024), 16, vx[i] | drop[i & 1], so, 0, 0);
    const uint32_t sob = BT ? __builtin_amdgcn_readfirstlane(kb * (LM_BK * 2) * R) : so;
#pragma unroll
    for (int i = 0; i < CPR; ++i) {
      const uint32_t d = !BT ? drop[i & 1] : kt < KT && kb * LM_BK + (i * 64 + lane) / CPR < C ? 0u : LM_OUT;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(br, lm_lds(st + Shape::X + i * 1024), 16, vb[i] | d, sob, 0, 0);
    }
  };
  f32x4 acc[FM][NB];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int ck = ((g & 1) << 1) | (g >> 1);
  auto add = [&](uint8_t* st, int next) {
    __builtin_amdgcn_s_waitcnt((((ST - 1) * NI) & 15) | ((((ST - 1) * NI) >> 4) << 14) | (15 << 8) | (7 << 4));
    asm volatile("" ::: "memory");
    u32x4 fx[FM][2], fb[NB][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = r * 128 + ((ck + 4 * h) ^ lm_swz(r)) * 16;
#pragma unroll
      for (int i = 0; i < FM; ++i) fx[i][h] = *reinterpret_cast<const u32x4*>(st + i * 2048 + at);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if constexpr (BT) {
          const uint8_t* b = st + Shape::X + (8 * ck + 32 * h + (r >> 2)) * (NB * 32) + j * 32 + (r & 3) * 8;
          fb[j][h] = lm_column(b, b + 4 * NB * 32);
        } else {
          fb[j][h] = *reinterpret_cast<const u32x4*>(st + Shape::X + j * 2048 + at);
        }
      }
    }
    // the stage is free once its reads have returned
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    load(st, next);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i) acc[i][j] = lm_mfma<F16>(fb[j][h], fx[i][h], acc[i][j]);
    __builtin_amdgcn_sched_barrier(0);
  };
  uint8_t* const sts[3] = {s0 + wave * Shape::BYTES, s1 + wave * Shape::BYTES, s2 + wave * Shape::BYTES};
#pragma unroll
  for (int u = 0; u < ST; ++u) load(sts[u], wave + W * u);
  for (int kt = wave; kt < KT; kt += W * ST) {
#pragma unroll
    for (int u = 0; u < ST; ++u) add(sts[u], kt + W * (u + ST));
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);  // the steps past the last have written their zeros
  __syncthreads();
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) red[((wave * FM + i) * NB + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  constexpr int LM_COLS = LM_ITEM + 1;
  static_assert(16 * NB * LM_COLS * 4 * 2 <= W * Shape::BYTES, "columns in a stage");
  float* const cols[2] = {reinterpret_cast<float*>(s1), reinterpret_cast<float*>(s1) + 16 * NB * LM_COLS};
  // quad: ranks 16 j + 4 g .. of slot 16 i + r
  const float s = a.scale != nullptr ? gld<float>(a.scale + l) : 1.f;
  for (int at = tid; at < FM * NB * 64; at += 64 * W) {
    f32x4 v = red[at];
#pragma unroll
    for (int w = 1; w < W; ++w) v += red[w * FM * NB * 64 + at];
    const int j = (at >> 6) % NB, in = at / (64 * NB) * 16 + (at & 15);
    const int rk = rank0 + 16 * j + 4 * ((at & 63) >> 4);
    if (rk >= a.RP) continue;
    const int slot = item * LM_ITEM + in, t = gld<int>(slots + in);
    const bool here = t >= 0 && rk < R;
    const f32x4 none = {0.f, 0.f, 0.f, 0.f};
    if (a.out != nullptr && here) gst<f32x4>(a.out + static_cast<int64_t>(t) * R + rk, v);
    if (a.pieces != nullptr && t >= 0) {
      LmPieces p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = lm_pieces(here ? v[i] * s : 0.f);
#pragma unroll
      for (int c = 0; c < 3; ++c)
        gst<u32x2>(a.pieces + (static_cast<int64_t>(t) * 3 + c) * a.RP + rk,
                   u32x2{p[0].p[c] | static_cast<uint32_t>(p[1].p[c]) << 16,
                         p[2].p[c] | static_cast<uint32_t>(p[3].p[c]) << 16});
    }
    if (a.pieces_t != nullptr) {
      f32x4 w = none;
      if (here) w = gld<f32x4>(a.act + static_cast<int64_t>(t) * R + rk);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cols[0][(16 * j + 4 * ((at & 63) >> 4) + i) * LM_COLS + in] = here ? v[i] * s : 0.f;
        cols[1][(16 * j + 4 * ((at & 63) >> 4) + i) * LM_COLS + in] = here ? w[i] * s : 0.f;
      }
    }
  }
  if (a.pieces_t == nullptr) return;
  // down the columns: 8 slots of a rank at a time
  __syncthreads();
  for (int q = tid; q < 2 * 16 * NB * (LM_ITEM / 8); q += 64 * W) {
    const int which = q / (16 * NB * (LM_ITEM / 8)), rank = q / (LM_ITEM / 8) % (16 * NB), in = q % (LM_ITEM / 8) * 8;
    if (rank0 + rank >= a.RP) continue;
    uint16_t part[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const LmPieces p = lm_pieces(cols[which][rank * LM_COLS + in + i]);
#pragma unroll
      for (int c = 0; c < 3; ++c) part[c][i] = p.p[c];
    }
    uint16_t* const to = which ? a.pieces_t2 : a.pieces_t;
#pragma unroll
    for (int c = 0; c < 3; ++c) {
      u32x4 raw;
      __builtin_memcpy(&raw, part[c], 16);
      gst<u32x4>(to + (static_cast<int64_t>(c) * a.RP + rank0 + rank) * a.slots + item * LM_ITEM + in, raw);
    }
  }
}

template <bool F16, bool BT, int NB>
__global__ __launch_bounds__(64 * LmShape<NB>::W) void lm_shrink_kernel(LmShrink a) {
  // a stage its own array: the compiler then knows which loads a read waits for
  constexpr int SIZE = LmShape<NB>::W * LmShape<NB>::BYTES;
  __shared__ __attribute__((aligned(16))) uint8_t s0[SIZE], s1[SIZE], s2[LmShape<NB>::ST == 3 ? SIZE : 16];
  static_assert(LmShape<NB>::W * LM_ITEM / 16 * NB * 1024 <= SIZE, "the sums fit a stage");
  lm_shrink<F16, BT, NB>(a, s0, s1, s2, reinterpret_cast<f32x4*>(s0));
}

// ---------------------------------------------------------------------------
// mm: out = x w^T (BT: x w) plus the pieces times the adapters' matrix
//   BT == false: w [n, k], bank [L, n, R]
//   BT == true:  w [k, n], bank [L, R, n]
// Bound by the MFMAs of the dense part, in the trace of a warm card: 8192 rows, n = k = 4096, rank
// 16: 201 us (1.37 PFLOP/s; 181 a library product without adapters), transposed 211 (209); 16
// adapters of rank 64 211.  4096 rows, n = k = 8192, a call with its plan and first product 408 us
// (library 347).
// ---------------------------------------------------------------------------
struct LmMm {
  const void* x;          // [T, k]
  const void* w;
  const void* bank;
  const void* bias;       // [n] or null
  const uint16_t* pieces; // [T, 3 RP]
  LmPlan plan;
  void* out;              // [T, n]; of several splits fp32 [splits, T, n]
  int T, k, n, L, R, RP;
  int splits, blocks;     // of the k axis, and workgroups of each
};

// 32-byte pieces of a transposed tile's row (BN / 16 of them): the 16 rows that a
// transposed read touches lie in 8 different ones of 256 bytes
template <int BN>
__device__ __forceinline__ int lm_tswz(int row) {
  if constexpr (BN >= 128) return (row & 3) | ((row >> 3) & 1) << 2;
  else return ((row >> 1) & 1) | ((row >> 3) & 1) << 1;
}

template <int N>
__device__ __forceinline__ void lm_wait_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));  // vmcnt(N) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// Where a tile lies in the call: m-tiles in groups of GM sweep the n-panels together,
// and each XCD has a contiguous run of that order (workgroup ids go to the 8 in turn).
struct LmPlace { int m0, n0, rows, cols, k0, steps, first; };  // first: PART's
template <int BM, int BN>
__device__ __forceinline__ LmPlace lm_place(const LmMm& p, int block) {
  const int nt = (p.n + BN - 1) / BN, mt = (p.T + BM - 1) / BM;
  const int total = nt * mt, per = (total + 7) / 8;
  const int slot = block >> 3, tile = (block & 7) * per + slot;
  if (slot >= per || tile >= total) return {0, 0, 0, 0, 0, 0, 0};
  constexpr int GM = BM >= 256 ? 4 : 8;
  const int grp = tile / (GM * nt), in = tile - grp * GM * nt, gsz = min(mt - grp * GM, GM);
  const int m0 = (grp * GM + in % gsz) * BM, n0 = in / gsz * BN;
  return {m0, n0, min(p.T - m0, BM), min(p.n - n0, BN), 0, (p.k + LM_BK - 1) / LM_BK, 0};
}

// the LDS of one step: w's rows, and x's, of two stages in two halves
struct LmStage { uint8_t *w, *x0, *x1; };

// One tile of BM = 16 FM WM rows and BN = 16 FN WN columns; WM * WN wavefronts of
// 16 FM x 16 FN.  w is the MFMA's first operand, so a lane's results are four
// consecutive columns of one row.
//
// Staging: 1 KB a DMA instruction straight into LDS, NST stages, each an array of its
// own (the compiler then knows which loads a read waits for).  Rows past the call or
// past n and 16-byte chunks past k load as zeros.
//
// A step (64 of k) is FM regions of one 16-row block of x each.  A region reads the
// fragment of the region after the next and issues its 2 FN MFMAs.  The step's one
// barrier stands before its last two regions, whose operands are in registers by then:
// behind it the stage is free for the loads of step kt + NST and the next stage is
// complete, so the last regions read the next step's first fragments.
//
// PART: only the steps [t.k0, t.k0 + t.steps), from the t.first-th of them on and round, rows
// in their own order, no adapters.
template <bool F16, bool BT, bool PART, int WM, int WN, int FM, int FN, int NST, typename OutT>
__device__ __forceinline__ void lm_tile(const LmMm& p, const LmPlace& t, LmStage s0, LmStage s1,
                                        LmStage s2, LmStage s3, i32x2* s_order) {
  constexpr int NW = WM * WN, BM = 16 * FM * WM, BN = 16 * FN * WN;
  constexpr int NIA = BM / 8 / NW, NIB = BN / 8 / NW, NI = NIA + NIB;
  constexpr int STAGE = (BM + BN) * 128;
  constexpr int FLY = (NST - 2) * NI;
  static_assert(NIA * 8 * NW == BM && NIB * 8 * NW == BN && NW % 2 == 0, "tile");
  static_assert(NST >= 2 && NST <= 4 && FLY < 64 && FM >= 2, "stages");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int r = lane & 15, g = lane >> 4;
  const int k = p.k, n = p.n, k0 = t.k0, KT = t.steps, last = (k + LM_BK - 1) / LM_BK - 1;
  const int m0 = t.m0, n0 = t.n0, rows = t.rows, cols = t.cols;

  for (int i = tid; i < BM; i += 64 * NW)
    s_order[i] = i >= rows ? i32x2{-1, p.L} : PART ? i32x2{m0 + i, p.L} : gld<i32x2>(p.plan.order + m0 + i);
  __syncthreads();

  const __amdgpu_buffer_rsrc_t ar =
      buf_rsrc(p.x, static_cast<uint32_t>(p.T) * static_cast<uint32_t>(k) * 2u);
  const __amdgpu_buffer_rsrc_t br =
      buf_rsrc(p.w, static_cast<uint32_t>(n) * static_cast<uint32_t>(k) * 2u);
  const int lr = lane >> 3, chunk = (lane & 7) ^ lr ^ (wave & 1);
  uint32_t va[NIA], vb[NIB];
#pragma unroll
  for (int i = 0; i < NIA; ++i) {
    const int row = s_order[8 * (NW * i + wave) + lr].x;
    va[i] = row >= 0 ? (static_cast<uint32_t>(row) * k + chunk * 8) * 2 : LM_OUT;
  }
  constexpr int CPW = BN / 8;  // 16-byte pieces of a transposed tile's row
  // Two stages: w's rows and the even instructions' rows of x first, then the odd ones'
  auto nth = [](int o) {
    return NST > 2 ? o : o < NIB ? NIA + o : o < NIB + NIA / 2 ? 2 * (o - NIB) : 2 * (o - NIB - NIA / 2) + 1;
  };
  // where instruction i of x's rows goes, and where block i of this wavefront's rows is
  auto to_x = [&](const LmStage& st, int i) {
    return NST > 2 ? st.x0 + (NW * i + wave) * 1024 : (i & 1 ? st.x1 : st.x0) + (NW * (i >> 1) + wave) * 1024;
  };
  auto block_x = [&](const LmStage& st, int i) {
    constexpr int H = FM / 2;
    return NST > 2 ? st.x0 + (wm * FM + i) * 2048 : i < H ? st.x0 + (wm * H + i) * 2048 : st.x1 + (wm * H + i - H) * 2048;
  };
  auto brow = [&](int i) { return ((NW * i + wave) * 64 + lane) / CPW; };
#pragma unroll
  for (int i = 0; i < NIB; ++i) {
    if constexpr (!BT) {
      const int row = 8 * (NW * i + wave) + lr;
      vb[i] = row < cols ? (static_cast<uint32_t>(n0 + row) * k + chunk * 8) * 2 : LM_OUT;
    } else {
      const int row = brow(i), c = lane % CPW;
      const int col = (((c >> 1) ^ lm_tswz<BN>(row)) * 2 + (c & 1)) * 8;
      vb[i] = col < cols ? (static_cast<uint32_t>(row) * n + n0 + col) * 2 : LM_OUT;
    }
  }
  const uint32_t tail = last * LM_BK + chunk * 8 < k ? 0u : LM_OUT;
  // Loads [first, first + count) of the NI of a stage, in the order of `nth`.  A step past
  // the last loads zeros: the steps stay free of branches.
  auto dma = [&](const LmStage& st, int kt, int first, int count) {
    int in = min(kt, KT - 1);
    if constexpr (PART) {
      in += t.first;
      if (in >= KT) in -= KT;
    }
    const int kb = k0 + in;
    const uint32_t drop = kt >= KT ? LM_OUT : 0u, dropa = kb == last ? drop | tail : drop;
    const uint32_t so = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(kb) * (LM_BK * 2));
    const uint32_t sob =
        BT ? __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(kb) * (LM_BK * 2) * n) : so;
#pragma unroll
    for (int o = 0; o < NI; ++o) {
      if (o < first || o >= first + count) continue;
      const int i = nth(o);
      if (i < NIA) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, lm_lds(to_x(st, i)), 16,
                                                 va[i < NIA ? i : 0] | dropa, so, 0, 0);
      } else {
        const int b = i < NIA ? 0 : i - NIA;
        const uint32_t d = !BT ? dropa : kb * LM_BK + brow(b) < k ? drop : LM_OUT;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            br, lm_lds(st.w + (NW * b + wave) * 1024), 16, vb[b] | d, sob, 0, 0);
      }
    }
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Half h of a step's fragment: lane (r, g) holds the 8 values of chunk ck + 4 h, ck =
  // 0, 2, 1, 3 for g = 0 .. 3.  The LDS serves lanes l and l + 32 together, and their
  // chunks have to differ in the lowest bit.
  const int ck = ((g & 1) << 1) | (g >> 1);
  struct Frag { u32x4 h[2]; };
  int fo[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) fo[h] = r * 128 + ((ck + 4 * h) ^ lm_swz(r)) * 16;
  auto frag = [&](const uint8_t* blk) {
    return Frag{{*reinterpret_cast<const u32x4*>(blk + fo[0]),
                 *reinterpret_cast<const u32x4*>(blk + fo[1])}};
  };
  // a transposed tile's rows c8 .. c8 + 7 (c8 % 8 == 0) of column block blk
  auto column = [&](const uint8_t* st, int blk, int c8) {
    const int row = c8 + (r >> 2);
    const uint8_t* a = st + row * (BN * 2) + (blk ^ lm_tswz<BN>(row)) * 32 + (r & 3) * 8;
    if constexpr (BN >= 128) return lm_column(a, a + 4 * BN * 2);  // row + 4: the same place
    const int row2 = row + 4;
    return lm_column(a, st + row2 * (BN * 2) + (blk ^ lm_tswz<BN>(row2)) * 32 + (r & 3) * 8);
  };
  auto frag_a = [&](const LmStage& st, int i) { return frag(block_x(st, i)); };
  auto frag_b = [&](const LmStage& st, int j) {
    if constexpr (BT)
      return Frag{{column(st.w, wn * FN + j, ck * 8), column(st.w, wn * FN + j, ck * 8 + 32)}};
    else
      return frag(st.w + (wn * FN + j) * 2048);
  };
  // A stage's loads go out PPR per region from the one behind the barrier on, over half
  // of the regions.
  constexpr int PPR = (2 * NI + FM - 1) / FM, R0 = FM - 2;
  // Two stages are too few for that: a load would have less than a step to arrive.  They
  // have a second barrier half a step before the first, in region RY: by then w's rows
  // and the first half of every wavefront's blocks of x have been read, and the loads of
  // these for step kt + 2 go out; those of the second half go out behind the barrier in
  // R0, and are waited for in RY.  Every load has a step and a half.
  constexpr int RY = FM / 2 - 2, NY = NIB + NIA / 2, NX = NIA / 2;
  constexpr int PY = (2 * NY + FM - 1) / FM, PX = (2 * NX + FM - 1) / FM;
  static_assert(NST > 2 || (FM >= 4 && NIA == 2 * WM && NIA % 2 == 0), "halves of x");
  Frag fb[FN], fa0, fa1;
  auto step = [&](const LmStage& pv, const LmStage& st, const LmStage& nx, int kt) {
    Frag fbx[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) fbx[j] = fb[j];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if constexpr (NST > 2) {
        if (i == R0) lm_wait_barrier<FLY>();
        if (i >= R0) dma(st, kt + NST, (i - R0) * PPR, PPR);
        else if ((i + 2) * PPR < NI) dma(pv, kt + NST - 1, (i + 2) * PPR, PPR);
      } else {
        if (i == RY || i == R0) lm_wait_barrier<NI>();
        // (first, count) within the part, no further than its end
        auto part = [&](const LmStage& to, int at, int base, int size, int first, int count) {
          if (first < size) dma(to, at, base + first, first + count < size ? count : size - first);
        };
        if (i >= R0) part(st, kt + 2, NY, NX, (i - R0) * PX, PX);
        else if (i >= RY) part(st, kt + 2, 0, NY, (i - RY) * PY, PY);
        else part(pv, kt + 1, NY, NX, (i + 2) * PX, PX);
      }
      const Frag fax = fa0;
      fa0 = fa1;
      fa1 = i < R0 ? frag_a(st, i + 2) : frag_a(nx, i - R0);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          acc[i][j] = lm_mfma<F16>(fbx[j].h[h], fax.h[h], acc[i][j]);
          if (i == FM - 1 && h == 0) fb[j] = frag_b(nx, j);
        }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const LmStage* const sts[4] = {&s0, &s1, &s2, &s3};
  dma(s0, 0, 0, NI);
  if constexpr (NST >= 3) {
    dma(s1, 1, 0, NI);
    if constexpr (NST == 4) dma(s2, 2, 0, NI);
    lm_wait_barrier<FLY>();
    if constexpr (NST == 4) dma(s3, 3, 0, 2 * PPR);  // the rest in step 0
    else dma(s2, 2, 0, 2 * PPR);
  } else {
    dma(s1, 1, 0, NY + (2 * PX < NX ? 2 * PX : NX));  // the rest in step 0
    lm_wait_barrier<NI>();
  }
  fa0 = frag_a(s0, 0);
  fa1 = frag_a(s0, 1);
#pragma unroll
  for (int j = 0; j < FN; ++j) fb[j] = frag_b(s0, j);
  // Whole rounds of the stages, then the rest: a loop that may end inside a round would
  // make the compiler, which follows the loads into each stage, wait at its head for loads
  // of later steps.
  const int rounds = KT / NST * NST;
#define LM_STEP(S_, KT_) step(*sts[(S_ + NST - 1) % NST], *sts[S_ % NST], *sts[(S_ + 1) % NST], KT_)
  for (int kt = 0; kt < rounds; kt += NST) {
    LM_STEP(0, kt);
    LM_STEP(1, kt + 1);
    if constexpr (NST >= 3) LM_STEP(2, kt + 2);
    if constexpr (NST == 4) LM_STEP(3, kt + 3);
  }
  if (KT - rounds >= 1) {
    LM_STEP(0, rounds);
    if constexpr (NST >= 3) {
      if (KT - rounds >= 2) {
        LM_STEP(1, rounds + 1);
        if constexpr (NST == 4) {
          if (KT - rounds == 3) LM_STEP(2, rounds + 2);
        }
      }
    }
  }
#undef LM_STEP
  // the loads of the steps past the last have written their zeros
  lm_wait_barrier<0>();

  // The adapters, one run of rows after another and 64 ranks of an adapter at a time, in two
  // stages: the bank's ranks take w's place in the first, and the three pieces of v x's place
  // there and both places of the second.  Ranks up to 16 need one stage, with the pieces side by
  // side in a row's 64 places and the bank's ranks once for each; the second stage has the next
  // run.  (The bank's ranks staged again for every piece, us a call: 8192 rows, n = k = 4096, 16
  // adapters of rank 64, 244 for 238; 1111 rows fp16, rank 40, with gradients 106 for 97.)  All
  // three pieces, for 16-bit outputs too: where the two parts cancel, what two leave, 2^-17 of
  // the adapters' part, may be more than the sum's half step.
  const int RP = p.RP, R = p.R;
  const bool one = RP == 16;
  const int E = one ? 3 * RP : RP, mask = one ? 15 : -1;
  struct Run { int l, at, end, e; };  // rows [at, end) of adapter l, from rank e on
  auto run_at = [&](int at) {
    const int l = at < rows ? __builtin_amdgcn_readfirstlane(s_order[at].y) : p.L;
    // the rows without an adapter are last
    if (l >= p.L) return Run{p.L, rows, rows, 0};
    int end = at;
#pragma unroll
    for (int i = 0; i < BM; i += 64) end += __popcll(__ballot(s_order[i + lane].y == l));
    return Run{l, at, end, 0};
  };
  auto after = [&](const Run& u) { return u.e + LM_BK < RP ? Run{u.l, u.at, u.end, u.e + LM_BK} : run_at(u.end); };
  const __amdgpu_buffer_rsrc_t pr_ =
      buf_rsrc(p.pieces, static_cast<uint32_t>(p.T) * static_cast<uint32_t>(RP) * 6u);
  auto last_piece = [](const LmStage& st) { return LmStage{nullptr, st.w, st.w + BM * 64}; };
  auto fetch = [&](const LmStage& st, const LmStage& next, const Run& u) {
    if (u.l >= p.L) return;
    const __amdgpu_buffer_rsrc_t lr_ =
        buf_rsrc(static_cast<const uint16_t*>(p.bank) + static_cast<int64_t>(u.l) * R * n,
                 static_cast<uint32_t>(R) * static_cast<uint32_t>(n) * 2u);
    const int e = u.e + chunk * 8;
#pragma unroll
    for (int i = 0; i < NIA; ++i) {
      const int row = 8 * (NW * i + wave) + lr;
      const bool own = row >= u.at && row < u.end && e < E;
      const uint32_t at = own ? (static_cast<uint32_t>(s_order[row].x) * 3 * RP + e) * 2 : LM_OUT;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(pr_, lm_lds(to_x(st, i)), 16, at, 0, 0, 0);
      if (!one) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(pr_, lm_lds(to_x(next, i)), 16, at, RP * 2, 0, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(pr_, lm_lds(to_x(last_piece(next), i)), 16, at, RP * 4, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < NIB; ++i) {
      uint32_t at;
      if constexpr (!BT) {
        const int row = 8 * (NW * i + wave) + lr, rk = e & mask;
        at = row < cols && e < E && rk < R ? (static_cast<uint32_t>(n0 + row) * R + rk) * 2 : LM_OUT;
      } else {
        const int row = brow(i), c = lane % CPW, rk = (u.e + row) & mask;
        const int col = (((c >> 1) ^ lm_tswz<BN>(row)) * 2 + (c & 1)) * 8;
        at = col < cols && u.e + row < E && rk < R ? (static_cast<uint32_t>(rk) * n + n0 + col) * 2 : LM_OUT;
      }
      __builtin_amdgcn_raw_ptr_buffer_load_lds(lr_, lm_lds(st.w + (NW * i + wave) * 1024), 16, at, 0, 0, 0);
    }
  };
  // Rows of other adapters in a block have zeros for their pieces.  What is not finite in the
  // bank is left for the end.
  const int w0 = wm * FM * 16;
  bool odd = false;
  auto adapt = [&](auto pieces, const LmStage& st, const LmStage& next, const Run& u) {
    if (u.at >= w0 + FM * 16 || u.end <= w0) return;
    u32x4 b[FN], lo[FN];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && u.e + 32 >= E) break;
      if (h == 0 || !one) {  // side by side, both halves meet the same ranks
        u16x2 top = {0, 0};
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if constexpr (BT) b[j] = column(st.w, wn * FN + j, ck * 8 + 32 * h);
          else b[j] = *reinterpret_cast<const u32x4*>(st.w + (wn * FN + j) * 2048 + fo[h]);
        }
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if constexpr (F16) lm_split(b[j], b[j], lo[j]);
          top = lm_top(b[j], top);
        }
        if (__builtin_expect(__any(lm_odd(top)), 0)) {
          odd = true;
#pragma unroll
          for (int j = 0; j < FN; ++j) b[j] = lm_part(b[j]).rest;
        }
      }
#pragma unroll
      for (int c = 0; c < pieces.value; ++c) {
        if (c > 0 && one) break;
        const LmStage& xs = c == 0 ? st : c == 1 ? next : last_piece(next);
        auto half_a = [&](int i) { return *reinterpret_cast<const u32x4*>(block_x(xs, i) + fo[h]); };
        // fp16's second piece with the first two of v
        const bool two = F16 && (c == 0 ? !one || h == 0 : c == 1);
        u32x4 a0 = half_a(0), a1 = half_a(1);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          const u32x4 a = a0;
          a0 = a1;
          if (i + 2 < FM) a1 = half_a(i + 2);
          if (w0 + 16 * i + 16 <= u.at || w0 + 16 * i >= u.end) continue;
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = lm_mfma<false>(b[j], a, acc[i][j]);
          if (two)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = lm_mfma<false>(lo[j], a, acc[i][j]);
        }
      }
    }
  };
  // of a k axis in splits, the last one has the adapters
  if (!PART && k0 + KT == last + 1) {
    constexpr std::integral_constant<int, 3> three{};
    constexpr std::integral_constant<int, 1> first{};
    Run u = run_at(0);
    if constexpr (NST == 4) {
      while (u.l < p.L) {  // as many as the stages hold at once
        Run q[NST];
#pragma unroll
        for (int i = 0; i < NST; ++i) {
          const bool more = i % 2 == 0 || one;
          q[i] = more ? u : Run{p.L, rows, rows, 0};
          if (more) u = after(u);
        }
#pragma unroll
        for (int i = 0; i < NST; ++i) fetch(*sts[i], *sts[i ^ 1], q[i]);
        lm_wait_barrier<0>();
#pragma unroll
        for (int i = 0; i < NST; i += 2) {
          adapt(three, *sts[i], *sts[i + 1], q[i]);
          if (one) adapt(first, *sts[i + 1], *sts[i], q[i + 1]);
        }
        if (u.l < p.L) lm_wait_barrier<0>();  // all have read what is there
      }
    } else {
      fetch(s0, s1, u);
      while (u.l < p.L) {  // of runs with one stage, the next one's loads beside this one's sums
        lm_wait_barrier<0>();
        const Run v = after(u);
        if (one) fetch(s1, s0, v);
        adapt(three, s0, s1, u);
        if (v.l >= p.L) break;
        lm_wait_barrier<0>();
        u = one ? after(v) : v;
        fetch(s0, s1, u);
        if (one) adapt(first, s1, s0, v);
      }
    }
  }
  // acc[i][j][q]: row 16 i + r, column 16 j + 4 g + q of the wavefront's.  The outputs go
  // through the wavefront's own part of the stages, PB blocks of rows at a time, so that
  // it stores runs of RBY bytes of a row, 16 bytes a lane.  16-byte chunk c of a row sits
  // at slot c ^ (row % CPR).
  constexpr int ES = sizeof(OutT), RBY = 16 * FN * ES, CPR = RBY / 16;
  constexpr int ROOM = STAGE / 4, PB = 16 * FM * RBY <= ROOM ? FM : FM / 2;
  static_assert(PB * 16 * RBY <= ROOM && NW <= 8 && 64 % CPR == 0, "epilogue");
  const LmStage& own = wave < 4 ? s0 : s1;
  uint8_t* const reg = (wave & 3) < 2 ? own.w + (wave & 1) * ROOM
                       : NST > 2      ? own.x0 + (wave & 1) * ROOM
                                      : (wave & 1 ? own.x1 : own.x0);
  __syncthreads();  // the last stages have been read
  f32x4 bias[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int c = (wn * FN + j) * 16 + 4 * g;
    bias[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (p.bias != nullptr && c < cols) {
      const u32x2 raw = gld<u32x2>(static_cast<const uint16_t*>(p.bias) + n0 + c);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint16_t h = static_cast<uint16_t>(raw[q >> 1] >> (16 * (q & 1)));
        bias[j][q] = F16 ? static_cast<float>(__builtin_bit_cast(_Float16, h)) : bf16_bits_to_f32(h);
      }
    }
  }
  constexpr int RPI = 64 / CPR;  // rows per store
  const int pr = lane / CPR, pcol = lane % CPR;
  const int col = wn * 16 * FN + pcol * (16 / ES);
#pragma unroll
  for (int i0 = 0; i0 < FM; i0 += PB) {
#pragma unroll
    for (int i = i0; i < i0 + PB; ++i) {
      uint8_t* const blk = reg + (i - i0) * 16 * RBY;
      f32x4 v[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) v[j] = acc[i][j] + bias[j];
      // What is not finite in the banks, times the first piece, for its own rows (-0 elsewhere,
      // which adds nothing).  Rare, and so a plain loop over the ranks.
      if (__builtin_expect(odd, 0)) {
#pragma unroll 1
        for (int q = lane; q < 256 * FN; q += 64) {
          const i32x2 t = s_order[w0 + 16 * i + q / (16 * FN)];
          const int c = wn * 16 * FN + q % (16 * FN);
          float sum = -0.f;
          if (t.x >= 0 && t.y < p.L && c < cols) {
            const uint16_t* const bank = static_cast<const uint16_t*>(p.bank) + static_cast<int64_t>(t.y) * R * n;
            const uint16_t* const piece = p.pieces + static_cast<int64_t>(t.x) * 3 * RP;
#pragma unroll 1
            for (int rk = 0; rk < R; ++rk) {
              const float f = lm_half<F16>(gld<uint16_t>(
                  bank + (BT ? static_cast<int64_t>(rk) * n + n0 + c : static_cast<int64_t>(n0 + c) * R + rk)));
              if (!__builtin_isfinite(f)) sum += bf16_bits_to_f32(gld<uint16_t>(piece + rk)) * f;
            }
          }
          reinterpret_cast<uint16_t*>(blk)[q] = static_cast<uint16_t>(sum != sum ? 0x7fc0u : __float_as_uint(sum) >> 16);
        }
        asm volatile("" ::: "memory");  // LDS operations of one wavefront complete in order
        u32x2 c[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) c[j] = *reinterpret_cast<const u32x2*>(blk + (r * 16 * FN + 16 * j + 4 * g) * 2);
        asm volatile("" ::: "memory");
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[j][e] += bf16_bits_to_f32(c[j][e >> 1] >> (16 * (e & 1)) & 0xffffu);
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        uint8_t* const at = blk + r * RBY;
        if constexpr (ES == 4) {
          *reinterpret_cast<f32x4*>(at + ((4 * j + g) ^ (r % CPR)) * 16) = v[j];
        } else {
          typedef OutT t4 __attribute__((ext_vector_type(4)));
          *reinterpret_cast<t4*>(at + ((2 * j + (g >> 1)) ^ (r % CPR)) * 16 + (g & 1) * 8) =
              __builtin_convertvector(v[j], t4);
        }
      }
    }
    // LDS operations of one wavefront complete in order
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < PB * 16; q += RPI) {
      const int lrow = q + pr;
      const u32x4 v = *reinterpret_cast<const u32x4*>(reg + lrow * RBY + (pcol ^ (lrow % CPR)) * 16);
      const int row = s_order[(wm * FM + i0) * 16 + lrow].x;
      if (row >= 0 && col < cols)
        __builtin_nontemporal_store(
            v, (MI_GLOBAL u32x4*)(static_cast<OutT*>(p.out) + static_cast<int64_t>(row) * n + n0 + col));
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <bool F16, bool BT, int WM, int WN, int FM, int FN, int NST, typename OutT>
__global__ __launch_bounds__(64 * WM * WN)
    __attribute__((amdgpu_waves_per_eu(2, 2))) void lm_mm_kernel(LmMm p) {
  constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN, X = BM * 128, W = BN * 128;
  __shared__ i32x2 s_order[BM];
  LmPlace t = lm_place<BM, BN>(p, p.splits > 1 ? blockIdx.x % p.blocks : blockIdx.x);
  if (t.rows == 0) return;
  if (p.splits > 1) {
    const int split = blockIdx.x / p.blocks, all = t.steps;
    t.k0 = all * split / p.splits;
    t.steps = all * (split + 1) / p.splits - t.k0;
    p.out = static_cast<OutT*>(p.out) + static_cast<int64_t>(split) * p.T * p.n;
  }
  if constexpr (NST == 2) {
    static_assert(BM == BN, "the parts of a stage");
    __shared__ __attribute__((aligned(16))) uint8_t w0[W], w1[W], e0[X / 2], e1[X / 2], o0[X / 2], o1[X / 2];
    const LmStage s0{w0, e0, o0}, s1{w1, e1, o1};
    lm_tile<F16, BT, false, WM, WN, FM, FN, NST, OutT>(p, t, s0, s1, s0, s1, s_order);
  } else {
    __shared__ __attribute__((aligned(16))) uint8_t a0[X + W], a1[X + W], a2[X + W], a3[NST == 4 ? X + W : 16];
    const LmStage s0{a0 + X, a0, a0}, s1{a1 + X, a1, a1}, s2{a2 + X, a2, a2}, s3{a3 + (NST == 4 ? X : 0), a3, a3};
    lm_tile<F16, BT, false, WM, WN, FM, FN, NST, OutT>(p, t, s0, s1, s2, s3, s_order);
  }
}

// ---------------------------------------------------------------------------
// Few rows: no plan, and two launches.
//
//   parts   the dense product's 64 x 64 tiles, split along k until they fill the chip,
//           into fp32 partial sums; beside them, in workgroups of the same launch, v
//           (or u) in fp32 as it stands, a wavefront for some ranks of a row
//   finish  four columns of a row: the partial sums in order, the bias, and R fp32
//           fmas for the adapter; in the backward pass, workgroups of the same
//           launch sum gA and gB over the rows, which are few
//
// Bound by w's reads and a launch's start and end: 64 rows of 64 adapters, n = k = 4096, rank 16:
// 12 and 5 us (45 MB; a read of that takes 7).
// ---------------------------------------------------------------------------
struct LmSmall {
  LmMm mm;                // w, x of the dense product; out: the partial sums [S, T, n]
  const void* x;          // [T, ca] rows that meet a (dots)
  const void* go;         // [T, cb] rows that meet b (backward)
  const void* a;          // [L, R, ca]
  const void* b;          // [L, cb, R]
  const int32_t* ids;
  const float* scale;
  const float* act_in;    // backward: the forward's act, or null
  float* v;               // [T, R] x a^T (backward: where act_in is null)
  float* u;               // [T, R] go b (backward)
  float* act;             // forward: v goes here too, or null
  const void* bias;
  void* out;              // [T, mm.n]
  void *ga, *gb;          // backward, or null
  int T, ca, cb, L, R;
  int splits, tiles, gemm, dots, fin;  // workgroups
};

template <bool F16>
__device__ __forceinline__ void lm_unpack(u32x4 q, float (&o)[8]) {
  if constexpr (F16) {
    const f16x8 h = __builtin_bit_cast(f16x8, q);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = static_cast<float>(h[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float(q[i] << 16);
      o[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ float lm_wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// ranks r0 .. r0 + 3 of x[t] a[l]^T
template <bool F16>
__device__ __forceinline__ void lm_dot_a(const LmSmall& p, int t, int r0) {
  const int lane = threadIdx.x & 63, l = gld<int32_t>(p.ids + t), k = p.ca;
  const bool none = l < 0 || l >= p.L;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  if (!none) {
    const uint16_t* const x = static_cast<const uint16_t*>(p.x) + static_cast<int64_t>(t) * k;
    const uint16_t* const a = static_cast<const uint16_t*>(p.a) + (static_cast<int64_t>(l) * p.R + r0) * k;
#pragma unroll 4
    for (int c = lane * 8; c < k; c += 512) {
      u32x4 qa[4];
      const u32x4 qx = gld<u32x4>(x + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) qa[i] = gld<u32x4>(a + static_cast<int64_t>(i) * k + c);
      float fx[8];
      lm_unpack<F16>(qx, fx);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float fa[8];
        lm_unpack<F16>(qa[i], fa);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[i] = __builtin_fmaf(fx[e], fa[e], sum[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[i] = lm_wave_sum(sum[i]);
  if (lane == 0) {
    const f32x4 v = {sum[0], sum[1], sum[2], sum[3]};
    const int64_t at = static_cast<int64_t>(t) * p.R + r0;
    gst<f32x4>(p.v + at, v);
    if (p.act != nullptr) gst<f32x4>(p.act + at, v);
  }
}

// ranks r0 .. r0 + 7 of go[t] b[l]: a lane has its own rows of b
template <bool F16>
__device__ __forceinline__ void lm_dot_b(const LmSmall& p, int t, int r0) {
  const int lane = threadIdx.x & 63, l = gld<int32_t>(p.ids + t);
  const bool none = l < 0 || l >= p.L;
  float sum[8] = {};
  if (!none) {
    const uint16_t* const go = static_cast<const uint16_t*>(p.go) + static_cast<int64_t>(t) * p.cb;
    const uint16_t* const b = static_cast<const uint16_t*>(p.b) + static_cast<int64_t>(l) * p.cb * p.R + r0;
#pragma unroll 8
    for (int c = lane; c < p.cb; c += 64) {
      const uint16_t h = gld<uint16_t>(go + c);
      float fb[8];
      lm_unpack<F16>(gld<u32x4>(b + static_cast<int64_t>(c) * p.R), fb);
      const float f = lm_half<F16>(h);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = __builtin_fmaf(f, fb[e], sum[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = lm_wave_sum(sum[e]);
  if (lane == 0) {
    float* const at = p.u + static_cast<int64_t>(t) * p.R + r0;
    gst<f32x4>(at, f32x4{sum[0], sum[1], sum[2], sum[3]});
    gst<f32x4>(at + 4, f32x4{sum[4], sum[5], sum[6], sum[7]});
  }
}

template <bool F16, bool BT>
__global__ __launch_bounds__(256) void lm_parts_kernel(LmSmall p) {
  constexpr int STAGE = 128 * 128;
  __shared__ __attribute__((aligned(16))) uint8_t s0[STAGE], s1[STAGE], s2[STAGE], s3[STAGE];
  __shared__ i32x2 s_order[64];
  const int block = blockIdx.x;
  if (block < p.gemm) {
    const int split = block / p.tiles, tile = block % p.tiles;
    const int mt = (p.T + 63) / 64, all = (p.mm.k + LM_BK - 1) / LM_BK;
    const int k0 = all * split / p.splits, k1 = all * (split + 1) / p.splits;
    auto stage = [](uint8_t* s) { return LmStage{s + STAGE / 2, s, s}; };
    LmMm mm = p.mm;
    mm.out = static_cast<float*>(p.mm.out) + static_cast<int64_t>(split) * p.T * mm.n;
    const int m0 = tile % mt * 64, n0 = tile / mt * 64;
    // Long parts of few row blocks start at their panel's own step: where k is a multiple of a
    // large power of two, tiles at the same step ask for lines that lie in a few memory
    // channels.  us, without and with it: n 8192, k 4096, 128 rows 44 and 30; n 2048, k 8192,
    // 256 rows 45 and 36; n = k = 4096, 192 rows 26 and 27, 256 rows 31 and 31; with six row
    // blocks and more (n 2048, k 8192, 384 rows) 45 and 47, with 32 steps (128 rows, n = k =
    // 4096) 21 and 21.
    const int first = mt <= 4 && k1 - k0 >= 40 ? tile / mt % (k1 - k0) : 0;
    lm_tile<F16, BT, true, 2, 2, 2, 2, 4, float>(
        mm, {m0, n0, min(p.T - m0, 64), min(mm.n - n0, 64), k0, k1 - k0, first}, stage(s0), stage(s1),
        stage(s2), stage(s3), s_order);
    return;
  }
  const int wave = (block - p.gemm) * 4 + (threadIdx.x >> 6), waves = p.dots * 4;
  // backward: u first, then v where it is not given
  const int nu = p.u != nullptr ? p.T * (p.R / 8) : 0, nv = p.v != nullptr ? p.T * (p.R / 4) : 0;
  for (int i = wave; i < nu + nv; i += waves) {
    if (i < nu) lm_dot_b<F16>(p, i / (p.R / 8), i % (p.R / 8) * 8);
    else lm_dot_a<F16>(p, (i - nu) / (p.R / 4), (i - nu) % (p.R / 4) * 4);
  }
}

// gA: 8 ranks and 512 columns of x of an adapter, a lane 8 x 8 of them (OTHER: gB).  The
// wavefronts take every fourth row each and add their sums in order.
constexpr int SG_COLS = 512;
template <bool F16, bool OTHER, typename OutT>
__device__ __forceinline__ void lm_small_grad(const LmSmall& p, int l, int r0, int c0, f32x4* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int C = OTHER ? p.cb : p.ca, at_c = c0 + lane * 8, c = min(at_c, C - 8);
  const uint16_t* const x = static_cast<const uint16_t*>(OTHER ? p.go : p.x) + c;
  const float* const f = (OTHER ? (p.act_in != nullptr ? p.act_in : p.v) : p.u) + r0;
  f32x4 acc[8][2];  // [rank][columns], OTHER: [column][ranks]
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  // the adapter's rows among 64 at a time, four rows' loads in flight
  for (int t0 = 0; t0 < p.T; t0 += 64) {
    const int at = t0 + lane;
    uint64_t own = __ballot(at < p.T && gld<int32_t>(p.ids + min(at, p.T - 1)) == l) & (0x1111111111111111ull << wave);
    while (own != 0) {
      u32x4 qx[4];
      f32x4 f0[4], f1[4];
      int n = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (own == 0) break;
        const int64_t t = t0 + __builtin_ctzll(own);
        own &= own - 1;
        qx[q] = gld<u32x4>(x + t * C);
        f0[q] = gld<f32x4>(f + t * p.R);
        f1[q] = gld<f32x4>(f + t * p.R + 4);
        ++n;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q >= n) break;
        float xs[8];
        lm_unpack<F16>(qx[q], xs);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int r = OTHER ? e : i;
            const float rank = r < 4 ? f0[q][r & 3] : f1[q][r & 3];
            acc[i][e >> 2][e & 3] = __builtin_fmaf(rank, xs[OTHER ? i : e], acc[i][e >> 2][e & 3]);
          }
      }
    }
  }
  const float s = p.scale != nullptr ? gld<float>(p.scale + l) : 1.f;
  OutT* const out = static_cast<OutT*>(OTHER ? p.gb : p.ga) + static_cast<int64_t>(l) * p.R * C;
  // half of the sums at a time; wavefront w then has those of index 4 half + w
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) red[((wave * 4 + i) * 2 + e) * 64 + lane] = acc[4 * half + i][e];
    __syncthreads();
    f32x4 v[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      v[e] = red[(wave * 2 + e) * 64 + lane];
#pragma unroll
      for (int w = 1; w < 4; ++w) v[e] += red[((w * 4 + wave) * 2 + e) * 64 + lane];
      v[e] *= s;
    }
    if (at_c >= C) continue;
    const int i = 4 * half + wave;
    OutT* const at = OTHER ? out + static_cast<int64_t>(c + i) * p.R + r0 : out + static_cast<int64_t>(r0 + i) * C + c;
    if constexpr (sizeof(OutT) == 4) {
      gst<f32x4>(at, v[0]);
      gst<f32x4>(at + 4, v[1]);
    } else {
      typedef OutT t8 __attribute__((ext_vector_type(8)));
      t8 o;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = static_cast<OutT>(v[e >> 2][e & 3]);
      gst<u32x4>(at, __builtin_bit_cast(u32x4, o));
    }
  }
}

// BT (backward): the adapter's part is s u a, else s v b^T
template <bool F16, bool BT, typename OutT, typename GradT>
__global__ __launch_bounds__(256) void lm_finish_kernel(LmSmall p) {
  const int n = p.mm.n, R = p.R;
  if constexpr (BT) {
    if (static_cast<int>(blockIdx.x) >= p.fin) {
      __shared__ __attribute__((aligned(16))) f32x4 red[4 * 4 * 2 * 64];
      const int pa = (p.ca + SG_COLS - 1) / SG_COLS, pb = (p.cb + SG_COLS - 1) / SG_COLS, r8 = R / 8;
      int i = blockIdx.x - p.fin;
      const int panel = i % (pa + pb);
      i /= pa + pb;
      if (panel < pa) lm_small_grad<F16, false, GradT>(p, i / r8, i % r8 * 8, panel * SG_COLS, red);
      else lm_small_grad<F16, true, GradT>(p, i / r8, i % r8 * 8, (panel - pa) * SG_COLS, red);
      return;
    }
  }
  const uint32_t quad = blockIdx.x * 256 + threadIdx.x, per = n / 4;
  const int t = quad / per, c = quad % per * 4;
  if (t >= p.T) return;
  const int l = gld<int32_t>(p.ids + t);
  const bool has = l >= 0 && l < p.L;
  const float* const parts = static_cast<const float*>(p.mm.out) + static_cast<int64_t>(t) * n + c;
  f32x4 sum = gld<f32x4>(parts);
#pragma unroll 4
  for (int i = 1; i < p.splits; ++i) sum += gld<f32x4>(parts + static_cast<int64_t>(i) * p.T * n);
  if (has) {
    const float* const f = (BT ? p.u : p.v) + static_cast<int64_t>(t) * R;
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
    if constexpr (BT) {
      const uint16_t* const bank = static_cast<const uint16_t*>(p.a) + static_cast<int64_t>(l) * R * n + c;
#pragma unroll 8
      for (int r = 0; r < R; ++r) {
        const u32x2 q = gld<u32x2>(bank + static_cast<int64_t>(r) * n);
        const float u = gld<float>(f + r);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          d[e] = __builtin_fmaf(u, lm_half<F16>(static_cast<uint16_t>(q[e >> 1] >> (16 * (e & 1)))), d[e]);
      }
    } else {
      const uint16_t* const bank = static_cast<const uint16_t*>(p.b) + (static_cast<int64_t>(l) * n + c) * R;
#pragma unroll 2
      for (int r = 0; r < R; r += 8) {
        const f32x4 f0 = gld<f32x4>(f + r), f1 = gld<f32x4>(f + r + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float b[8];
          lm_unpack<F16>(gld<u32x4>(bank + static_cast<int64_t>(e) * R + r), b);
#pragma unroll
          for (int i = 0; i < 8; ++i) d[e] = __builtin_fmaf(i < 4 ? f0[i & 3] : f1[i & 3], b[i], d[e]);
        }
      }
    }
    const float s = p.scale != nullptr ? gld<float>(p.scale + l) : 1.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(s, d[e], sum[e]);
  }
  if (p.bias != nullptr) {
    const u32x2 q = gld<u32x2>(static_cast<const uint16_t*>(p.bias) + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += lm_half<F16>(static_cast<uint16_t>(q[e >> 1] >> (16 * (e & 1))));
  }
  OutT* const o = static_cast<OutT*>(p.out) + static_cast<int64_t>(t) * n + c;
  if constexpr (sizeof(OutT) == 4) {
    gst<f32x4>(o, sum);
  } else {
    typedef OutT t4 __attribute__((ext_vector_type(4)));
    gst<u32x2>(o, __builtin_bit_cast(u32x2, __builtin_convertvector(sum, t4)));
  }
}

// ---------------------------------------------------------------------------
// One row, rank 32 at most: one launch, bound by the reads of w.  A wavefront has ONE_C rows
// of w and streams them whole lines at a time (four rows instead of two: n = k = 4096, rank
// 16: 14.1 us for 11.3); every workgroup computes v again beside them, its wavefronts RW ranks
// each (their loads hit in the L2: 128 KB a workgroup at rank 16, k 4096).  Taken where that
// costs less than a second launch; us in one launch and two: n = k = 4096, rank 16, 11.3 and
// 14.1; n 1024, rank 32, k 4096 11.6 and 13.1, k 8192 17.8 and 16.6; n 64, rank 32, k 16384 28
// and 18; n 4096, rank 32, k 6144 16.8 and 20.9, k 28672 61 and 62.
// ---------------------------------------------------------------------------
constexpr int ONE_W = 8, ONE_C = 2;  // wavefronts, rows of w for each
template <bool F16, int RW, typename OutT>
__global__ __launch_bounds__(64 * ONE_W) void lm_one_kernel(LmSmall p) {
  __shared__ float s_v[ONE_W * RW];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k = p.ca, n = p.cb, R = p.R;
  const int n0 = (blockIdx.x * ONE_W + wave) * ONE_C, r0 = wave * RW;
  const int l = __builtin_amdgcn_readfirstlane(gld<int32_t>(p.ids));
  const bool has = l >= 0 && l < p.L;
  const uint16_t* const x = static_cast<const uint16_t*>(p.x);
  const uint16_t* const w = static_cast<const uint16_t*>(p.mm.w);
  const uint16_t* const a = static_cast<const uint16_t*>(p.a) + static_cast<int64_t>(has ? l : 0) * R * k;
  float sum[ONE_C] = {}, v[RW] = {};
#pragma unroll 4
  for (int c = lane * 8; c < k; c += 512) {
    u32x4 qw[ONE_C], qa[RW];
    const u32x4 qx = gld<u32x4>(x + c);
#pragma unroll
    for (int i = 0; i < ONE_C; ++i) qw[i] = gld_nt<u32x4>(w + static_cast<int64_t>(min(n0 + i, n - 1)) * k + c);
    // rows past the ranks are read again, and not used
    if (has)
#pragma unroll
      for (int i = 0; i < RW; ++i) qa[i] = gld<u32x4>(a + static_cast<int64_t>(min(r0 + i, R - 1)) * k + c);
    float fx[8], f[8];
    lm_unpack<F16>(qx, fx);
#pragma unroll
    for (int i = 0; i < ONE_C; ++i) {
      lm_unpack<F16>(qw[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[i] = __builtin_fmaf(fx[e], f[e], sum[i]);
    }
    if (has)
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        lm_unpack<F16>(qa[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i] = __builtin_fmaf(fx[e], f[e], v[i]);
      }
  }
  // lane r has rank r of the wavefront's rows of b
  float b[ONE_C];
  const uint16_t* const bank = static_cast<const uint16_t*>(p.b) + static_cast<int64_t>(has ? l : 0) * n * R;
#pragma unroll
  for (int i = 0; i < ONE_C; ++i)
    b[i] = has && lane < R ? lm_half<F16>(gld<uint16_t>(bank + static_cast<int64_t>(min(n0 + i, n - 1)) * R + lane)) : 0.f;
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const float all = lm_wave_sum(v[i]);
    if (lane == 0) s_v[r0 + i] = has ? all : 0.f;
    if (p.act != nullptr && blockIdx.x == 0 && lane == 0 && r0 + i < R) gst<float>(p.act + r0 + i, has ? all : 0.f);
  }
  __syncthreads();
  const float s = has && p.scale != nullptr ? gld<float>(p.scale + l) : 1.f;
  const float vr = lane < R ? s_v[lane] * s : 0.f;
#pragma unroll
  for (int i = 0; i < ONE_C; ++i) {
    // a rank's product is a term of the wavefront's sum, as the columns' are
    float all = lm_wave_sum(has ? __builtin_fmaf(vr, b[i], sum[i]) : sum[i]);
    if (lane != 0 || n0 + i >= n) continue;
    if (p.bias != nullptr) all += lm_half<F16>(gld<uint16_t>(static_cast<const uint16_t*>(p.bias) + n0 + i));
    gst<OutT>(static_cast<OutT*>(p.out) + n0 + i, static_cast<OutT>(all));
  }
}

// ---------------------------------------------------------------------------
// grads: for a chunk of an adapter's rows, 128 columns of x (or go) and 16 NB ranks,
//   ROWS == false: ga[l, r, c] = sum_t u[t, r] x[t, c]
//   ROWS == true:  gb[l, c, r] = sum_t v[t, r] go[t, c]
// A step is 64 rows: those of x, and 64 slots of the transposed pieces, both by loads
// straight into LDS; x is read down its columns.  A wavefront has 32 columns.  Bound by the
// reads of x and go, once for all ranks up to 64: 8192 rows, n = k = 4096, rank 16: 29 us (134 MB:
// 4.7 TB/s; the L2s fetch 148) and 5 for the partial sums.
// ---------------------------------------------------------------------------
struct LmGrad {
  const void* x;             // [T, C]
  const uint16_t* pieces_t;  // [3 RP, slots]
  LmPlan plan;
  float* part;               // [places, R, C] (ROWS: [places, C, R])
  void* out;                 // [L, R, C] (ROWS: [L, C, R])
  int C, R, RP, slots;
};

constexpr int GR_BN = 128, GR_BK = 64, GR_X = GR_BK * GR_BN * 2;
constexpr int GR_ROWS = 2048;  // rows of a chunk at most
template <int NB>
struct LmGradShape {
  static constexpr int PI = (6 * NB + 3) / 4;   // a wavefront's loads of pieces: 8 rows of 64 slots each
  static constexpr int BYTES = GR_X + PI * 4096;
  static constexpr int ST = NB == 2 ? 2 : 3;    // stages; with two a second workgroup fits
};

template <bool F16, bool ROWS, int NB, typename OutT>
__device__ __forceinline__ void lm_grad(const LmGrad& a, uint8_t* st0, uint8_t* st1, uint8_t* st2,
                                        const int* s_rows, i32x4 ch, int c0, int rank0) {
  using Shape = LmGradShape<NB>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4, lr = lane >> 3;
  int C = a.C, RP = a.RP, s0 = ch.y * LM_ITEM, n = ch.z * LM_ITEM;  // slots
  const int R = a.R, KT = (n + GR_BK - 1) / GR_BK;
  constexpr int CPW = GR_BN / 8, NX = GR_X / 1024 / 4, PI = Shape::PI, ST = Shape::ST;
  const uint16_t* const x = static_cast<const uint16_t*>(a.x);
  const int chunk = (lane & 7) ^ lr;
  auto load = [&](uint8_t* st, int kt) {
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int at = (4 * i + wave) * 64 + lane, row = at / CPW, c = at % CPW;
      const int col = c0 + (((c >> 1) ^ lm_tswz<GR_BN>(row)) * 2 + (c & 1)) * 8;
      const int t = kt * GR_BK + row < n ? s_rows[kt * GR_BK + row] : -1;
      const uint16_t* src = t >= 0 && col < C ? x + static_cast<int64_t>(t) * C + col : a.plan.zeros;
      __builtin_amdgcn_global_load_lds((const MI_GLOBAL void*)(src), lm_lds(st + (4 * i + wave) * 1024), 16, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < PI; ++i) {
      // rows 8 (PI wave + i) .. of [rank block][piece][16 ranks]
      const int row = 8 * (PI * wave + i) + lr, b = row / 48, c = row / 16 % 3, rk = rank0 + 16 * b + (row & 15);
      const int slot = kt * GR_BK + (chunk ^ ((row >> 3) & 1)) * 8;
      const uint16_t* src = b < NB && rk < RP && slot < n
                                ? a.pieces_t + (static_cast<int64_t>(c) * RP + rk) * a.slots + s0 + slot : a.plan.zeros;
      __builtin_amdgcn_global_load_lds((const MI_GLOBAL void*)(src), lm_lds(st + GR_X + (PI * wave + i) * 1024), 16, 0, 0);
    }
  };
  f32x4 acc[NB][2];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[b][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // apart: what is not finite in x taken on its own
  auto add = [&](auto apart, const uint8_t* st) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int ck = (((g & 1) << 1) | (g >> 1)) + 4 * h;  // this lane's 8 slots
      u32x4 fx[2], fl[2];
      LmOdd part[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = 8 * ck + (r >> 2);
        const uint8_t* at = st + row * (GR_BN * 2) + ((wave * 2 + j) ^ lm_tswz<GR_BN>(row)) * 32 + (r & 3) * 8;
        fx[j] = lm_column(at, at + 4 * GR_BN * 2);
        if constexpr (F16) lm_split(fx[j], fx[j], fl[j]);
        if constexpr (apart.value) {
          part[j] = lm_part(fx[j]);
          fx[j] = part[j].rest;
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          const u32x4 fp = *reinterpret_cast<const u32x4*>(st + GR_X + (b * 3 + c) * 2048 + r * 128 + (ck ^ lm_swz(r)) * 16);
          auto mfma = [&](u32x4 x, f32x4 to) { return ROWS ? lm_mfma<false>(fp, x, to) : lm_mfma<false>(x, fp, to); };
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            acc[b][j] = mfma(fx[j], acc[b][j]);
            if constexpr (F16) {
              if (c < 2) acc[b][j] = mfma(fl[j], acc[b][j]);
            }
            if constexpr (apart.value) {
              if (c == 0) acc[b][j] = mfma(part[j].odd, acc[b][j]);
            }
          }
        }
    }
  };
  // a step past the last loads zeros
  constexpr int NI = NX + PI;
  const int rounds = KT / ST * ST;
  auto all = [&](auto apart) {
    load(st0, 0);
    if constexpr (ST == 3) load(st1, 1);
    auto step = [&](const uint8_t* st, uint8_t* to, int kt) {
      lm_wait_barrier<(ST - 2) * NI>();
      load(to, kt + ST - 1);
      add(apart, st);
    };
    // whole rounds of the stages, then the rest
    if constexpr (ST == 3) {
      for (int kt = 0; kt < rounds; kt += ST) {
        step(st0, st2, kt);
        step(st1, st0, kt + 1);
        step(st2, st1, kt + 2);
      }
      if (KT - rounds >= 1) {
        step(st0, st2, rounds);
        if (KT - rounds == 2) step(st1, st0, rounds + 1);
      }
    } else {
      for (int kt = 0; kt < rounds; kt += ST) {
        step(st0, st1, kt);
        step(st1, st0, kt + 1);
      }
      if (KT - rounds == 1) step(st0, st1, rounds);
    }
    lm_wait_barrier<0>();  // no load writes to LDS after the end
  };
  all(std::false_type{});
  // Where a wavefront's sums are not all finite, they are taken again with what is not finite in x
  // apart.  (A look at the values of x instead: 31 us for 29.)  The vote lies in a stage: more LDS
  // would leave a CU one workgroup.
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int j = 0; j < 2; ++j) sum += acc[b][j] * 0.f;
  const bool mine = __any(!(sum[0] + sum[1] + sum[2] + sum[3] == 0.f));
  int* const vote = reinterpret_cast<int*>(st0);
  if (lane == 0) vote[wave] = mine;
  __syncthreads();
  if (__builtin_expect(__builtin_amdgcn_readfirstlane(vote[0] | vote[1] | vote[2] | vote[3]), 0)) {
    lm_wait_barrier<0>();  // all have read the votes
    // nothing that the second pass derives from these is kept over the first
    asm volatile("" : "+s"(C), "+s"(RP), "+s"(s0), "+s"(n), "+s"(c0), "+s"(rank0));
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[b][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    all(std::true_type{});
  }
  // four ranks of column r (ROWS), or four columns of rank r
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = c0 + wave * 32 + 16 * j + (ROWS ? r : 4 * g);
      const int rk = rank0 + 16 * b + (ROWS ? 4 * g : r);
      if (col >= C || rk >= R) continue;
      const int64_t in = ROWS ? static_cast<int64_t>(col) * R + rk : static_cast<int64_t>(rk) * C + col;
      const int64_t size = static_cast<int64_t>(R) * C;
      if (ch.w >= 0) {
        gst<f32x4>(a.part + ch.w * size + in, acc[b][j]);
      } else if constexpr (sizeof(OutT) == 4) {
        gst<f32x4>(static_cast<float*>(a.out) + ch.x * size + in, acc[b][j]);
      } else {
        typedef OutT t4 __attribute__((ext_vector_type(4)));
        gst<u32x2>(static_cast<OutT*>(a.out) + ch.x * size + in,
                   __builtin_bit_cast(u32x2, __builtin_convertvector(acc[b][j], t4)));
      }
    }
}

template <bool F16, int NB, typename OutT>
__global__ __launch_bounds__(256) void lm_grad_kernel(LmGrad ga, LmGrad gb) {
  constexpr int SIZE = LmGradShape<NB>::BYTES;
  __shared__ __attribute__((aligned(16))) uint8_t st0[SIZE], st1[SIZE], st2[LmGradShape<NB>::ST == 3 ? SIZE : 16];
  __shared__ int s_rows[GR_ROWS];
  const int chunk = blockIdx.y;
  if (chunk >= gld<int>(ga.plan.totals + 1)) return;
  i32x4 ch = gld<i32x4>(ga.plan.chunks + chunk);
#pragma unroll
  for (int i = 0; i < 4; ++i) ch[i] = __builtin_amdgcn_readfirstlane(ch[i]);
  for (int i = threadIdx.x; i < ch.z * LM_ITEM; i += 256) s_rows[i] = gld<int>(ga.plan.slot_row + ch.y * LM_ITEM + i);
  __syncthreads();
  const int pa = (ga.C + GR_BN - 1) / GR_BN;
  const int rank0 = blockIdx.z * 16 * NB;
  if (static_cast<int>(blockIdx.x) < pa)
    lm_grad<F16, false, NB, OutT>(ga, st0, st1, st2, s_rows, ch, blockIdx.x * GR_BN, rank0);
  else
    lm_grad<F16, true, NB, OutT>(gb, st0, st1, st2, s_rows, ch, (blockIdx.x - pa) * GR_BN, rank0);
}

// four values a thread, gA's and then gB's, of an adapter with partial sums
template <typename OutT>
__global__ __launch_bounds__(256) void lm_reduce_kernel(LmGrad ga, LmGrad gb) {
  const i32x4 span = gld<i32x4>(ga.plan.spans + blockIdx.y);
  if (span.z < 0) return;
  const int64_t na = static_cast<int64_t>(ga.R) * ga.C, nb = static_cast<int64_t>(gb.R) * gb.C;
  int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= na + nb) return;
  const bool second = i >= na;
  const int64_t size = second ? nb : na;
  if (second) i -= na;
  const float* const part = (second ? gb.part : ga.part) + span.z * size + i;
  f32x4 v = gld<f32x4>(part);
#pragma unroll 8
  for (int c = 1; c < span.y; ++c) v += gld<f32x4>(part + c * size);
  void* const out = second ? gb.out : ga.out;
  if constexpr (sizeof(OutT) == 4) {
    gst<f32x4>(static_cast<float*>(out) + blockIdx.y * size + i, v);
  } else {
    typedef OutT t4 __attribute__((ext_vector_type(4)));
    gst<u32x2>(static_cast<OutT*>(out) + blockIdx.y * size + i,
               __builtin_bit_cast(u32x2, __builtin_convertvector(v, t4)));
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
struct LmSizes {
  int64_t T, N, K, L, R;
  int64_t rp() const { return (R + 15) / 16 * 16; }
  // rows of one pass: a row's place in x or go is a 31-bit byte offset
  int64_t pass() const {
    const int64_t wide = N > K ? N : K, fit = ((1LL << 31) - 1) / (2 * wide) & ~255LL;
    const int64_t pieces = ((1LL << 31) - 1) / (6 * rp()) & ~255LL;  // and in the pieces
    int64_t most = fit < (1LL << 22) ? fit : 1LL << 22;
    if (pieces < most) most = pieces;
    return T < most ? T : most;
  }
  static int64_t items(int64_t t, int64_t l) { return t / LM_ITEM + (l + 1 < t ? l + 1 : t) + 1; }
  // Items of a chunk: as many as leave 512 workgroups of the gradients' kernel, but 128 rows
  // at least and 512 at most; of very many rows a 32nd of them up to GR_ROWS, which keeps the
  // partial sums few
  int64_t chunk_items() const {
    const int64_t panels = (K + GR_BN - 1) / GR_BN + (N + GR_BN - 1) / GR_BN;
    int64_t rows = T * panels / 512;
    if (rows > 512) rows = T / 32 < 512 ? 512 : T / 32;
    rows = rows < 128 ? 128 : rows > GR_ROWS ? GR_ROWS : rows;
    return rows / LM_ITEM;
  }
  int64_t chunks() const { return L + items(T, L) / chunk_items() + 1; }
  // those of adapters that have several: each but an adapter's last is full
  int64_t places() const { return 2 * (items(T, L) / chunk_items()) + 2; }
};

// Splits of the k axis of few rows' tiles: 64 x 64 tiles on 256 CUs, 8 steps each at least.
int lm_splits(int64_t T, int64_t n, int64_t k) {
  const int64_t tiles = (T + 63) / 64 * ((n + 63) / 64), steps = (k + LM_BK - 1) / LM_BK;
  int64_t s = 256 / tiles;
  if (s > steps / 8) s = steps / 8;
  return static_cast<int>(s < 1 ? 1 : s);
}

// The same of many rows and a narrow result, 16 steps at least: the parts are written and read
// once more.  us a call, unsplit and in 2, 3 and 4: 3817 rows, n 96, k 4760 (120 tiles, 75 steps)
// 46, 40, 45, 42; 4096 rows, n 64, k 8192 (64, 128) 51, 44, 43, 43; 1100 rows, n 256, k 4096 (72, 64)
// 30, 28, 28, 31; 2100 rows, n 72, k 2056 (66, 33) 28, 27, 26, 28; 2000 rows, n 128, k 2048 (64, 32)
// 24, 25, 25, 25; with more tiles 1100 rows, n 512, k 8192 (144, 128) 46, 50, 44, 48; 1500 rows, n
// 576, k 4096 (216, 64) 31, 35, 37, 39.
int lm_wide_splits(int64_t T, int64_t n, int64_t k) {
  const int64_t tiles = (T + 63) / 64 * ((n + 63) / 64), steps = (k + LM_BK - 1) / LM_BK;
  int64_t s = 256 / tiles;
  if (s > steps / 16) s = steps / 16;
  return static_cast<int>(s < 1 ? 1 : s);
}

// Few rows: as long as the fmas of the finish, and in the backward pass of the adapters'
// gradients, cost less than the plan and the launches that the MFMAs need.  us, few rows and
// many, forward: n = k = 4096, rank 16, 256 rows 31 and 35, 320 rows 46 and 39; rank 64, 96 rows
// 31 and 33, 192 rows 44 and 36; n 1024, k 2048, rank 16, 1024 rows 22 and 29; n 512, k 4096,
// rank 32, 768 rows (rows * k * rank: 100M) 29 and 31; n 256, k 4096, rank 64, 400 rows (104M)
// 30 and 29; n 1024, k 8192, rank 32, 400 rows 43 and 40; n 8192, k 4096, rank 16, 128
// rows 30 and 36; past the balance n 2048, k 8192, rank 16, 480 rows 52 and 49.  With the backward pass: n = k
// = 4096, rank 16, 256 rows 69 and 80; rank 64, 128 rows (84M) 71 and 84, 192 rows (126M) 96
// and 87; n 1024, k 2048, rank 16, 256 rows 31 and 52.
// Up to 32 rows the adapters decide, which the call cannot see: many rows pay for each by itself.
// Forward, k 4096: n 4096, rank 16, 32 rows of one adapter 14 and 26, of 32 adapters 15 and 45;
// rank 256, one 38 and 30, 32 adapters 51 and 176; n 28672, rank 64, one 62 and 49, 32 adapters
// 109 and 107; rank 256, one 127 and 57, 32 adapters 295 and 243, 8 rows of 8 adapters 88 and 106.
// Backward alone: n 28672, rank 256, one 156 and 153, 32 adapters 511 and 1181.
bool lm_small(const LmSizes& s, bool backward) {
  if (s.T <= 32) return true;
  if (backward) return s.T <= 256 && s.T * (s.N + s.K) * (s.R + 16) <= 100000000;
  return s.T <= 1024 && s.T * s.N * (s.R + 16) <= 36000000 && s.T * s.K * s.R <= 100000000;
}

struct LmCarve {
  uint8_t* at;
  size_t used = 0;
  template <typename T>
  T* take(int64_t n) {
    T* const p = reinterpret_cast<T*>(at + used);
    used += (static_cast<size_t>(n) * sizeof(T) + 255) & ~static_cast<size_t>(255);
    return at == nullptr ? nullptr : p;
  }
};

struct LmSpace {
  LmPlan plan;
  uint16_t *pieces, *ut, *vt;
  float *act, *part_a, *part_b;
  float *v, *u, *parts;  // few rows
  size_t bytes;
};

// what of many rows' space is not proportional to them
struct LmMany {
  int64_t parts;           // of a split k axis
  int64_t chunks, places;  // of the gradients
};

// fp32 partial sums of a pass of `rows`; few where the k axis is not split
int64_t lm_parts(int64_t rows, int64_t on, int64_t in) {
  const int64_t sp = rows > 0 ? lm_wide_splits(rows, on, in) : 1;
  return sp > 1 ? sp * rows * on : 0;
}

LmSpace lm_space_many(const LmSizes& s, bool backward, const LmMany& m, void* base) {
  LmCarve c{static_cast<uint8_t*>(base)};
  LmSpace o{};
  const int64_t items = LmSizes::items(s.T, s.L);
  o.plan.rank = c.take<int>(s.T);
  o.plan.counts = c.take<int>(64 * (s.L + 1));
  o.plan.order = c.take<i32x2>(s.T);
  o.plan.item_id = c.take<int>(items);
  o.plan.slot_row = c.take<int>(items * LM_ITEM);
  o.plan.chunks = c.take<i32x4>(m.chunks);
  o.plan.spans = c.take<i32x4>(s.L);
  o.plan.totals = c.take<int>(4);
  o.plan.zeros = c.take<uint16_t>(8);
  o.pieces = c.take<uint16_t>(s.T * 3 * s.rp());
  o.parts = c.take<float>(m.parts);
  if (backward) {
    o.ut = c.take<uint16_t>(items * LM_ITEM * 3 * s.rp());
    o.vt = c.take<uint16_t>(items * LM_ITEM * 3 * s.rp());
    o.act = c.take<float>(s.T * s.R);
    o.part_a = c.take<float>(m.places * s.R * s.K);
    o.part_b = c.take<float>(m.places * s.R * s.N);
  }
  o.bytes = c.used;
  return o;
}

LmSpace lm_space(const LmSizes& s, bool backward, void* base) {
  if (s.T > 0 && lm_small(s, backward)) {
    LmCarve c{static_cast<uint8_t*>(base)};
    LmSpace o{};
    o.v = c.take<float>(s.T * s.R);
    o.u = c.take<float>(backward ? s.T * s.R : 0);
    o.parts = c.take<float>(s.T * (backward ? lm_splits(s.T, s.K, s.N) * s.K : lm_splits(s.T, s.N, s.K) * s.N));
    o.bytes = c.used;
    return o;
  }
  // the passes over the rows: all of one size but the last, which may have more splits
  const int64_t pass = s.T > 0 ? s.pass() : 1, on = backward ? s.K : s.N, in = backward ? s.N : s.K;
  const int64_t parts = lm_parts(pass, on, in), rest = lm_parts(s.T % pass, on, in);
  return lm_space_many(s, backward, {parts > rest ? parts : rest, s.chunks(), s.places()}, base);
}

// Bytes that are enough for s.T rows and for every smaller number: a caller has one workspace
// for its largest batch.  The need itself falls where the way of computing changes.
size_t lm_space_upto(const LmSizes& s, bool backward) {
  LmSizes a = s;
  size_t most = 0;
  auto also = [&](size_t bytes) { most = bytes > most ? bytes : most; };
  a.T = 0;
  if (backward) also(lm_space(a, backward, nullptr).bytes);
  // few rows: up to the end of every 64, whose splits are the same, and the last of them
  for (int64_t t = 0; t < s.T; t += 64) {
    a.T = t + 64 < s.T ? t + 64 : s.T;
    while (a.T > t && !lm_small(a, backward)) --a.T;
    if (a.T == t) break;
    also(lm_space(a, backward, nullptr).bytes);
  }
  a.T = s.T;
  if (s.T == 0 || lm_small(a, backward)) return most;
  // many: the proportional part at the most rows, the rest each where it is the largest
  const int64_t on = backward ? s.K : s.N, in = backward ? s.N : s.K;
  LmMany m{lm_parts(s.pass(), on, in), s.chunks(), s.places()};
  for (int64_t t = 64; t < s.pass() && t <= 64 * 128; t += 64) {  // beyond, two parts are too many
    const int64_t parts = lm_parts(t, on, in);
    if (parts > m.parts) m.parts = parts;
  }
  for (int64_t c = s.chunk_items() - 1; c > 0; --c) {  // the most rows with chunks of c items
    int64_t low = 0, high = s.T;  // chunk_items() <= c at low, > c at high
    while (high - low > 1) {
      a.T = low + (high - low) / 2;
      (a.chunk_items() > c ? high : low) = a.T;
    }
    a.T = low;
    if (low == 0 || a.chunk_items() < c) continue;
    if (a.chunks() > m.chunks) m.chunks = a.chunks();
    if (a.places() > m.places) m.places = a.places();
  }
  also(lm_space_many(s, backward, m, nullptr).bytes);
  return most;
}

mi_status lm_check(const char* what, const LmSizes& s, mi_dtype dt) {
  MI_REQUIRE(dt == MI_BF16 || dt == MI_F16, "%s: x, w and the banks must be bf16 or fp16", what);
  MI_REQUIRE(s.T >= 0 && s.T < (1LL << 31) - 256, "%s: rows out of range (%lld)", what, (long long)s.T);
  MI_REQUIRE(s.N >= 8 && s.N % 8 == 0, "%s: n %% 8 == 0 required (got n=%lld)", what, (long long)s.N);
  MI_REQUIRE(s.K >= 8 && s.K % 8 == 0, "%s: k %% 8 == 0 required (got k=%lld)", what, (long long)s.K);
  MI_REQUIRE(s.R >= 8 && s.R % 8 == 0 && s.R <= LM_MAX_RANK,
             "%s: rank must be a multiple of 8 in [8, %d] (got %lld)", what, LM_MAX_RANK, (long long)s.R);
  MI_REQUIRE(s.L >= 1 && s.L <= LM_MAX_ADAPTERS, "%s: num_adapters must be in [1, %d] (got %lld)", what,
             LM_MAX_ADAPTERS, (long long)s.L);
  MI_REQUIRE_SUPPORTED(s.N < (1LL << 20) && s.K < (1LL << 20) && s.N * s.K < (1LL << 30),
                       "%s: n and k below 2^20 and n * k below 2^30 required (w must fit one "
                       "31-bit buffer range; got n=%lld, k=%lld)", what, (long long)s.N, (long long)s.K);
  return MI_OK;
}

mi_status lm_plan(const LmSizes& s, int64_t rows, const int32_t* ids, const LmPlan& p, hipStream_t st) {
  // 64 chunks at most, of 1024 rows each at least
  int64_t chunk = (rows + 63) / 64;
  chunk = chunk <= PL_T ? PL_T : (chunk + PL_T - 1) / PL_T * PL_T;
  const int64_t blocks = rows > 0 ? (rows + chunk - 1) / chunk : 1;
  const dim3 grid(static_cast<unsigned>(blocks));
  const int T = static_cast<int>(rows), L = static_cast<int>(s.L), c = static_cast<int>(chunk);
  const int ci = static_cast<int>(s.chunk_items());
  if (rows <= PL_ONE) {
    hipLaunchKernelGGL(lm_place_kernel<true>, dim3(1), dim3(PL_T), 0, st, ids, T, L, c, ci, p);
    return launch_status("mm_lora (plan)");
  }
  hipLaunchKernelGGL(lm_count_kernel, grid, dim3(PL_T), 0, st, ids, T, L, c, p);
  const mi_status one = launch_status("mm_lora (plan)");
  if (one != MI_OK) return one;
  hipLaunchKernelGGL(lm_place_kernel<false>, grid, dim3(PL_T), 0, st, ids, T, L, c, ci, p);
  return launch_status("mm_lora (plan)");
}

template <bool F16, bool BT>
mi_status lm_shrink_run(const LmShrink& a, int64_t items, hipStream_t st) {
  const int nb = a.RP / 16;
#define LM_SHRINK(NB_)                                                                              \
  hipLaunchKernelGGL((lm_shrink_kernel<F16, BT, NB_>),                                              \
                     dim3(static_cast<unsigned>(items), static_cast<unsigned>((nb + NB_ - 1) / NB_)), \
                     dim3(64 * LmShape<NB_>::W), 0, st, a)
  // All ranks a workgroup, up to 64, where the rows fill the chip; else the ranks go to
  // several, which read the rows again, from the L2 (493 rows, 7640 columns, rank 48: 37 us
  // in one workgroup of 4 wavefronts, whose 119 steps are then 30 one after another)
  const int64_t full = a.T / LM_ITEM;
  if (nb == 1 || full < 64) LM_SHRINK(1);
  else if (nb == 2 || full < 128) LM_SHRINK(2);
  else LM_SHRINK(4);
#undef LM_SHRINK
  return launch_status("mm_lora (shrink)");
}

template <bool F16, bool BT, int WM, int WN, int FM, int FN, int NST, typename OutT>
mi_status lm_mm_launch(LmMm a, int splits, hipStream_t st) {
  constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN;
  const int64_t tiles = static_cast<int64_t>((a.T + BM - 1) / BM) * ((a.n + BN - 1) / BN);
  a.splits = splits;
  a.blocks = static_cast<int>((tiles + 7) / 8 * 8);
  hipLaunchKernelGGL((lm_mm_kernel<F16, BT, WM, WN, FM, FN, NST, OutT>),
                     dim3(static_cast<unsigned>(a.blocks) * splits), dim3(64 * WM * WN), 0, st, a);
  return launch_status("mm_lora (product)");
}

// Which tiles: us a call, plan and first product among them, n = k = 4096: 512 rows 64 x 64
// 34, 128 x 128 41; 768 rows 48 and 42; 2048 rows 128 x 128 67, 256 x 256 83; 3000 rows 97 and
// 91; n = k = 8192: 320 rows 64 x 64 78, 128 x 128 66; 1024 rows 128 x 128 121, 256 x 256 149;
// 1280 rows 168 and 152: each as long as the tiles run in one round of two workgroups per CU.
// Where the 64 x 64 tiles leave CUs idle, the k axis is split and the parts are added
// (parts: fp32 [splits, T, n]).
template <bool F16, bool BT, typename OutT>
mi_status lm_mm(const LmMm& a, float* parts, const int32_t* ids, hipStream_t st) {
  auto tiles = [&](int64_t bm, int64_t bn) { return (a.T + bm - 1) / bm * ((a.n + bn - 1) / bn); };
  const int splits = lm_wide_splits(a.T, a.n, a.k);
  if (splits > 1) {
    LmMm p = a;
    p.out = parts;
    p.bias = nullptr;
    const mi_status one = lm_mm_launch<F16, BT, 2, 2, 2, 2, 4, float>(p, splits, st);
    if (one != MI_OK) return one;
    LmSmall f{};  // no adapter is left to add
    f.mm = p;
    f.splits = splits;
    f.ids = ids;
    f.bias = a.bias;
    f.out = a.out;
    f.T = a.T;
    f.fin = static_cast<int>((static_cast<int64_t>(a.T) * (a.n / 4) + 255) / 256);
    hipLaunchKernelGGL((lm_finish_kernel<F16, false, OutT, float>), dim3(f.fin), dim3(256), 0, st, f);
    return launch_status("mm_lora (sums)");
  }
  if (tiles(64, 64) <= 512) return lm_mm_launch<F16, BT, 2, 2, 2, 2, 4, OutT>(a, 1, st);
  if (tiles(128, 128) > 512) return lm_mm_launch<F16, BT, 2, 4, 8, 4, 2, OutT>(a, 1, st);
  return lm_mm_launch<F16, BT, 2, 2, 4, 4, 2, OutT>(a, 1, st);
}

template <bool F16, bool BT, typename OutT, typename GradT>
mi_status lm_small_run(LmSmall p, hipStream_t st) {
  const char* what = BT ? "mm_lora_backward (few rows)" : "mm_lora (few rows)";
  if constexpr (!BT) {
    if (p.T == 1 && p.R <= 4 * ONE_W && (p.ca <= 6144 || p.cb >= 4096)) {
      auto one = [&](auto rw) {
        constexpr int RW = decltype(rw)::value;
        hipLaunchKernelGGL((lm_one_kernel<F16, RW, OutT>),
                           dim3(static_cast<unsigned>((p.cb + ONE_W * ONE_C - 1) / (ONE_W * ONE_C))),
                           dim3(64 * ONE_W), 0, st, p);
        return launch_status("mm_lora (one row)");
      };
      return p.R <= 2 * ONE_W ? one(std::integral_constant<int, 2>{}) : one(std::integral_constant<int, 4>{});
    }
  }
  const bool dense = p.out != nullptr;
  p.splits = lm_splits(p.T, p.mm.n, p.mm.k);
  p.tiles = (p.T + 63) / 64 * ((p.mm.n + 63) / 64);
  p.gemm = dense ? p.tiles * p.splits : 0;
  const int dots = (p.u != nullptr ? p.T * (p.R / 8) : 0) + (p.v != nullptr ? p.T * (p.R / 4) : 0);
  p.dots = (dots + 3) / 4 < 1024 ? (dots + 3) / 4 : 1024;
  p.fin = dense ? static_cast<int>((static_cast<int64_t>(p.T) * (p.mm.n / 4) + 255) / 256) : 0;
  hipLaunchKernelGGL((lm_parts_kernel<F16, BT>), dim3(p.gemm + p.dots), dim3(256), 0, st, p);
  const mi_status one = launch_status(what);
  if (one != MI_OK) return one;
  const int grads = p.ga == nullptr ? 0 : p.L * (p.R / 8) * ((p.ca + SG_COLS - 1) / SG_COLS + (p.cb + SG_COLS - 1) / SG_COLS);
  hipLaunchKernelGGL((lm_finish_kernel<F16, BT, OutT, GradT>), dim3(p.fin + grads), dim3(256), 0, st, p);
  return launch_status(what);
}

}  // namespace
}  // namespace mi

extern "C" size_t mi_mm_lora_workspace_size(int64_t m, int64_t n, int64_t k, int64_t num_adapters,
                                            int64_t rank, int backward) {
  const mi::LmSizes s{m, n, k, num_adapters, rank};
  if (mi::lm_check("mm_lora_workspace_size", s, MI_BF16) != MI_OK) return 0;
  return mi::lm_space_upto(s, backward != 0);
}

extern "C" mi_status mi_mm_lora(const void* x, int64_t m, int64_t k, mi_dtype dtype, const void* w,
                                int64_t n, const void* lora_a, const void* lora_b,
                                int64_t num_adapters, int64_t rank, const int32_t* lora_ids,
                                const float* lora_scale, const void* bias, void* out,
                                mi_dtype out_dtype, float* act, void* workspace,
                                size_t workspace_bytes, void* stream) {
  using namespace mi;
  clear_error();
  const char* what = "mm_lora";
  const LmSizes s{m, n, k, num_adapters, rank};
  mi_status st = lm_check(what, s, dtype);
  if (st != MI_OK) return st;
  MI_REQUIRE(out_dtype == MI_BF16 || out_dtype == MI_F16 || out_dtype == MI_F32,
             "%s: out_dtype must be bf16, fp16 or fp32", what);
  MI_REQUIRE_SUPPORTED(out_dtype == MI_F32 || out_dtype == dtype,
                       "%s: out_dtype must be x's type or fp32", what);
  if (m == 0) return MI_OK;
  MI_REQUIRE(x != nullptr && w != nullptr && lora_a != nullptr && lora_b != nullptr &&
                 lora_ids != nullptr && out != nullptr,
             "%s: x, w, lora_a, lora_b, lora_ids or out is null", what);
  MI_REQUIRE(aligned16(x) && aligned16(w) && aligned16(lora_a) && aligned16(lora_b) &&
                 aligned16(bias) && aligned16(out) && aligned16(act),
             "%s: x, w, lora_a, lora_b, bias, out and act must be 16-byte aligned", what);
  const int64_t ob = m * n * (out_dtype == MI_F32 ? 4 : 2), ab = m * rank * 4;
  const int64_t bank = num_adapters * rank * 2;
  auto clear_of = [&](const void* o, int64_t bytes) {
    return !overlap(o, bytes, x, m * k * 2) && !overlap(o, bytes, w, n * k * 2) &&
           !overlap(o, bytes, lora_a, bank * k) && !overlap(o, bytes, lora_b, bank * n) &&
           !overlap(o, bytes, lora_ids, m * 4) && !overlap(o, bytes, lora_scale, num_adapters * 4) &&
           !overlap(o, bytes, bias, n * 2) && !overlap(o, bytes, workspace, workspace_bytes);
  };
  MI_REQUIRE(clear_of(out, ob) && clear_of(act, ab) && !overlap(out, ob, act, ab),
             "%s: out and act may not overlap an input, the workspace or each other", what);
  const LmSpace sp = lm_space(s, false, workspace);
  MI_REQUIRE(workspace != nullptr && (reinterpret_cast<uintptr_t>(workspace) & 255) == 0 &&
                 workspace_bytes >= sp.bytes,
             "%s: the workspace needs %zu bytes, aligned to 256 (got %zu)", what, sp.bytes, workspace_bytes);
  hipStream_t hs = static_cast<hipStream_t>(stream);
  const int64_t es = out_dtype == MI_F32 ? 4 : 2;
  if (lm_small(s, false)) {
    LmSmall p{};
    p.mm.x = p.x = x;
    p.mm.w = w;
    p.mm.T = p.T = static_cast<int>(m);
    p.mm.k = p.ca = static_cast<int>(k);
    p.mm.n = p.cb = static_cast<int>(n);
    p.mm.L = p.L = static_cast<int>(num_adapters);
    p.R = static_cast<int>(rank);
    p.mm.out = sp.parts;
    p.a = lora_a;
    p.b = lora_b;
    p.ids = lora_ids;
    p.scale = lora_scale;
    p.v = sp.v;
    p.act = act;
    p.bias = bias;
    p.out = out;
    return dtype == MI_F16 ? (es == 4 ? lm_small_run<true, false, float, float>(p, hs)
                                      : lm_small_run<true, false, _Float16, float>(p, hs))
                           : (es == 4 ? lm_small_run<false, false, float, float>(p, hs)
                                      : lm_small_run<false, false, __bf16, float>(p, hs));
  }
  for (int64_t t0 = 0; t0 < m; t0 += s.pass()) {
    const int64_t rows = m - t0 < s.pass() ? m - t0 : s.pass();
    st = lm_plan(s, rows, lora_ids + t0, sp.plan, hs);
    if (st != MI_OK) return st;
    LmShrink a{};
    a.x = static_cast<const uint16_t*>(x) + t0 * k;
    a.bank = lora_a;
    a.scale = lora_scale;
    a.plan = sp.plan;
    a.out = act == nullptr ? nullptr : act + t0 * rank;
    a.pieces = sp.pieces;
    a.T = static_cast<int>(rows);
    a.C = static_cast<int>(k);
    a.L = static_cast<int>(num_adapters);
    a.R = static_cast<int>(rank);
    a.RP = static_cast<int>(s.rp());
    const int64_t items = LmSizes::items(rows, num_adapters);
    st = dtype == MI_F16 ? lm_shrink_run<true, false>(a, items, hs) : lm_shrink_run<false, false>(a, items, hs);
    if (st != MI_OK) return st;
    LmMm p{};
    p.x = a.x;
    p.w = w;
    p.bank = lora_b;
    p.bias = bias;
    p.pieces = sp.pieces;
    p.plan = sp.plan;
    p.out = static_cast<uint8_t*>(out) + t0 * n * es;
    p.T = a.T;
    p.k = static_cast<int>(k);
    p.n = static_cast<int>(n);
    p.L = a.L;
    p.R = a.R;
    p.RP = a.RP;
    const int32_t* const at = lora_ids + t0;
    st = dtype == MI_F16
             ? (es == 4 ? lm_mm<true, false, float>(p, sp.parts, at, hs) : lm_mm<true, false, _Float16>(p, sp.parts, at, hs))
             : (es == 4 ? lm_mm<false, false, float>(p, sp.parts, at, hs) : lm_mm<false, false, __bf16>(p, sp.parts, at, hs));
    if (st != MI_OK) return st;
  }
  return MI_OK;
}

extern "C" mi_status mi_mm_lora_backward(const void* grad_out, const void* x, int64_t m, int64_t k,
                                         mi_dtype dtype, const void* w, int64_t n,
                                         const void* lora_a, const void* lora_b,
                                         int64_t num_adapters, int64_t rank,
                                         const int32_t* lora_ids, const float* lora_scale,
                                         const float* act, void* grad_x, void* grad_a,
                                         void* grad_b, mi_dtype grad_dtype, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  using namespace mi;
  clear_error();
  const char* what = "mm_lora_backward";
  const LmSizes s{m, n, k, num_adapters, rank};
  mi_status st = lm_check(what, s, dtype);
  if (st != MI_OK) return st;
  MI_REQUIRE(grad_dtype == MI_F32 || grad_dtype == dtype,
             "%s: grad_a and grad_b must be fp32 or of x's type", what);
  const bool banks = grad_a != nullptr || grad_b != nullptr;
  MI_REQUIRE((grad_a == nullptr) == (grad_b == nullptr), "%s: grad_a and grad_b are given together", what);
  MI_REQUIRE(banks || grad_x != nullptr, "%s: no gradient is asked for", what);
  MI_REQUIRE(lora_a != nullptr && lora_b != nullptr, "%s: lora_a or lora_b is null", what);
  MI_REQUIRE(m == 0 || (grad_out != nullptr && lora_ids != nullptr &&
                        (grad_x == nullptr || w != nullptr) && (!banks || x != nullptr)),
             "%s: grad_out, x, w or lora_ids is null", what);
  MI_REQUIRE(aligned16(grad_out) && aligned16(x) && aligned16(w) && aligned16(lora_a) &&
                 aligned16(lora_b) && aligned16(act) && aligned16(grad_x) && aligned16(grad_a) &&
                 aligned16(grad_b),
             "%s: the tensors must be 16-byte aligned", what);
  // a grid has at most 2^32 - 1 threads along x: those of few rows' gradients are 1 / 16 of the banks
  MI_REQUIRE_SUPPORTED(!banks || num_adapters * rank * (n + k) < (1LL << 35),
                       "%s: num_adapters * rank * (n + k) below 2^35 required for the adapters' gradients", what);
  if (m == 0 && !banks) return MI_OK;
  const int64_t bank = num_adapters * rank, ges = grad_dtype == MI_F32 ? 4 : 2;
  const struct { const void* p; int64_t n; } outs[3] = {
      {grad_x, m * k * 2}, {grad_a, bank * k * ges}, {grad_b, bank * n * ges}},
      ins[9] = {{grad_out, m * n * 2}, {x, m * k * 2}, {w, n * k * 2}, {lora_a, bank * k * 2},
                {lora_b, bank * n * 2}, {lora_ids, m * 4}, {lora_scale, num_adapters * 4},
                {act, m * rank * 4}, {workspace, static_cast<int64_t>(workspace_bytes)}};
  for (int i = 0; i < 3; ++i) {
    for (const auto& in : ins)
      MI_REQUIRE(!overlap(outs[i].p, outs[i].n, in.p, in.n),
                 "%s: a gradient may not overlap an input or the workspace", what);
    for (int j = 0; j < i; ++j)
      MI_REQUIRE(!overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n),
                 "%s: the gradients may not overlap each other", what);
  }
  const LmSpace sp = lm_space(s, true, workspace);
  MI_REQUIRE(workspace != nullptr && (reinterpret_cast<uintptr_t>(workspace) & 255) == 0 &&
                 workspace_bytes >= sp.bytes,
             "%s: the workspace needs %zu bytes, aligned to 256 (got %zu)", what, sp.bytes, workspace_bytes);
  hipStream_t hs = static_cast<hipStream_t>(stream);
  const bool f16 = dtype == MI_F16, several = s.pass() < m;
  if (m > 0 && lm_small(s, true)) {
    LmSmall p{};
    p.mm.x = p.go = grad_out;
    p.x = x;
    p.mm.w = w;
    p.mm.T = p.T = static_cast<int>(m);
    p.mm.k = p.cb = static_cast<int>(n);
    p.mm.n = p.ca = static_cast<int>(k);
    p.mm.L = p.L = static_cast<int>(num_adapters);
    p.R = static_cast<int>(rank);
    p.mm.out = sp.parts;
    p.a = lora_a;
    p.b = lora_b;
    p.ids = lora_ids;
    p.scale = lora_scale;
    p.act_in = act;
    p.v = banks && act == nullptr ? sp.v : nullptr;
    p.u = sp.u;
    p.out = grad_x;
    p.ga = grad_a;
    p.gb = grad_b;
    return f16 ? (ges == 4 ? lm_small_run<true, true, _Float16, float>(p, hs)
                           : lm_small_run<true, true, _Float16, _Float16>(p, hs))
               : (ges == 4 ? lm_small_run<false, true, __bf16, float>(p, hs)
                           : lm_small_run<false, true, __bf16, __bf16>(p, hs));
  }
  auto shrink = [&](int64_t rows) {
    LmShrink a{};
    a.scale = lora_scale;
    a.plan = sp.plan;
    a.T = static_cast<int>(rows);
    a.L = static_cast<int>(num_adapters);
    a.R = static_cast<int>(rank);
    a.RP = static_cast<int>(s.rp());
    return a;
  };
  MI_REQUIRE_SUPPORTED(!several || !banks,
                       "%s: the adapters' gradients take at most %lld rows of these sizes", what,
                       (long long)s.pass());
  if (banks && m == 0) {
    st = lm_plan(s, 0, lora_ids, sp.plan, hs);
    if (st != MI_OK) return st;
  }
  for (int64_t t0 = 0; t0 < m; t0 += s.pass()) {
    const int64_t rows = m - t0 < s.pass() ? m - t0 : s.pass();
    st = lm_plan(s, rows, lora_ids + t0, sp.plan, hs);
    if (st != MI_OK) return st;
    const int64_t items = LmSizes::items(rows, num_adapters);
    const float* v = act;
    if (banks && act == nullptr) {
      LmShrink a = shrink(rows);
      a.x = x;
      a.bank = lora_a;
      a.C = static_cast<int>(k);
      a.out = sp.act;
      st = f16 ? lm_shrink_run<true, false>(a, items, hs) : lm_shrink_run<false, false>(a, items, hs);
      if (st != MI_OK) return st;
      v = sp.act;
    }
    LmShrink a = shrink(rows);
    a.x = static_cast<const uint16_t*>(grad_out) + t0 * n;
    a.bank = lora_b;
    a.C = static_cast<int>(n);
    a.pieces = grad_x == nullptr ? nullptr : sp.pieces;
    a.slots = static_cast<int>(LmSizes::items(m, num_adapters) * LM_ITEM);
    if (banks) {
      a.act = v;
      a.pieces_t = sp.ut;
      a.pieces_t2 = sp.vt;
    }
    st = f16 ? lm_shrink_run<true, true>(a, items, hs) : lm_shrink_run<false, true>(a, items, hs);
    if (st != MI_OK) return st;
    if (grad_x != nullptr) {
      LmMm p{};
      p.x = a.x;
      p.w = w;
      p.bank = lora_a;
      p.pieces = sp.pieces;
      p.plan = sp.plan;
      p.out = static_cast<uint16_t*>(grad_x) + t0 * k;
      p.T = a.T;
      p.k = static_cast<int>(n);
      p.n = static_cast<int>(k);
      p.L = a.L;
      p.R = a.R;
      p.RP = a.RP;
      const int32_t* const at = lora_ids + t0;
      st = f16 ? lm_mm<true, true, _Float16>(p, sp.parts, at, hs) : lm_mm<false, true, __bf16>(p, sp.parts, at, hs);
      if (st != MI_OK) return st;
    }
  }
  if (!banks) return MI_OK;
  LmGrad ga{};
  ga.x = x;
  ga.pieces_t = sp.ut;
  ga.plan = sp.plan;
  ga.part = sp.part_a;
  ga.out = grad_a;
  ga.C = static_cast<int>(k);
  ga.R = static_cast<int>(rank);
  ga.RP = static_cast<int>(s.rp());
  ga.slots = static_cast<int>(LmSizes::items(m, num_adapters) * LM_ITEM);
  LmGrad gb = ga;
  gb.x = grad_out;
  gb.pieces_t = sp.vt;
  gb.part = sp.part_b;
  gb.out = grad_b;
  gb.C = static_cast<int>(n);
  const unsigned panels = static_cast<unsigned>((k + GR_BN - 1) / GR_BN + (n + GR_BN - 1) / GR_BN);
  const int nb = ga.RP / 16, per = nb == 1 ? 1 : nb == 2 ? 2 : 4;
  const dim3 grid(panels, static_cast<unsigned>(s.chunks()), static_cast<unsigned>((nb + per - 1) / per));
  auto launch = [&](auto f, auto o) {
    constexpr bool F16 = decltype(f)::value;
    using OutT = decltype(o);
    if (per == 1) hipLaunchKernelGGL((lm_grad_kernel<F16, 1, OutT>), grid, dim3(256), 0, hs, ga, gb);
    else if (per == 2) hipLaunchKernelGGL((lm_grad_kernel<F16, 2, OutT>), grid, dim3(256), 0, hs, ga, gb);
    else hipLaunchKernelGGL((lm_grad_kernel<F16, 4, OutT>), grid, dim3(256), 0, hs, ga, gb);
    const mi_status one = launch_status("mm_lora_backward (adapters)");
    if (one != MI_OK || LmSizes::items(m, num_adapters) <= s.chunk_items()) return one;
    hipLaunchKernelGGL((lm_reduce_kernel<OutT>),
                       dim3(static_cast<unsigned>((rank * (n + k) / 4 + 255) / 256), static_cast<unsigned>(num_adapters)),
                       dim3(256), 0, hs, ga, gb);
    return launch_status("mm_lora_backward (sums)");
  };
  if (f16) return ges == 4 ? launch(std::true_type{}, float{}) : launch(std::true_type{}, _Float16{});
  return ges == 4 ? launch(std::false_type{}, float{}) : launch(std::false_type{}, __bf16{});
}
