// Matrix products of e4m3 codes with one fp32 scale per block of 128, on gfx950.
//
//   out[m, n] = sum_B sa[m, B] * sb[n / 128, B] * sum_{k in B} a[m, k] * b[n, k]
//
// with B the blocks of 128 along k: a carries a scale per 1 x 128 block (its
// own per row), b one per 128 x 128 block.  The grouped form does this for the
// rows [m_indptr[e], m_indptr[e+1]) of every expert e with b[e], sb[e].
//
// The inner sum of a block is one v_mfma_f32_16x16x128_f8f6f4 from a zero
// accumulator; its four fp32 results per lane are then added to the running
// sums with one fma each, the factor being sa * sb.  b is the MFMA's first
// operand, so a lane's results share one row of a (column lane % 16 of the
// result) and its factor is one register per 16 rows, and the lane holds four
// consecutive output columns.
//
// Precision.  That MFMA sums 8 consecutive products aligned to the largest
// exponent among them and keeps 13 bits below it (measured: 2^3 beside 2^16 is
// kept, 2^2 is not, at any of the 8 places; beyond them everything is fp32).  A
// product of two e4m3 codes has 6 fraction bits, so only products under 2^-7 of
// their group's largest lose any: at most 7 * 2^-13 of a group's largest term,
// 1.5e-5 of the result on normally distributed codes.  That is far below the
// rounding to a 16-bit output and accepted there for twice the rate.  An fp32
// output would show it: there the codes are converted to fp16 (exact) and
// multiplied with v_mfma_f32_16x16x32_f16, which sums in fp32 throughout.
#include "common.hpp"

namespace mi {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_void_ptr;

constexpr int F8_MAX_EXPERTS = 1024;
constexpr int F8_GROUP_M = 8;
constexpr int F8_BK = 128;             // one scale block: one 128-byte LDS row
// a lane offset past every descriptor's range: its load gives zero, its store is dropped
constexpr uint32_t F8_OUT = 0x80000000u;

__device__ __forceinline__ lds_void_ptr f8_lds(void* p) { return (lds_void_ptr)(p); }

// Chunk c (16 bytes) of LDS row R sits at slot c ^ f8_swz(R): the even and the odd
// ones of 16 rows take 8 different slots each, so the 16 rows of a fragment read
// cover all 64 banks.  Depends on R % 16 only: every 16-row block is read at the
// same offsets.
__device__ __forceinline__ int f8_swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }

struct F8Args {
  const uint8_t* a;        // [m_rows, k]
  const float* sa;         // [m_rows, sc]
  const uint8_t* b;        // [E, n, k]
  const float* sb;         // [E, nb, sc]
  const int32_t* m_indptr; // [E + 1], or null: one group of all rows
  void* out;               // [m_rows, n]
  int m_rows, k, n, E;
  int sc;                  // scale columns: 4 * ceil(k / 512)
  int nb;                  // scale rows of one b: ceil(n / 128)
};

// Wavefront 0 walks m_indptr: first row (s_row0, clamped) and first tile
// (s_t0) of every expert; entry E holds the ends.
template <int BM>
__device__ __forceinline__ void f8_walk(const int32_t* __restrict__ m_indptr, int m_rows, int E,
                                        int* s_t0, int* s_row0) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) / 64;
  const int e0 = lane * per;
  int c = 0;
  for (int e = e0; e < min(e0 + per, E); ++e) {
    const int s = min(max(m_indptr[e], 0), m_rows);
    const int t = min(max(m_indptr[e + 1], s), m_rows);
    s_row0[e] = s;
    c += (t - s + BM - 1) / BM;
    s_t0[e] = c;  // tiles of this lane's experts up to e; the lanes before are added below
  }
  int incl = c;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int v = __shfl_up(incl, off, 64);
    if (lane >= off) incl += v;
  }
  int prev = incl - c;
  for (int e = e0; e < min(e0 + per, E); ++e) {
    const int upto = s_t0[e] + incl - c;
    s_t0[e] = prev;
    prev = upto;
  }
  if (lane == 63) {
    s_t0[E] = incl;
    s_row0[E] = min(max(m_indptr[E], 0), m_rows);
  }
}

// the last e with pre[e] <= mt
__device__ __forceinline__ int f8_owner(const int* pre, int E, int mt) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= mt) lo = mid; else hi = mid;
  }
  return lo;
}

// m-tile and n-panel of the L-th tile: F8_GROUP_M m-tiles sweep the n-panels together
__device__ __forceinline__ void f8_order(long L, int count, int nt, int& mt, int& ni) {
  const long span = static_cast<long>(F8_GROUP_M) * nt;
  const int grp = static_cast<int>(L / span);
  const int first = grp * F8_GROUP_M;
  const int gsize = min(count - first, F8_GROUP_M);
  const int in_grp = static_cast<int>(L - static_cast<long>(grp) * span);
  mt = first + in_grp % gsize;
  ni = in_grp / gsize;
}

// four consecutive outputs of one row, rounded once to nearest even; an offset
// past the descriptor's range drops the store
template <typename OutT>
__device__ __forceinline__ void f8_store4(__amdgpu_buffer_rsrc_t r, uint32_t off, f32x4 v) {
  if constexpr (sizeof(OutT) == 4) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, off, 0, 0);
  } else {
    typedef OutT t4 __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b64(
        __builtin_bit_cast(u32x2, __builtin_convertvector(v, t4)), r, off, 0, 0);
  }
}

// a row's 32 codes of one lane as the MFMA takes them: raw, or as fp16
template <bool EXACT>
struct F8Frag {
  i32x8 v;
  __device__ F8Frag() {}
  __device__ explicit F8Frag(i32x8 c) : v(c) {}
};
template <>
struct F8Frag<true> {
  f16x8 v[4];
  __device__ F8Frag() {}
  __device__ explicit F8Frag(i32x8 c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], 1.f, false);
      const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], 1.f, true);
      v[i / 2][4 * (i & 1)] = lo[0];
      v[i / 2][4 * (i & 1) + 1] = lo[1];
      v[i / 2][4 * (i & 1) + 2] = hi[0];
      v[i / 2][4 * (i & 1) + 3] = hi[1];
    }
  }
};
// the block's product of 16 rows of b (result rows) and 16 of a (result columns)
__device__ __forceinline__ f32x4 f8_block(const F8Frag<false>& b, const F8Frag<false>& a) {
  const f32x4 z = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, z, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 f8_block(const F8Frag<true>& b, const F8Frag<true>& a) {
  f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 4; ++c) d = __builtin_amdgcn_mfma_f32_16x16x32_f16(b.v[c], a.v[c], d, 0, 0, 0);
  return d;
}

// One tile of BM = 16 FM WM rows and BN = 16 FN WN columns; WM * WN wavefronts.
// `rows` (1..BM) of the tile belong to the group.
//
// Staging: 8 rows of 128 bytes per DMA instruction straight into LDS, two
// stages.  Rows past the group or past n, and 16-byte chunks past k, load as
// zeros.  a's scales of four steps (16 bytes a row) go into one of two small
// LDS buffers, b's of 64 steps sit in one register, a lane each.
//
// A step is FM regions of one 16-row block of a each.  A region reads the
// fragment of the region after the next and issues its FN MFMAs; beside each the
// result of the last but one is added to the sums, so nothing is waited for
// where it is made.  The step's one barrier stands before its last two regions,
// whose operands are in registers by then: behind it the stage is free for the
// loads of step kt+2, and the next stage, loaded a step ago, is complete, so the
// last regions read the next step's first fragments while their MFMAs run.
template <int WM, int WN, int FM, int FN, typename OutT>
__device__ __forceinline__ void f8_tile(const F8Args& p, uint8_t* s0, uint8_t* s1, float* ssa0,
                                        float* ssa1, int e, int m0, int rows, int n0) {
  constexpr int NW = WM * WN, BM = 16 * FM * WM, BN = 16 * FN * WN;
  constexpr int NIA = BM / 8 / NW, NIB = BN / 8 / NW;  // DMA instructions per wavefront
  static_assert(NW % 4 == 0 && NIA * 8 * NW == BM && NIB * 8 * NW == BN, "tile");
  static_assert(BM % 64 == 0 && BM / 64 <= NW && 128 % (16 * FN) == 0 && FM >= 2 && FN >= 2, "tile");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int k = p.k, n = p.n, KT = (k + F8_BK - 1) / F8_BK;
  const int cols = min(n - n0, BN);

  const __amdgpu_buffer_rsrc_t ar = buf_rsrc(p.a + static_cast<long>(m0) * k,
                                             static_cast<uint32_t>(rows) * k);
  const __amdgpu_buffer_rsrc_t br = buf_rsrc(p.b + (static_cast<long>(e) * n + n0) * k,
                                             static_cast<uint32_t>(cols) * k);
  const __amdgpu_buffer_rsrc_t sar = buf_rsrc(p.sa + static_cast<long>(m0) * p.sc,
                                              static_cast<uint32_t>(rows) * p.sc * 4);
  // this wavefront's columns lie in one 128-column block of b
  const int sbrow = min((n0 + wn * 16 * FN) / 128, p.nb - 1);
  const float* sbp = p.sb + (static_cast<long>(e) * p.nb + sbrow) * p.sc;

  // DMA instruction i fills LDS rows 8 (NW i + wave) ..: lane l takes row l / 8
  // of them and chunk (l % 8) ^ f8_swz(row)
  const int lr = lane >> 3, chunk = (lane & 7) ^ lr ^ (wave & 1);
  uint32_t va[NIA], vb[NIB];
#pragma unroll
  for (int i = 0; i < NIA; ++i) {
    const int row = 8 * (NW * i + wave) + lr;
    va[i] = row < rows ? static_cast<uint32_t>(row) * k + chunk * 16 : F8_OUT;
  }
#pragma unroll
  for (int i = 0; i < NIB; ++i) {
    const int row = 8 * (NW * i + wave) + lr;
    vb[i] = row < cols ? static_cast<uint32_t>(row) * k + chunk * 16 : F8_OUT;
  }
  const uint32_t tail = (KT - 1) * F8_BK + chunk * 16 < k ? 0u : F8_OUT;
  // A step past the last loads zeros (its lane offsets are out of range): the
  // steps stay free of branches, which keep the compiler from moving a region's
  // additions into the next step.
  auto dma = [&](uint8_t* st, int kt) {
    const uint32_t so = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(min(kt, KT - 1)) * F8_BK);
    const uint32_t drop = kt < KT - 1 ? 0u : kt == KT - 1 ? tail : F8_OUT;
#pragma unroll
    for (int i = 0; i < NIA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, f8_lds(st + (NW * i + wave) * 1024), 16,
                                               va[i] | drop, so, 0, 0);
#pragma unroll
    for (int i = 0; i < NIB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(br, f8_lds(st + (BM + 8 * (NW * i + wave)) * 128),
                                               16, vb[i] | drop, so, 0, 0);
  };
  // 64 rows' scales per wavefront; wavefronts past the tile's rows load the same again
  const int swave = wave % (BM / 64), srow = swave * 64 + lane;
  const uint32_t vsa = srow < rows ? static_cast<uint32_t>(srow) * p.sc * 4 : F8_OUT;
  auto dma_scales = [&](float* buf, int kt) {  // kt a multiple of 4
    const uint32_t so = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(min(kt, p.sc - 4)) * 4);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(sar, f8_lds(buf + swave * 256), 16, vsa, so, 0, 0);
  };

  // fragments: lane (r, g) holds chunks c and c + 4 of row r of a 16-row block,
  // c = 0, 2, 1, 3 for g = 0 .. 3; a and b use the same chunks, so the order of k
  // inside the MFMA is theirs.  The LDS serves lanes l and l + 32 together: their
  // chunks have to differ in the lowest bit, which 0, 1, 2, 3 does not give (every
  // read then took twice its 4 cycles: 323 against 260 us at m 4096, n = k = 8192)
  const int r = lane & 15, g = lane >> 4;
  uint32_t fo[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    fo[h] = r * 128 + (((((g & 1) << 1) | (g >> 1)) + 4 * h) ^ f8_swz(r)) * 16;
  auto frag = [&](const uint8_t* st, int blk) {
    const u32x4 x = *reinterpret_cast<const u32x4*>(st + blk * 2048 + fo[0]);
    const u32x4 y = *reinterpret_cast<const u32x4*>(st + blk * 2048 + fo[1]);
    return i32x8{(int)x[0], (int)x[1], (int)x[2], (int)x[3],
                 (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  using Frag = F8Frag<sizeof(OutT) == 4>;
  const int ablk = wm * FM, bblk = BM / 16 + wn * FN;
  const int srd = (wm * FM * 16 + r) * 4;  // this lane's row of a scale buffer
  float sbv = 0.f;                         // b's scales of 64 steps
  i32x8 fb[FN];                            // b's fragments of the step
  i32x8 fa0, fa1;                          // a's of the next two regions,
  float sa0, sa1;                          // and their scales
  float f = 0.f;                           // the factor of the last region
  f32x4 d0 = {0.f, 0.f, 0.f, 0.f}, d1 = d0;  // the last two results, not yet added

  auto step = [&](auto S, uint8_t* st, uint8_t* nx, int kt) {
    constexpr int s = decltype(S)::value;
    float* const sc = s < 4 ? ssa0 : ssa1;
    float* const sc_nx = s < 4 ? ssa1 : ssa0;
    const float sb = __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sbv), kt & 63));
    Frag fbx[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) fbx[j] = Frag(fb[j]);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if (i == FM - 2) {
        __syncthreads();
        dma(st, kt + 2);
        if constexpr ((s & 3) == 0) dma_scales(sc_nx, kt + 4);
      }
      const Frag fax(fa0);
      const float f_prev = f;
      f = sa0 * sb;
      fa0 = fa1;
      sa0 = sa1;
      if (i < FM - 2) {
        fa1 = frag(st, ablk + i + 2);
        sa1 = sc[srd + 64 * (i + 2) + (s & 3)];
      } else {
        fa1 = frag(nx, ablk + i + 2 - FM);
        sa1 = (s & 3) < 3 ? sc[srd + 64 * (i + 2 - FM) + (s & 3) + 1]
                          : sc_nx[srd + 64 * (i + 2 - FM)];
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const f32x4 d2 = f8_block(fbx[j], fax);
        __builtin_amdgcn_sched_barrier(0);
        if (i == FM - 1) fb[j] = frag(nx, bblk + j);
        f32x4& o = acc[j >= 2 ? i : (i + FM - 1) % FM][(j + FN - 2) % FN];
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = __builtin_fmaf(d0[q], j >= 2 ? f : f_prev, o[q]);
        asm volatile("" : "+v"(o));  // the sum is complete here, not later
        d0 = d1;
        d1 = d2;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  dma(s0, 0);
  dma_scales(ssa0, 0);
  __syncthreads();
  dma(s1, 1);
  fa0 = frag(s0, ablk);
  fa1 = frag(s0, ablk + 1);
  sa0 = ssa0[srd];
  sa1 = ssa0[srd + 64];
#pragma unroll
  for (int j = 0; j < FN; ++j) fb[j] = frag(s0, bblk + j);
  for (int kt = 0; kt < KT; kt += 8) {
    if ((kt & 63) == 0) sbv = sbp[min(kt + lane, p.sc - 1)];
#define F8_STEP(S_, ST_, NX_)                                       \
  step(std::integral_constant<int, S_>{}, ST_, NX_, kt + S_);        \
  if (kt + S_ + 1 >= KT) break;
    F8_STEP(0, s0, s1)
    F8_STEP(1, s1, s0)
    F8_STEP(2, s0, s1)
    F8_STEP(3, s1, s0)
    F8_STEP(4, s0, s1)
    F8_STEP(5, s1, s0)
    F8_STEP(6, s0, s1)
    F8_STEP(7, s1, s0)
#undef F8_STEP
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    acc[FM - 1][FN - 2][q] = __builtin_fmaf(d0[q], f, acc[FM - 1][FN - 2][q]);
    acc[FM - 1][FN - 1][q] = __builtin_fmaf(d1[q], f, acc[FM - 1][FN - 1][q]);
  }

  // acc[i][j][q]: row (wm FM + i) 16 + r, column (wn FN + j) 16 + 4 g + q
  constexpr int ES = sizeof(OutT);
  const __amdgpu_buffer_rsrc_t orsrc =
      buf_rsrc(static_cast<OutT*>(p.out) + static_cast<long>(m0) * n,
               static_cast<uint32_t>(rows) * n * ES);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int row = (wm * FM + i) * 16 + r;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int col = (wn * FN + j) * 16 + 4 * g;
      f8_store4<OutT>(orsrc, row < rows && col < cols
                                 ? (static_cast<uint32_t>(row) * n + n0 + col) * ES : F8_OUT,
                      acc[i][j]);
    }
  }
}

// two wavefronts per SIMD: 256 registers each, all of them usable by the VALU,
// which adds the MFMAs' results
template <int WM, int WN, int FM, int FN, typename OutT>
__global__ __launch_bounds__(64 * WM * WN)
    __attribute__((amdgpu_waves_per_eu(2, 2))) void f8_mm_kernel(F8Args p) {
  constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN;
  __shared__ __attribute__((aligned(16))) uint8_t s0[(BM + BN) * F8_BK];
  __shared__ __attribute__((aligned(16))) uint8_t s1[(BM + BN) * F8_BK];
  __shared__ __attribute__((aligned(16))) float ssa0[BM * 4];
  __shared__ __attribute__((aligned(16))) float ssa1[BM * 4];
  const int nt = (p.n + BN - 1) / BN;
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  int e = 0, m0, rows, mt, ni;
  if (p.m_indptr == nullptr) {
    const int count = (p.m_rows + BM - 1) / BM;
    const long total = static_cast<long>(count) * nt, run = (total + 7) / 8;
    const long L = xcd * run + slot;
    if (slot >= run || L >= total) return;
    f8_order(L, count, nt, mt, ni);
    m0 = mt * BM;
    rows = min(p.m_rows - m0, BM);
  } else {
    // the walk's tables live in stage 1, which step 0 overwrites after a barrier
    static_assert((BM + BN) * F8_BK >= 2 * (F8_MAX_EXPERTS + 1) * 4, "tables");
    int* const s_t0 = reinterpret_cast<int*>(s1);
    int* const s_row0 = s_t0 + (F8_MAX_EXPERTS + 1);
    if ((threadIdx.x >> 6) == 0) f8_walk<BM>(p.m_indptr, p.m_rows, p.E, s_t0, s_row0);
    __syncthreads();
    const int count = s_t0[p.E];
    const long total = static_cast<long>(count) * nt, run = (total + 7) / 8;
    const long L = xcd * run + slot;
    if (slot >= run || L >= total) return;
    f8_order(L, count, nt, mt, ni);
    e = f8_owner(s_t0, p.E, mt);
    m0 = s_row0[e] + (mt - s_t0[e]) * BM;
    // the group's own end, read again: the next group's first row is another
    // number where m_indptr decreases
    rows = min(min(max(p.m_indptr[e + 1], s_row0[e]), p.m_rows) - m0, BM);
  }
  f8_tile<WM, WN, FM, FN, OutT>(p, s0, s1, ssa0, ssa1, __builtin_amdgcn_readfirstlane(e),
                                __builtin_amdgcn_readfirstlane(m0),
                                __builtin_amdgcn_readfirstlane(rows),
                                __builtin_amdgcn_readfirstlane(ni * BN));
}

template <int WM, int WN, int FM, int FN, typename OutT>
mi_status f8_launch(const F8Args& p, hipStream_t stream, const char* what) {
  constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN;
  // an upper bound on the tiles: a group's last tile may be partial, and there
  // are no more such groups than rows
  long tiles = (static_cast<long>(p.m_rows) + BM - 1) / BM;
  if (p.m_indptr != nullptr) tiles += p.E < p.m_rows ? p.E : p.m_rows;
  tiles *= (p.n + BN - 1) / BN;
  const long G = (tiles + 7) / 8 * 8;
  MI_REQUIRE(G < (1L << 31), "%s: problem too large", what);
  hipLaunchKernelGGL((f8_mm_kernel<WM, WN, FM, FN, OutT>), dim3(static_cast<unsigned>(G)),
                     dim3(64 * WM * WN), 0, stream, p);
  return launch_status(what);
}

template <typename OutT>
mi_status f8_dispatch(const F8Args& p, hipStream_t s, const char* what) {
  // fp32 outputs: the fp16 fragments take twice the registers, 128 x 64 tiles
  if constexpr (sizeof(OutT) == 4) {
    return f8_launch<2, 2, 4, 2, OutT>(p, s, what);
  } else {
    // 256 x 256 tiles halve the bytes each MFMA needs (m 4096, n = k = 8192: 243
    // against 288 us), but only where they fill the chip: m 1024 has 128 of them,
    // 90 against 69 us.  Groups' rows are known on the device only: the average.
    const long rows = p.m_rows / p.E;
    const long tiles = (rows + 255) / 256 * ((p.n + 255) / 256) * p.E;
    if (rows >= 192 && tiles >= 192) return f8_launch<2, 4, 8, 4, OutT>(p, s, what);
    return f8_launch<2, 2, 4, 4, OutT>(p, s, what);
  }
}

mi_status f8_run(const F8Args& p, int64_t m_rows, int64_t k, int64_t n, int64_t batch,
                 mi_dtype out_dtype, void* stream, const char* what) {
  MI_REQUIRE(m_rows >= 0 && m_rows < (1LL << 31) - 256, "%s: rows out of range (%lld)", what,
             (long long)m_rows);
  MI_REQUIRE(batch >= 1 && batch <= F8_MAX_EXPERTS, "%s: batch_size must be in [1, %d] (got %lld)",
             what, F8_MAX_EXPERTS, (long long)batch);
  MI_REQUIRE(n >= 16 && n % 16 == 0, "%s: n %% 16 == 0 required (got n=%lld)", what,
             (long long)n);
  MI_REQUIRE(k >= 16 && k % 16 == 0, "%s: k %% 16 == 0 required (got k=%lld)", what,
             (long long)k);
  MI_REQUIRE_SUPPORTED(k < (1LL << 22) && n < (1LL << 20),
                       "%s: k < 4194304 and n < 1048576 required (a tile's rows must fit one "
                       "31-bit buffer range; got k=%lld, n=%lld)", what, (long long)k,
                       (long long)n);
  MI_REQUIRE(out_dtype == MI_BF16 || out_dtype == MI_F16 || out_dtype == MI_F32,
             "%s: out_dtype must be bf16, fp16 or fp32", what);
  MI_REQUIRE(p.b != nullptr && p.sb != nullptr, "%s: b or b_scale is null", what);
  if (m_rows == 0) return MI_OK;
  MI_REQUIRE(p.a != nullptr && p.sa != nullptr && p.out != nullptr,
             "%s: a, a_scale or out is null", what);
  MI_REQUIRE(aligned16(p.a) && aligned16(p.b) && aligned16(p.sa) && aligned16(p.sb) &&
                 aligned16(p.out),
             "%s: a, b, their scales and out must be 16-byte aligned", what);
  F8Args q = p;
  q.m_rows = static_cast<int>(m_rows);
  q.k = static_cast<int>(k);
  q.n = static_cast<int>(n);
  q.E = static_cast<int>(batch);
  q.sc = static_cast<int>((k + 511) / 512 * 4);
  q.nb = static_cast<int>((n + 127) / 128);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (out_dtype == MI_BF16) return f8_dispatch<__bf16>(q, s, what);
  if (out_dtype == MI_F16) return f8_dispatch<_Float16>(q, s, what);
  return f8_dispatch<float>(q, s, what);
}

}  // namespace
}  // namespace mi

extern "C" mi_status mi_mm_fp8_block(const uint8_t* a, const float* a_scale, int64_t m, int64_t k,
                                     const uint8_t* b, const float* b_scale, int64_t n, void* out,
                                     mi_dtype out_dtype, void* stream) {
  using namespace mi;
  clear_error();
  F8Args p{};
  p.a = a;
  p.sa = a_scale;
  p.b = b;
  p.sb = b_scale;
  p.out = out;
  return f8_run(p, m, k, n, 1, out_dtype, stream, "mm_fp8_block");
}

extern "C" mi_status mi_grouped_mm_fp8_block(const uint8_t* a, const float* a_scale,
                                             int64_t m_rows, int64_t k, const uint8_t* b,
                                             const float* b_scale, int64_t batch, int64_t n,
                                             const int32_t* m_indptr, void* out,
                                             mi_dtype out_dtype, void* stream) {
  using namespace mi;
  clear_error();
  MI_REQUIRE(m_indptr != nullptr, "grouped_mm_fp8_block: m_indptr is null");
  F8Args p{};
  p.a = a;
  p.sa = a_scale;
  p.b = b;
  p.sb = b_scale;
  p.m_indptr = m_indptr;
  p.out = out;
  return f8_run(p, m_rows, k, n, batch, out_dtype, stream, "grouped_mm_fp8_block");
}
