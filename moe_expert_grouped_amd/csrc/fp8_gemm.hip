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
// their group's largest lose any: at most 7 * 2^-13 = 8.5e-4 of a group's largest
// term.  That bound is under a rounding to bf16 (2^-8) but over one to fp16 (2^-11),
// and an output that nearly cancels keeps the error of its terms.  On normally
// distributed codes the error is 2e-5 of the outputs' rms, 6e-5 and 9e-5 with one
// column of k in 64 20 and 100 times larger (a CPU model, k 4096); it then exceeds
// fp16's half step for 2, 8 and 11 outputs in a hundred, bf16's for 0.4, 0.9 and 1.5,
// all small ones.  16-bit outputs accept that for twice the rate, and the entry points
// say so; a caller who needs fp32 sums asks for an fp32 output.  There the codes are
// converted to fp16 (exact) and multiplied with v_mfma_f32_16x16x32_f16, which sums in
// fp32 throughout.
#include "common.hpp"

namespace mi {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_void_ptr;

constexpr int F8_MAX_EXPERTS = 1024;
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
  int zero_outside;        // out's rows outside the groups are zeroed
};

// inclusive sum over the wavefront's lanes
__device__ __forceinline__ uint32_t f8_scan(uint32_t v) {
#define F8_DPP(CTRL_, ROWS_) \
  v += __builtin_amdgcn_update_dpp(0, v, CTRL_, ROWS_, 0xf, true);
  F8_DPP(0x111, 0xf)  // row_shr 1, 2, 4, 8: within 16 lanes
  F8_DPP(0x112, 0xf)
  F8_DPP(0x114, 0xf)
  F8_DPP(0x118, 0xf)
  F8_DPP(0x142, 0xa)  // row_bcast 15: rows 0, 2 into 1, 3
  F8_DPP(0x143, 0xc)  // row_bcast 31: the lower half into the upper
#undef F8_DPP
  return v;
}

// m-tile and n-panel of the L-th tile of a group of `count` m-tiles: GM of them
// sweep the n-panels together
template <uint32_t GM>
__device__ __forceinline__ void f8_order(uint32_t L, uint32_t count, uint32_t nt, int& mt,
                                         int& ni) {
  const uint32_t span = GM * nt;
  const uint32_t grp = L / span;
  const uint32_t first = grp * GM;
  const uint32_t gsize = min(count - first, GM);
  const uint32_t in_grp = L - grp * span;
  // The m-tiles turn by one every 8 panels: consecutive tiles of one place then
  // are not all of the same height (128 very unequal experts, n 7168, k 2048: 684 us
  // without, 679 with; 64 experts of about 256 rows, n = k = 4096: 354 both)
  ni = in_grp / gsize;
  mt = first + (in_grp % gsize + ni / 8) % gsize;
}

struct F8Tile {
  int e, m0, rows, n0;  // rows == 0: this workgroup has no tile
  bool alone;           // the group's only m-tile
};

// The tile of BM rows and BN columns of this workgroup.  The grid is an upper
// bound on the tiles; workgroup ids go to the 8 XCDs in turn.  Each XCD has
// neighbours of the list of tiles, which its L2 serves: without groups one
// contiguous run, of groups' tiles chunks of up to CM, what an XCD runs at once,
// from the whole list.  With one run each an XCD may get all of a large group's
// full tiles.  One run and chunks, us: 64 experts of about 256 rows, n = k = 4096, 367
// and 354, of 256 rows each 297 both; very unequal groups go either way: 128 experts,
// k 7168, n 1536, 16384 rows 348 and 338, n 2048, 4096 rows 346 and 356; k 2048, n 7168,
// 32768 rows 675 and 679.
// The list has group after group, so that a place's b panels are a group's and its
// rows of a stay in L2 over their panels (m-tiles of several groups sweeping together
// took 2.5% more on very unequal experts, before the steps that followed).
// Every wavefront reads m_indptr itself: a lane has ceil(E / 64) experts, and
// where that is more than one, a second round resolves the lane's.
template <int BM, int BN, uint32_t CM>
__device__ __forceinline__ F8Tile f8_find(const F8Args& p) {
  const int lane = threadIdx.x & 63;
  const int per = (p.E + 63) / 64;
  const uint32_t nt = (p.n + BN - 1) / BN;
  const uint32_t xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  auto bounds = [&](int e, int& s, int& t) {  // rows of expert e, clamped
    if (p.m_indptr == nullptr) {
      s = 0;
      t = p.m_rows;
    } else {
      s = min(max(p.m_indptr[e], 0), p.m_rows);
      t = min(max(p.m_indptr[e + 1], s), p.m_rows);
    }
  };
  auto tiles = [](int s, int t) { return static_cast<uint32_t>(t - s + BM - 1) / BM; };
  F8Tile f{0, 0, 0, 0, false};
  uint32_t cnt = 0;
  int s = 0, t = 0;
  for (int e = lane * per; e < min((lane + 1) * per, p.E); ++e) {
    bounds(e, s, t);
    cnt += tiles(s, t);
  }
  uint32_t upto = f8_scan(cnt), before = upto - cnt;  // this lane's place in the list of tiles
  const uint32_t count = __builtin_amdgcn_readlane(upto, 63);
  const uint32_t total = count * nt;
  const uint32_t rounds =
      p.m_indptr == nullptr ? 1u : max((total + 8 * CM - 1) / (8 * CM), 1u);
  const uint32_t chunk = max((total + 8 * rounds - 1) / (8 * rounds), 1u);
  const uint32_t round = slot / chunk, L = (round * 8 + xcd) * chunk + slot % chunk;
  if (round >= rounds || L >= total) return f;
  int owner = __builtin_popcountll(__ballot(upto * nt <= L));
  f.e = owner * per;
  if (per > 1) {
    const uint32_t base = __builtin_amdgcn_readlane(before, owner);
    const int e = f.e + lane;
    s = t = 0;
    if (lane < per && e < p.E) bounds(e, s, t);
    cnt = tiles(s, t);
    upto = base + f8_scan(cnt);
    before = upto - cnt;
    owner = __builtin_popcountll(__ballot(upto * nt <= L));
    f.e += owner;
  }
  const int s_own = __builtin_amdgcn_readlane(s, owner), t_own = __builtin_amdgcn_readlane(t, owner);
  // 256-row tiles, 4, 6 and 8 together: m 4096, n = k = 8192 222.9, 222.9 and 223.2 us,
  // very unequal groups 679, 678 and 680; 64-row tiles, 8 and 16 at m 256: 30.1 and 30.2
  int mt, ni;
  f8_order<BM >= 256 ? 6 : 8>(L - __builtin_amdgcn_readlane(before, owner) * nt,
                              __builtin_amdgcn_readlane(cnt, owner), nt, mt, ni);
  f.m0 = s_own + mt * BM;
  f.n0 = ni * BN;
  // all so where m_indptr is what it has to be; the tiles of groups that overlap may
  // pass 32 bits, and then no tile outside the operands may come of it
  const bool in = f.e < p.E && static_cast<uint32_t>(ni) < nt && f.m0 >= s_own && f.m0 < t_own;
  f.rows = in ? min(t_own - f.m0, BM) : 0;
  f.alone = t_own - s_own <= BM;
  return f;
}

// Zeros to out's rows before the first group and behind the last one, this
// workgroup's share of them.
template <typename OutT>
__device__ __forceinline__ void f8_zero_outside(const F8Args& p) {
  if (!p.zero_outside) return;
  const int first = min(max(p.m_indptr[0], 0), p.m_rows);
  const int last = min(max(p.m_indptr[p.E], first), p.m_rows);
  if (first == 0 && last == p.m_rows) return;
  const int64_t per_row = static_cast<int64_t>(p.n) * sizeof(OutT) / 16;  // 16-byte pieces
  const int64_t head = first * per_row, all = head + (p.m_rows - last) * per_row;
  char* const out = static_cast<char*>(p.out);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < all;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    gst<u32x4>(out + (i < head ? i : i - head + last * per_row) * 16, u32x4{0, 0, 0, 0});
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
// a quarter of it on top of d: the four of a block depend on each other, so those
// of several blocks are issued in turn (block after block and in turn, us: 64 experts of
// about 256 rows, n = k = 4096, 587 and 581; m 4096, n = k = 8192 457 and 451; m 333,
// n 1744, k 2064 9.6 and 9.5)
__device__ __forceinline__ f32x4 f8_quarter(const F8Frag<true>& b, const F8Frag<true>& a, int c,
                                            f32x4 d) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(b.v[c], a.v[c], d, 0, 0, 0);
}

// at most N of this wavefront's loads are outstanding, its LDS reads have
// returned, and every wavefront is here
template <int N>
__device__ __forceinline__ void f8_wait_barrier() {
  // no access may move across, in the compiler either
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));  // vmcnt(N) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// the LDS rows of one step: the tile's rows 0 .. 127 and 128 .. of a, and of b.
// A pointer to one array, or to its half, is known at compile time wherever LDS is
// read (the compiler then knows which of the loads in flight a read waits for; one
// chosen at run time would wait for all).
struct F8Stage {
  uint8_t *a0, *a1, *b0, *b1;
};

// One tile of BM = 16 FM WM rows and BN = 16 FN WN columns; WM * WN wavefronts.
// `rows` (1..BM) of the tile belong to the group.
//
// Staging: 8 rows of 128 bytes per DMA instruction straight into LDS, NST
// stages (two to four).  Rows past the group or past n, and 16-byte chunks past k,
// load as zeros.  a's scales of four steps (16 bytes a row) go into one of two (with
// three stages three) small LDS buffers, b's of 64 steps sit in one register, a lane
// each.
//
// A step is FM regions of one 16-row block of a each.  A region reads the
// fragment of the region after the next and issues its FN MFMAs; beside each the
// result of the last but one is added to the sums (with fp32 outputs the last
// region's), so nothing is waited for where it is made.  The step's one barrier
// stands before its last two regions, whose operands are in registers by then:
// behind it the stage is free for the loads of step kt+NST, and the next stage is
// complete (the wait leaves the loads of the later ones in flight), so the last
// regions read the next step's first fragments while their MFMAs run.
template <int WM, int WN, int FM, int FN, int NST, bool STREAM, typename OutT>
__device__ __forceinline__ void f8_tile(const F8Args& p, F8Stage s0, F8Stage s1, F8Stage s2,
                                        F8Stage s3, float* ssa0, float* ssa1, float* ssa2,
                                        uint8_t* reg, const F8Tile& t) {
  const int e = t.e, m0 = t.m0, rows = t.rows, n0 = t.n0;
  constexpr int NW = WM * WN, BM = 16 * FM * WM, BN = 16 * FN * WN;
  constexpr int NIA = BM / 8 / NW, NIB = BN / 8 / NW;  // DMA instructions per wavefront
  // the loads of the stages after the next may be in flight at a step's barrier
  // (the scales' among them, which are read two steps after their load at least)
  constexpr int FLY = (NST - 2) * (NIA + NIB);
  static_assert(NST >= 2 && NST <= 4 && FLY < 64, "stages");
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
  // Where a stage is in pieces every wavefront has rows in both: SPLIT_A half of its
  // rows of a in 0 .. 127 and half in 128 .., SPLIT the same of its rows of b.  Else
  // they are consecutive, and those of b are in one 128-column block.
  constexpr bool SPLIT = NST == 3, SPLIT_A = BM == 256;
  static_assert(!SPLIT || BN == 256, "split");
  const int sbrow = SPLIT ? n0 / 128 : min((n0 + wn * 16 * FN) / 128, p.nb - 1);
  const float* sbp = p.sb + (static_cast<long>(e) * p.nb + sbrow) * p.sc;
  const float* sbp1 = sbp + (SPLIT && sbrow + 1 < p.nb ? p.sc : 0);

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
  // STREAM: the steps go through the blocks of k from `rot` on, a multiple of 4
  // (one load of a's scales), and round the end; every n-panel of b and every group
  // has its own start.  With one start for all, workgroups ask for the same bytes of
  // rows that are a multiple of 4096 apart, and those lie in a few memory channels.
  const int rot = STREAM && k % 4096 == 0 ? (n0 / BN + e) % (KT / 4) * 4 : 0;
  auto block = [&](int kt) { return !STREAM || kt + rot < KT ? kt + rot : kt + rot - KT; };
  // A step past the last loads zeros (its lane offsets are out of range): the
  // steps stay free of branches, which keep the compiler from moving a region's
  // additions into the next step.
  // Pieces [first, first + count) of the NI loads of a stage.
  constexpr int NI = NIA + NIB;
  auto dma = [&](const F8Stage& st, int kt, int first, int count) {
    const int kb = block(min(kt, KT - 1));  // KT - 1 itself has the tail: rot is 0 then
    const uint32_t so = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(kb) * F8_BK);
    const uint32_t drop = kt >= KT ? F8_OUT : kb == KT - 1 ? tail : 0u;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (i < first || i >= first + count) continue;
      if (i < NIA)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            ar, f8_lds(NW * i < 16 ? st.a0 + (NW * i + wave) * 1024
                                   : st.a1 + (NW * i - 16 + wave) * 1024),
            16, va[i < NIA ? i : 0] | drop, so, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            br, f8_lds(NW * (i - NIA) < 16 ? st.b0 + (NW * (i - NIA) + wave) * 1024
                                           : st.b1 + (NW * (i - NIA) - 16 + wave) * 1024),
            16, vb[i < NIA ? 0 : i - NIA] | drop, so, 0, STREAM ? 2 : 0);
    }
  };
  // 64 rows' scales per wavefront; wavefronts past the tile's rows load the same again
  const int swave = wave % (BM / 64), srow = swave * 64 + lane;
  const uint32_t vsa = srow < rows ? static_cast<uint32_t>(srow) * p.sc * 4 : F8_OUT;
  auto dma_scales = [&](float* buf, int kt) {  // kt a multiple of 4
    const uint32_t so =
        __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(kt < KT ? block(kt) : 0) * 4);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(sar, f8_lds(buf + swave * 256), 16, vsa, so, 0, 0);
  };

  // fragments: lane (r, g) holds chunks c and c + 4 of row r of a 16-row block,
  // c = 0, 2, 1, 3 for g = 0 .. 3; a and b use the same chunks, so the order of k
  // inside the MFMA is theirs.  The LDS serves lanes l and l + 32 together: their
  // chunks have to differ in the lowest bit, which 0, 1, 2, 3 does not give (every
  // read then takes twice its 4 cycles: 226 against 222 us at m 4096, n = k = 8192)
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

  constexpr bool EXACT = sizeof(OutT) == 4;
  using Frag = F8Frag<EXACT>;
  auto frag_a = [&](const F8Stage& st, int i) {
    return SPLIT_A ? frag(i < FM / 2 ? st.a0 : st.a1, wm * (FM / 2) + i % (FM / 2))
                   : frag(st.a0, wm * FM + i);
  };
  // block j of this wavefront's columns
  auto frag_b = [&](const F8Stage& st, int j) {
    return SPLIT ? frag(j < FN / 2 ? st.b0 : st.b1, wn * (FN / 2) + j % (FN / 2))
                 : frag(st.b0, wn * FN + j);
  };
  const int srd = (wm * (SPLIT_A ? 64 : FM * 16) + r) * 4;  // this lane's row of a scale buffer
  auto soff = [](int i) { return SPLIT_A && i >= FM / 2 ? 512 + 64 * (i - FM / 2) : 64 * i; };
  float sbv = 0.f, sbv1 = 0.f;             // b's scales of 64 steps
  i32x8 fb[FN];                            // b's fragments of the step
  i32x8 fa0, fa1;                          // a's of the next two regions,
  float sa0, sa1;                          // and their scales
  float f = 0.f, f1 = 0.f;                 // the factors of the last region, by block of b
  // results not yet added: the last two, of fp32 outputs the last region's
  constexpr int ND = EXACT ? FN : 2;
  f32x4 d[ND];
#pragma unroll
  for (int j = 0; j < ND; ++j) d[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto add = [](f32x4& o, f32x4 v, float by) {
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = __builtin_fmaf(v[q], by, o[q]);
  };

  // A stage's loads go out PPR per region from the one behind the barrier on, over
  // half of the regions: all at once they hold up the MFMAs behind them, later
  // they would not arrive in time.
  constexpr int PPR = (2 * NI + FM - 1) / FM;
  auto step = [&](auto S, const F8Stage& pv, const F8Stage& st, const F8Stage& nx, int kt) {
    constexpr int s = decltype(S)::value;
    // with three stages the unrolled steps are 12 and the scale buffers three
    float* const sc = s < 4 ? ssa0 : s < 8 ? ssa1 : ssa2;
    float* const sc_nx = s < 4 ? ssa1 : s < 8 && NST == 3 ? ssa2 : ssa0;
    const float sb = __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sbv), block(kt) & 63));
    const float sb1 =
        !SPLIT ? sb
               : __builtin_bit_cast(float, __builtin_amdgcn_readlane(
                                               __builtin_bit_cast(int, sbv1), block(kt) & 63));
    Frag fbx[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) fbx[j] = Frag(fb[j]);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if (i == FM - 2) {
        f8_wait_barrier<FLY>();
        if constexpr ((s & 3) == 0) dma_scales(sc_nx, kt + 4);
      }
      constexpr int R0 = FM - 2;  // the region behind the barrier
      if (i >= R0) dma(st, kt + NST, (i - R0) * PPR, PPR);
      else if ((i + 2) * PPR < NI) dma(pv, kt + NST - 1, (i + 2) * PPR, PPR);
      const Frag fax(fa0);
      const float f_prev = f, f1_prev = f1;
      f = sa0 * sb;
      f1 = SPLIT ? sa0 * sb1 : f;
      fa0 = fa1;
      sa0 = sa1;
      if (i < FM - 2) {
        fa1 = frag_a(st, i + 2);
        sa1 = sc[srd + soff(i + 2) + (s & 3)];
      } else {
        fa1 = frag_a(nx, i + 2 - FM);
        sa1 = (s & 3) < 3 ? sc[srd + 64 * (i + 2 - FM) + (s & 3) + 1]
                          : sc_nx[srd + 64 * (i + 2 - FM)];
      }
      // the sum is complete at its asm, not later
      if constexpr (EXACT) {
        f32x4 dn[FN];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            dn[j] = f8_quarter(fbx[j], fax, c, c ? dn[j] : f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if (i == FM - 1) fb[j] = frag_b(nx, j);
          f32x4& o = acc[(i + FM - 1) % FM][j];
          add(o, d[j], SPLIT && j >= FN / 2 ? f1_prev : f_prev);
          asm volatile("" : "+v"(o));
          d[j] = dn[j];
        }
        __builtin_amdgcn_sched_barrier(0);
      } else {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const f32x4 d2 = f8_block(fbx[j], fax);
          __builtin_amdgcn_sched_barrier(0);
          if (i == FM - 1) fb[j] = frag_b(nx, j);
          f32x4& o = acc[j >= 2 ? i : (i + FM - 1) % FM][(j + FN - 2) % FN];
          const bool second = SPLIT && (j + FN - 2) % FN >= FN / 2;
          add(o, d[0], j >= 2 ? (second ? f1 : f) : (second ? f1_prev : f_prev));
          asm volatile("" : "+v"(o));
          d[0] = d[1];
          d[1] = d2;
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  };

  // b's scales of the 64 blocks that block kb is one of; before the stages, as a
  // wait for them would be a wait for everything before them
  auto load_sb = [&](int kb) {
    const int c = min((kb & ~63) + lane, p.sc - 1);
    sbv = sbp[c];
    if constexpr (SPLIT) sbv1 = sbp1[c];
  };
  load_sb(block(0));
  dma(s0, 0, 0, NI);
  dma_scales(ssa0, 0);
  if constexpr (NST >= 3) dma(s1, 1, 0, NI);
  if constexpr (NST == 4) dma(s2, 2, 0, NI);
  f8_wait_barrier<FLY>();
  dma(NST == 4 ? s3 : NST == 3 ? s2 : s1, NST - 1, 0, 2 * PPR);  // the rest in step 0
  fa0 = frag_a(s0, 0);
  fa1 = frag_a(s0, 1);
  sa0 = ssa0[srd];
  sa1 = ssa0[srd + 64];
#pragma unroll
  for (int j = 0; j < FN; ++j) fb[j] = frag_b(s0, j);
  const F8Stage* const sts[4] = {&s0, &s1, &s2, &s3};
  constexpr int UNROLL = NST == 3 ? 12 : 8;
  for (int kt = 0; kt < KT; kt += UNROLL) {
#define F8_STEP(S_)                                                                       \
  if (S_ % 4 == 0 && KT > 64 && kt + S_ > 0 && (block(kt + S_) & 63) < 4)                 \
    load_sb(block(kt + S_));                                                              \
  step(std::integral_constant<int, S_>{}, *sts[(S_ + NST - 1) % NST], *sts[S_ % NST],     \
       *sts[(S_ + 1) % NST], kt + S_);                                                    \
  if (kt + S_ + 1 >= KT) break;
    F8_STEP(0)
    F8_STEP(1)
    F8_STEP(2)
    F8_STEP(3)
    F8_STEP(4)
    F8_STEP(5)
    F8_STEP(6)
    F8_STEP(7)
    if constexpr (UNROLL == 12) {
      F8_STEP(8)
      F8_STEP(9)
      F8_STEP(10)
      F8_STEP(11)
    }
#undef F8_STEP
  }
  // the loads of the steps past the last write (zeros) to LDS: not after this
  // workgroup's end
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
#pragma unroll
  for (int j = 0; j < ND; ++j)
    add(acc[FM - 1][FN - ND + j], d[j], SPLIT && FN - ND + j >= FN / 2 ? f1 : f);

  // acc[i][j][q]: row 16 i + r, column 16 j + 4 g + q of the wavefront's.  Its
  // outputs go through its own part of the stages (`reg`, free after the barrier)
  // so that it stores whole runs of RB bytes of a row (SPLIT: two of half), 16 bytes
  // a lane, instead of 8 bytes from each of 64 places.  16-byte chunk c of a row sits at
  // slot c ^ (row % CPR).  The stores are streaming (non-temporal): they cover
  // whole 64-byte pieces at least and the outputs do not push operands out of L2
  // (128 very unequal experts: 687 us with ordinary stores, 679 streaming; 8-byte stores
  // from the lanes themselves took 10% more than these rows when they were replaced).
  constexpr int ES = sizeof(OutT), RB = 16 * FN * ES, CPR = RB / 16, REG = 16 * FM * RB;
  static_assert(REG <= 16 * 1024 && 64 % CPR == 0, "epilogue");
  f8_wait_barrier<0>();
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int row = 16 * i + r;
      if constexpr (ES == 4) {
        *reinterpret_cast<f32x4*>(reg + row * RB + ((4 * j + g) ^ (r % CPR)) * 16) = acc[i][j];
      } else {
        typedef OutT t4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<t4*>(reg + row * RB + ((2 * j + (g >> 1)) ^ (r % CPR)) * 16 +
                               (g & 1) * 8) = __builtin_convertvector(acc[i][j], t4);
      }
    }
  const __amdgpu_buffer_rsrc_t orsrc =
      buf_rsrc(static_cast<OutT*>(p.out) + static_cast<long>(m0) * n,
               static_cast<uint32_t>(rows) * n * ES);
  constexpr int RPI = 64 / CPR;  // rows per store
  const int pr = lane / CPR, pc = lane % CPR;
  const int lc = pc * (16 / ES);
  const int col = SPLIT ? wn * 8 * FN + lc + (lc < 8 * FN ? 0 : 128 - 8 * FN) : wn * 16 * FN + lc;
#pragma unroll
  for (int r0 = 0; r0 < 16 * FM; r0 += RPI) {
    const int lrow = r0 + pr;
    const int row = SPLIT_A ? wm * 64 + lrow + (lrow & 64) : wm * FM * 16 + lrow;
    const u32x4 v = *reinterpret_cast<const u32x4*>(reg + lrow * RB + (pc ^ (lrow % CPR)) * 16);
    __builtin_amdgcn_raw_buffer_store_b128(
        v, orsrc, row < rows && col < cols ? (static_cast<uint32_t>(row) * n + n0 + col) * ES : F8_OUT,
        0, 2);
  }
}

// Tiles of one shape.  Two wavefronts per SIMD: 256 registers each, all of them
// usable by the VALU, which adds the MFMAs' results.
template <int WM, int WN, int FM, int FN, int NST, bool STREAM, typename OutT>
__device__ __forceinline__ void f8_mid_tile(const F8Args& p, const F8Stage* st, float* ssa0,
                                            float* ssa1, uint8_t* reg, const F8Tile& t) {
  if constexpr (FM >= 4) {
    if (t.rows <= 8 * FM * WM) {  // a group's last tile: half the work
      f8_tile<WM, WN, FM / 2, FN, NST, STREAM, OutT>(p, st[0], st[1], st[2], st[3], ssa0, ssa1,
                                                     ssa0, reg, t);
      return;
    }
  }
  f8_tile<WM, WN, FM, FN, NST, STREAM, OutT>(p, st[0], st[1], st[2], st[3], ssa0, ssa1, ssa0, reg,
                                             t);
}
template <int WM, int WN, int FM, int FN, int NST, bool STREAM, typename OutT>
__global__ __launch_bounds__(64 * WM * WN)
    __attribute__((amdgpu_waves_per_eu(2, 2))) void f8_mm_kernel(F8Args p) {
  constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN, STAGE = (BM + BN) * F8_BK;
  // each stage its own array: the compiler then knows which loads a read waits for
  __shared__ __attribute__((aligned(16))) uint8_t s0[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t s1[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t s2[NST == 4 ? STAGE : 16];
  __shared__ __attribute__((aligned(16))) uint8_t s3[NST == 4 ? STAGE : 16];
  __shared__ __attribute__((aligned(16))) float ssa0[BM * 4];
  __shared__ __attribute__((aligned(16))) float ssa1[BM * 4];
  f8_zero_outside<OutT>(p);
  const F8Tile t = f8_find<BM, BN, 64>(p);  // two workgroups per CU
  if (t.rows == 0) return;
  static_assert(BM <= 128 && BN <= 128, "halves");
  constexpr int B = BM * F8_BK;  // b's rows follow a's
  auto stage = [](uint8_t* s) { return F8Stage{s, s, s + B, s + B}; };
  const F8Stage st[4] = {stage(s0), stage(s1), stage(NST == 4 ? s2 : s0), stage(NST == 4 ? s3 : s1)};
  // a wavefront's part of the stages for its outputs
  constexpr int NW = WM * WN, REG = 16 * FM * 16 * FN * sizeof(OutT);
  static_assert(NW / 2 * REG <= STAGE, "epilogue");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* const reg = (wave < NW / 2 ? s0 : s1) + wave % (NW / 2) * REG;
  if (STREAM && t.alone)
    f8_mid_tile<WM, WN, FM, FN, NST, STREAM, OutT>(p, st, ssa0, ssa1, reg, t);
  else
    f8_mid_tile<WM, WN, FM, FN, NST, false, OutT>(p, st, ssa0, ssa1, reg, t);
}

// 256 x 256 tiles; a group's last tile, where it has at most 128 or 64 rows, does a
// half or a quarter of the work.  It keeps its place among the group's tiles,
// which share b's panels in L2.  Such a low tile's step is shorter than its loads
// take, so it has three stages of 48 KB where the tall one has two of 64: LDS arrays
// that make up either.  Two stages and three, us: 128 experts, n 7168, k 2048, of 128
// rows each 438 and 404, of very unequal rows 693 and 678; 64 of about 256 rows,
// n = k = 4096, where few tiles are low, 348 and 354.
template <bool STREAM, typename OutT>
__device__ __forceinline__ void f8_large_tile(const F8Args& p, uint8_t* s0, uint8_t* s1,
                                              uint8_t* t0, uint8_t* t1, uint8_t* u, float* ssa0,
                                              float* ssa1, float* ssa2, uint8_t* reg,
                                              const F8Tile& t) {
  constexpr int Q = 128 * F8_BK;
  if (t.rows > 128) {
    const F8Stage st0{s0, t0, s0 + Q, s0 + 2 * Q}, st1{s1, t1, s1 + Q, s1 + 2 * Q};
    f8_tile<2, 4, 8, 4, 2, STREAM, OutT>(p, st0, st1, st0, st1, ssa0, ssa1, ssa0, reg, t);
  } else {
    const F8Stage st0{s0, s0, s0 + Q, s0 + 2 * Q}, st1{s1, s1, s1 + Q, s1 + 2 * Q},
        st2{u, u, t0, t1};
    if (t.rows > 64)
      f8_tile<2, 4, 4, 4, 3, STREAM, OutT>(p, st0, st1, st2, st0, ssa0, ssa1, ssa2, reg, t);
    else
      f8_tile<1, 8, 4, 2, 3, STREAM, OutT>(p, st0, st1, st2, st0, ssa0, ssa1, ssa2, reg, t);
  }
}
template <bool STREAM, typename OutT>
__global__ __launch_bounds__(512)
    __attribute__((amdgpu_waves_per_eu(2, 2))) void f8_mm_large_kernel(F8Args p) {
  constexpr int Q = 128 * F8_BK;  // 128 rows
  __shared__ __attribute__((aligned(16))) uint8_t s0[3 * Q], s1[3 * Q], t0[Q], t1[Q], u[Q];
  __shared__ __attribute__((aligned(16))) float ssa0[256 * 4], ssa1[256 * 4], ssa2[128 * 4];
  f8_zero_outside<OutT>(p);
  const F8Tile t = f8_find<256, 256, 32>(p);
  if (t.rows == 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* const reg = wave < 3   ? s0 + wave * Q
                       : wave < 6 ? s1 + (wave - 3) * Q
                                  : (wave < 7 ? t0 : t1);
  if (STREAM && t.alone)
    f8_large_tile<STREAM, OutT>(p, s0, s1, t0, t1, u, ssa0, ssa1, ssa2, reg, t);
  else
    f8_large_tile<false, OutT>(p, s0, s1, t0, t1, u, ssa0, ssa1, ssa2, reg, t);
}

// ---------------------------------------------------------------------------
// Few rows: the call streams b from memory, so every wavefront loads it
// straight into MFMA operands (no LDS, no barrier) with P steps in flight.  A
// workgroup has 16 FM rows and 16 FN columns; its NW wavefronts take the
// steps (128 columns of k) in turn, NW consecutive lines of each row of b at a
// time, and their sums are added in wavefront order in LDS at the end.
// ---------------------------------------------------------------------------
template <int FM, int FN, int NW, int P, typename OutT>
__global__ __launch_bounds__(64 * NW) void f8_mm_few_kernel(F8Args p) {
  constexpr int BM = 16 * FM, BN = 16 * FN;
  static_assert(128 % BN == 0, "one b scale per step");
  __shared__ __attribute__((aligned(16))) f32x4 red[NW * FM * FN * 64];
  f8_zero_outside<OutT>(p);
  const F8Tile t = f8_find<BM, BN, 1u << 26>(p);
  if (t.rows == 0) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int k = p.k, n = p.n, KT = (k + F8_BK - 1) / F8_BK;
  const int cols = min(n - t.n0, BN);
  const int r = lane & 15, g = lane >> 4;
  const __amdgpu_buffer_rsrc_t ar = buf_rsrc(p.a + static_cast<long>(t.m0) * k,
                                             static_cast<uint32_t>(t.rows) * k);
  const __amdgpu_buffer_rsrc_t br = buf_rsrc(p.b + (static_cast<long>(t.e) * n + t.n0) * k,
                                             static_cast<uint32_t>(cols) * k);
  const __amdgpu_buffer_rsrc_t sar = buf_rsrc(p.sa + static_cast<long>(t.m0) * p.sc,
                                              static_cast<uint32_t>(t.rows) * p.sc * 4);
  const float* sbp = p.sb + (static_cast<long>(t.e) * p.nb + t.n0 / 128) * p.sc;

  // lane (r, g): chunks g and g + 4 of row r
  uint32_t va[FM], vs[FM], vb[FN];
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const bool in = 16 * i + r < t.rows;
    va[i] = in ? static_cast<uint32_t>(16 * i + r) * k + g * 16 : F8_OUT;
    vs[i] = in ? static_cast<uint32_t>(16 * i + r) * p.sc * 4 : F8_OUT;
  }
#pragma unroll
  for (int j = 0; j < FN; ++j)
    vb[j] = 16 * j + r < cols ? static_cast<uint32_t>(16 * j + r) * k + g * 16 : F8_OUT;
  const int last = (KT - 1) * F8_BK + g * 16;
  const uint32_t tail0 = last < k ? 0u : F8_OUT, tail1 = last + 64 < k ? 0u : F8_OUT;

  struct Slot {
    u32x4 a[FM][2], b[FN][2];
    float s[FM];
  } slot[P];
  // step kt >= KT loads zeros, its scales among them
  auto load = [&](Slot& q, int kt) {
    const uint32_t so = __builtin_amdgcn_readfirstlane(min(kt, KT - 1) * F8_BK);
    const uint32_t all = kt < KT ? 0u : F8_OUT;
    const uint32_t d0 = kt == KT - 1 ? tail0 : all, d1 = kt == KT - 1 ? tail1 : all;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      q.b[j][0] = buf_ld128(br, vb[j] | d0, so);
      q.b[j][1] = buf_ld128(br, (vb[j] + 64) | d1, so);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      q.a[i][0] = buf_ld128(ar, va[i] | d0, so);
      q.a[i][1] = buf_ld128(ar, (va[i] + 64) | d1, so);
      q.s[i] = __uint_as_float(buf_ld32(sar, vs[i] | all, so / (F8_BK / 4)));
    }
  };
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  using Frag = F8Frag<sizeof(OutT) == 4>;
  auto frag = [](const u32x4& x, const u32x4& y) {
    return Frag(i32x8{(int)x[0], (int)x[1], (int)x[2], (int)x[3],
                      (int)y[0], (int)y[1], (int)y[2], (int)y[3]});
  };
  float sbv = 0.f;  // b's scales of this wavefront's next 64 steps, a lane each
  auto add = [&](const Slot& q, int it) {
    const float sb = __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sbv), it & 63));
    Frag fb[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j] = frag(q.b[j][0], q.b[j][1]);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const Frag fa = frag(q.a[i][0], q.a[i][1]);
      const float f = q.s[i] * sb;
      f32x4 d[FN];
      if constexpr (sizeof(OutT) == 4) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            d[j] = f8_quarter(fb[j], fa, c, c ? d[j] : f32x4{0.f, 0.f, 0.f, 0.f});
      } else {
#pragma unroll
        for (int j = 0; j < FN; ++j) d[j] = f8_block(fb[j], fa);
      }
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][j][c] = __builtin_fmaf(d[j][c], f, acc[i][j][c]);
    }
  };
#pragma unroll
  for (int u = 0; u < P; ++u) {
    load(slot[u], wave + NW * u);
    __builtin_amdgcn_sched_barrier(0);  // slots in order: the loop's waits stay exact
  }
  const int IT = (KT + NW - 1) / NW;
  static_assert(64 % P == 0, "the scale register is refilled between rounds");
  for (int it = 0; it < IT; it += P) {
    if ((it & 63) == 0) {
      const int kt = wave + NW * (it + lane);
      sbv = kt < KT ? sbp[kt] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < P; ++u) {
      add(slot[u], it + u);
      load(slot[u], wave + NW * (it + u + P));
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) red[((wave * FM + i) * FN + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  constexpr int ES = sizeof(OutT);
  const __amdgpu_buffer_rsrc_t orsrc =
      buf_rsrc(static_cast<OutT*>(p.out) + static_cast<long>(t.m0) * n,
               static_cast<uint32_t>(t.rows) * n * ES);
  for (int q = tid; q < FM * FN * 64; q += 64 * NW) {
    f32x4 v = red[q];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += red[w * FM * FN * 64 + q];
    // quad q: block (i, j) = q / 64, row 16 i + q % 16, columns 16 j + 4 ((q % 64) / 16) ..
    const int i = q / (64 * FN), j = (q / 64) % FN;
    const int row = 16 * i + (q & 15), col = 16 * j + 4 * ((q & 63) >> 4);
    f8_store4<OutT>(orsrc, row < t.rows && col < cols
                               ? (static_cast<uint32_t>(row) * n + t.n0 + col) * ES : F8_OUT, v);
  }
}

// An upper bound on the tiles: a group's last one may be partial, and there are
// no more such groups than rows.  Then 8 for every round of chunks of cm tiles.
mi_status f8_grid(const F8Args& p, int bm, int bn, long cm, int threads, const char* what,
                  dim3* grid) {
  long tiles = (static_cast<long>(p.m_rows) + bm - 1) / bm;
  if (p.m_indptr != nullptr) tiles += p.E < p.m_rows ? p.E : p.m_rows;
  tiles *= (p.n + bn - 1) / bn;
  const long g = (tiles + 7) / 8 * 8 + 8 * ((tiles + 8 * cm - 1) / (8 * cm));
  MI_REQUIRE(g * threads < (1L << 32), "%s: more tiles than one launch takes", what);
  *grid = dim3(static_cast<unsigned>(g));
  return MI_OK;
}

// Whether groups of one m-tile stream b: its panels are read once, and where all of b
// is large the next call would hardly find them in the 256 MB memory-side cache.
// Then b is loaded with the non-temporal policy, and with k a multiple of 4096 every
// panel has its own first step (us; n 2048, 64 experts of 16 rows: k 4096 neither 129,
// non-temporal 120, both 85; k 2560, 335 MB, 61 and 55; k 2048, 268 MB, which the next
// call of a loop partly finds again, 43 and 45; 128 experts of 15 MB, very unequal: 682
// and 679, with groups of several m-tiles streamed too 708).  Panels found in the cache
// lose (16 experts of 1 MB 9.5 and 11.5).
bool f8_stream_b(const F8Args& p) {
  return p.m_indptr != nullptr && static_cast<int64_t>(p.E) * p.n * p.k >= (128LL << 20);
}

#define F8_LAUNCH(KERNEL_, BM_, BN_, CM_, THREADS_)                      \
  do {                                                                 \
    dim3 grid;                                                         \
    const mi_status st = f8_grid(p, BM_, BN_, CM_, THREADS_, what, &grid); \
    if (st != MI_OK) return st;                                        \
    hipLaunchKernelGGL((KERNEL_), grid, dim3(THREADS_), 0, stream, p); \
    return launch_status(what);                                        \
  } while (0)

template <int WM, int WN, int FM, int FN, int NST, typename OutT>
mi_status f8_launch(const F8Args& p, hipStream_t stream, const char* what) {
  if (f8_stream_b(p))
    F8_LAUNCH((f8_mm_kernel<WM, WN, FM, FN, NST, true, OutT>), 16 * FM * WM, 16 * FN * WN, 64,
              64 * WM * WN);
  F8_LAUNCH((f8_mm_kernel<WM, WN, FM, FN, NST, false, OutT>), 16 * FM * WM, 16 * FN * WN, 64,
            64 * WM * WN);
}

template <typename OutT>
mi_status f8_launch_large(const F8Args& p, hipStream_t stream, const char* what) {
  if (f8_stream_b(p)) F8_LAUNCH((f8_mm_large_kernel<true, OutT>), 256, 256, 32, 512);
  F8_LAUNCH((f8_mm_large_kernel<false, OutT>), 256, 256, 32, 512);
}

template <int FM, int FN, int NW, int P, typename OutT>
mi_status f8_launch_few(const F8Args& p, hipStream_t stream, const char* what) {
  F8_LAUNCH((f8_mm_few_kernel<FM, FN, NW, P, OutT>), 16 * FM, 16 * FN, 1L << 26, 64 * NW);
}
#undef F8_LAUNCH

template <typename OutT>
mi_status f8_dispatch(const F8Args& p, hipStream_t s, const char* what) {
  // By the sizes the host knows: of groups' rows only their average.  Times in us,
  // of dense products at n = k = 8192 unless said otherwise.
  const bool grouped = p.m_indptr != nullptr;
  const long E = p.E, rows = (p.m_rows + E - 1) / E, n = p.n;
  auto tiles = [&](long bm, long bn) { return (rows + bm - 1) / bm * ((n + bn - 1) / bn); };
  const long active = E < p.m_rows ? E : p.m_rows;  // groups that have rows, at most
  // Few rows.  Dense: as long as the tiles run in one round, or where no other tile
  // would read b less often (m 16: 15.2 against 17.3 for 64 x 64 tiles; m 24, two
  // rounds: 27.6 against 17.3).  Groups: up to 10 rows, beyond which some have two
  // tiles of 16 and b is read twice (8 experts, n 1024, k 4096: 10 rows 9.0 against
  // 10.5, 12 rows 15.7), in one round (n 2048, k 2048: two rounds, 2 rows 8.5 against
  // 7.7) or two where a group has one row or the MFMAs are the slower ones of fp32
  // outputs (64 experts, n 2048, k 4096: 8 rows in all 12.7 against 16.3, 16 rows 26.8
  // against 21.9).  16 columns per workgroup while that is one round, 32 leave CUs
  // idle there (m 1, n = k = 4096: 5.3 against 6.9; m 4, n = k = 8192: 14.4 against
  // 12.2).  Eight wavefronts with a step each in flight: more of them, or more steps,
  // hold more lines than they gain (m 4: four with two steps 13.1, eight with two 13.1,
  // sixteen with one 13.5).
  if (grouped ? rows <= 10 && active * ((n + 15) / 16) <= 256 : tiles(16, 16) <= 256)
    return f8_launch_few<1, 1, 8, 1, OutT>(p, s, what);
  const long at_most = rows <= 1 || sizeof(OutT) == 4 ? 512 : 256;
  if (grouped ? rows <= 10 && active * ((n + 31) / 32) <= at_most
              : rows <= 16 || tiles(16, 32) <= 256)
    return f8_launch_few<1, 2, 8, 1, OutT>(p, s, what);
  // 64 x 64 tiles with four stages.  Dense: while they run in one round of two
  // workgroups per CU (m 256: 31 against 42 for 128 x 128; m 384: 47 against 43).
  // Groups of up to 48 rows: where the 128 x 128 tiles leave a first or second round
  // of 512 at most half full (8 experts, n = k = 4096, 16 rows: 23 against 31; n 2048,
  // k 4096, 48 experts of 12 and 48 rows 65 and 75 against 72 and 76, 32 of 16 rows 44
  // against 40, 64 of 16 rows 89 against 85).  In a third round it is no rule: 80 experts
  // of 16 rows 115 against 122, of 48 rows 129 against 126; 72 of 40 rows 119 against 117.
  const long panels = active * ((n + 127) / 128);
  if (grouped ? rows <= 48 && (panels <= 256 || (panels > 512 && panels <= 768))
              : tiles(64, 64) <= 512)
    return f8_launch<2, 2, 2, 2, 4, OutT>(p, s, what);
  if constexpr (sizeof(OutT) == 2) {
    // 256 x 256 tiles have the fewest bytes per MFMA, but one runs per CU, not two.
    // They are taken where the 128 x 128 tiles need more than one round (n = k = 4096:
    // m 2048, one round of 512, 44 against 35, m 2304 44 against 53; 16 groups of 192
    // rows 70 against 91; where very unequal groups fill a second round of the large
    // tiles they lose: 12 of 256 rows on average, k 2048, 55 against 45).  A group has
    // half a tile more than its rows fill.  Below 56 rows the 128-row tiles are better
    // (64 experts, n 2048, k 4096: 80 rows 97 against 99, 48 rows 89 against 87).
    const long m_tiles = grouped ? E * (2 * rows + 128) / 256 : (rows + 127) / 128;
    if (rows >= 56 && m_tiles * ((n + 127) / 128) > 512)
      return f8_launch_large<OutT>(p, s, what);
  }
  // fp32 outputs stay here: fp16 fragments of a 256-row tile would not fit the
  // registers (m 4096: 436; with 128 x 64 tiles 569)
  return f8_launch<2, 2, 4, 4, 2, OutT>(p, s, what);
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
  const int64_t sc = mi_fp8_scale_cols(k) * 4, ob = m_rows * n * (out_dtype == MI_F32 ? 4 : 2);
  MI_REQUIRE(!overlap(p.out, ob, p.a, m_rows * k) && !overlap(p.out, ob, p.sa, m_rows * sc) &&
                 !overlap(p.out, ob, p.b, batch * n * k) &&
                 !overlap(p.out, ob, p.sb, batch * ((n + 127) / 128) * sc) &&
                 !overlap(p.out, ob, p.m_indptr, (batch + 1) * 4),
             "%s: out may not overlap an input", what);
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
                                             const int32_t* m_indptr, int zero_outside,
                                             void* out, mi_dtype out_dtype, void* stream) {
  using namespace mi;
  clear_error();
  MI_REQUIRE(m_indptr != nullptr, "grouped_mm_fp8_block: m_indptr is null");
  F8Args p{};
  p.a = a;
  p.sa = a_scale;
  p.b = b;
  p.sb = b_scale;
  p.m_indptr = m_indptr;
  p.zero_outside = zero_outside != 0;
  p.out = out;
  return f8_run(p, m_rows, k, n, batch, out_dtype, stream, "grouped_mm_fp8_block");
}
