// Grouped product on MXFP4 weights (moe_mxfp4_product): c[r] = a[row(r)] b[e]^T
// for the rows r of expert e, with a in MXFP4 or MXFP8, on the block-scaled
// matrix instruction v_mfma_scale_f32_16x16x128_f8f6f4 (its two operands have
// formats of their own), fp32 sums.
//
// Lane l of an operand fragment (16 rows x 128 of K) holds row l % 16; with g =
// l / 16, of MXFP4 codes the 16 bytes of K block g, of MXFP8 codes bytes 16g ..
// and 64 + 16g .. of the step, and the scale byte of K block g (checked on
// the device against exact products; MXFP4 x MXFP4 sums came out exact, a scale
// byte 255 gives NaN).  The weights are the first operand, so a lane's result
// is 4 consecutive columns of one row.
#include "gemm_common.h"
#include "row_vec.h"

#include <algorithm>

namespace moe {
namespace {

using gg::OOB;
using gg::make_rsrc;
using gg::u32x4_t;
typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));

constexpr int KSTEP = 128;   // K of one scaled MFMA
constexpr int FMT_FP8 = 0, FMT_FP4 = 4;   // format fields of the instruction

// Row tile i (of 16 rows, counted over the experts in order) -> expert and rows
// [m0, mlim).  Every wave finds it by itself: lane l counts the tiles of experts
// l*per .. of the offsets, a prefix sum over the lanes and a ballot give the
// lane that holds tile i, and that lane's registers the rest.  The offsets are
// loaded all at once; this takes about 1 us and saves the launch that would
// build a table.  Offsets are cut to [0, rows] so that no index leaves c.
// False when i is no tile.
__device__ __forceinline__ bool find_tile(const Mx4Args& a, int lane, int i, int& e, int& m0, int& mlim) {
  constexpr int BM = 16;
  if (a.offsets == nullptr) {
    if (i >= (a.rows + BM - 1) / BM) return false;
    e = 0;
    m0 = i * BM;
    mlim = a.rows;
    return true;
  }
  constexpr int PER = 8;             // experts a lane at most
  const int per = (a.E + 63) / 64, e0 = lane * per;
  int o[PER + 1], cnt[PER], sum = 0;
#pragma unroll
  for (int q = 0; q <= PER; ++q) {
    o[q] = 0;
    if (q <= per) o[q] = a.offsets[min(e0 + q, a.E)];
  }
#pragma unroll
  for (int q = 0; q <= PER; ++q) o[q] = min(max(o[q], 0), a.rows);
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    cnt[q] = q < per ? max(0, o[q + 1] - o[q] + BM - 1) / BM : 0;
    sum += cnt[q];
  }
  int inc = sum;   // inclusive prefix sum over the lanes: within rows of 16, then over the rows
  inc += __builtin_amdgcn_update_dpp(0, inc, 0x111, 0xF, 0xF, false);   // row_shr 1, 2, 4, 8
  inc += __builtin_amdgcn_update_dpp(0, inc, 0x112, 0xF, 0xF, false);
  inc += __builtin_amdgcn_update_dpp(0, inc, 0x114, 0xF, 0xF, false);
  inc += __builtin_amdgcn_update_dpp(0, inc, 0x118, 0xF, 0xF, false);
  inc += __builtin_amdgcn_update_dpp(0, inc, 0x142, 0xA, 0xF, false);   // row_bcast 15 into rows 1 and 3
  inc += __builtin_amdgcn_update_dpp(0, inc, 0x143, 0xC, 0xF, false);   // row_bcast 31 into rows 2 and 3
  const uint64_t hit = __ballot(inc > i);
  if (hit == 0) return false;
  const int src = __builtin_ctzll(hit);
  int local = i - __builtin_amdgcn_readlane(inc - sum, src);
  int q = 0, first = __builtin_amdgcn_readlane(o[0], src), last = __builtin_amdgcn_readlane(o[1], src);
#pragma unroll
  for (int u = 0; u < PER - 1; ++u) {
    const int c = __builtin_amdgcn_readlane(cnt[u], src);
    if (q == u && local >= c) {
      local -= c;
      q = u + 1;
      first = __builtin_amdgcn_readlane(o[u + 1], src);
      last = __builtin_amdgcn_readlane(o[u + 2], src);
    }
  }
  e = src * per + q;
  m0 = first + local * BM;
  mlim = last;
  return true;
}

// f / row_div by the multiplier and shift the host chose (f < 2^31; exact)
__device__ __forceinline__ int div_by(uint32_t f, uint32_t mul, int shift) { return (int)(((uint64_t)f * mul) >> shift); }

// A's row for entry f of the row map (for row f of c without one), or -1 (reads as zeros)
__device__ __forceinline__ int a_row(const Mx4Args& a, int f) {
  const int s = a.row_map == nullptr ? f : f < 0 ? -1 : div_by((uint32_t)f, a.div_mul, a.div_shift);
  return (uint32_t)s < (uint32_t)a.a_rows ? s : -1;
}

// 4 consecutive columns n .. of one row of c
__device__ __forceinline__ void store4(const Mx4Args& a, int m, int n, f32x4_t v) {
  const int64_t at = (int64_t)m * a.ldc + n;
  const int cnt = min(4, a.N - n);
  if (a.c_bf16) {
    bf16_t* p = static_cast<bf16_t*>(a.c) + at;
    if (cnt == 4) {
      typedef uint32_t u32x2u_t __attribute__((ext_vector_type(2), aligned(2)));
      *reinterpret_cast<u32x2u_t*>(p) = u32x2u_t{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
    } else {
      for (int i = 0; i < cnt; ++i) p[i] = cvt_bf16(v[i]);
    }
  } else {
    float* p = static_cast<float*>(a.c) + at;
    if (cnt == 4) {
      typedef float f32x4u_t __attribute__((ext_vector_type(4), aligned(4)));
      *reinterpret_cast<f32x4u_t*>(p) = f32x4u_t{v[0], v[1], v[2], v[3]};
    } else {
      for (int i = 0; i < cnt; ++i) p[i] = v[i];
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows per expert: the weights go straight into registers (each byte has
// one reader, so LDS would only add a stop).  A block takes 16 rows and CF x 16
// columns; its four waves split K, so that even one expert's weights are read
// by many waves, and their sums are added in wave order through LDS.
// SC4: KB % 4 == 0, a K step's four scale bytes of a row are one aligned word.
//
// Bound by the latency of what a wave reads one after the other (offsets, row
// map, operands) and by HBM: 32 rows on as many experts' 1536 x 2048, 50 MB:
// 13.4 us, of which launching takes 2.
// ---------------------------------------------------------------------------
template <bool FP8, bool SC4, int CF>
__global__ __launch_bounds__(256) void mx4_stream_kernel(Mx4Args a, int n_groups) {
  constexpr int NW = 4;
  // K steps whose loads are in flight together; of a short K more would be steps that are not there (64 tokens at 2048
  // x 768: 12.2 us with 4, 10.4 with 2)
  constexpr int U = CF == 4 ? 2 : 4;
  __shared__ f32x4_t s_acc[NW][CF][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, rl = lane & 15;
  const int tile = blockIdx.x / n_groups, n0 = blockIdx.x % n_groups * (16 * CF);
  int e, m0, mlim;
  if (!find_tile(a, lane, tile, e, m0, mlim)) return;
  const uint32_t pb = (uint32_t)a.KB * 16, pa = FP8 ? (uint32_t)a.K : pb;   // code bytes of a row
  const auto rb = make_rsrc(a.b + (size_t)e * a.N * pb, (uint32_t)a.N * pb);
  const auto rsb = make_rsrc(a.sb + (size_t)e * a.N * a.KB, (uint32_t)a.N * a.KB);
  const auto ra = make_rsrc(a.a, (uint32_t)a.a_rows * pa);
  const auto rsa = make_rsrc(a.sa, (uint32_t)a.a_rows * a.KB);
  const int m = m0 + rl;
  const int entry = m >= mlim ? -1 : a.row_map ? a.row_map[m] : m;   // (used below the weights' loads: they go first)
  f32x4_t acc[CF];
#pragma unroll
  for (int c = 0; c < CF; ++c) acc[c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int nk = (a.K + KSTEP - 1) / KSTEP;
  const int per = (nk + NW - 1) / NW;
  const int k0 = wave * per, k1 = min(nk, k0 + per);
  auto scale = [&](__amdgpu_buffer_rsrc_t r, uint32_t row, bool ok, int kt) -> int {
    if constexpr (SC4) return __builtin_amdgcn_raw_buffer_load_b32(r, ok ? row + 4 * kt : OOB, 0, 0);
    else return __builtin_amdgcn_raw_buffer_load_b8(r, ok && 4 * kt + g < a.KB ? row + 4 * kt + g : OOB, 0, 0);
  };
  for (int kt0 = k0; kt0 < k1; kt0 += U) {
    u32x4_t cb[CF][U], ca[U], cah[U];
    int sb[CF][U], sa[U];
#pragma unroll
    for (int c = 0; c < CF; ++c) {
      const int n = n0 + 16 * c + rl;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int kt = kt0 + u;
        const uint32_t kb = (uint32_t)kt * 64 + 16 * g;
        const bool in = kt < k1 && n < a.N;
        cb[c][u] = __builtin_amdgcn_raw_buffer_load_b128(rb, in && kb < pb ? (uint32_t)n * pb + kb : OOB, 0, 0);
        sb[c][u] = scale(rsb, (uint32_t)n * a.KB, in, kt);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    const int row = entry < 0 ? -1 : a_row(a, entry);
    const bool mok = row >= 0;
    const uint32_t oa = mok ? (uint32_t)row * pa : 0, osa = mok ? (uint32_t)row * a.KB : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kt = kt0 + u;
      const bool in = kt < k1;
      const uint32_t ka = (uint32_t)kt * (FP8 ? 128 : 64) + 16 * g;
      ca[u] = __builtin_amdgcn_raw_buffer_load_b128(ra, in && mok && ka < pa ? oa + ka : OOB, 0, 0);
      if constexpr (FP8)
        cah[u] = __builtin_amdgcn_raw_buffer_load_b128(ra, in && mok && ka + 64 < pa ? oa + ka + 64 : OOB, 0, 0);
      else
        cah[u] = u32x4_t{0u, 0u, 0u, 0u};
      sa[u] = scale(rsa, osa, in && mok, kt);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const i32x8_t fa = {(int)ca[u][0], (int)ca[u][1], (int)ca[u][2], (int)ca[u][3],
                          (int)cah[u][0], (int)cah[u][1], (int)cah[u][2], (int)cah[u][3]};
      const int xa = SC4 ? (int)((uint32_t)sa[u] >> (8 * g)) : sa[u];
#pragma unroll
      for (int c = 0; c < CF; ++c) {
        const i32x8_t fb = {(int)cb[c][u][0], (int)cb[c][u][1], (int)cb[c][u][2], (int)cb[c][u][3], 0, 0, 0, 0};
        const int xb = SC4 ? (int)((uint32_t)sb[c][u] >> (8 * g)) : sb[c][u];
        acc[c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, fa, acc[c], FMT_FP4, FP8 ? FMT_FP8 : FMT_FP4, 0,
                                                                  xb, 0, xa);
      }
    }
  }
  static_assert(CF <= NW, "a wave for the sums of each fragment");
#pragma unroll
  for (int c = 0; c < CF; ++c) s_acc[wave][c][lane] = acc[c];
  __syncthreads();
  if (wave >= CF) return;
  f32x4_t sum = s_acc[0][wave][lane];
#pragma unroll
  for (int w = 1; w < NW; ++w) sum += s_acc[w][wave][lane];
  const int n = n0 + 16 * wave + 4 * g;
  if (m < mlim && n < a.N) store4(a, m, n, sum);
}

// ---------------------------------------------------------------------------
// Many rows per expert: BM x BN tiles, operands through LDS, resident blocks
// that walk over the tiles.
//
// K advances by stages of KST (256 with MXFP4 rows, 128 with MXFP8: either way
// 128 bytes, a whole line, per row of A).  Two stages of LDS: while one is
// multiplied, the other receives the next by buffer-to-LDS DMA (16 bytes a
// lane; lanes outside a row, its K or the tile read zeros through an
// out-of-range offset).  Code rows are cut in 16-byte chunks, XOR-swizzled
// within 128 bytes, so that a fragment's 64 chunks cover every bank equally;
// with MXFP8 rows, B's 64-byte rows lie in pairs.
//
// A unit is one MFMA step of K (SS of them per stage): FM rows of FN products a
// wave.  Its fragments are read ahead: A's three rows before their use (ring of
// four), B's during the unit before (two sets).  Row PB of a stage's last unit,
// where the wave's last read of the stage has been issued, is the stage's only
// barrier: it publishes the next stage and frees this one, into which the DMA
// of the stage after the next then runs, DPR instructions a row.  All of it
// goes between the products, one instruction or two after each.  The stages of
// consecutive tiles follow each other without a gap: the next tile's operands
// arrive while this one's last products run and its results leave, through a
// piece of LDS of each wave's own, no barrier, in whole lines (stores of 64
// bytes of a row cost 14%) and past the caches (nothing here reads them again;
// 310 -> 294 us).
//
// Scales: the words of a row's four K blocks come by DMA too, one K step of 64
// rows an instruction.  A lane reads one word for four fragments and gets its
// byte of each by a 4 x 4 transpose over four lanes; the instruction's byte
// select picks it.  Where K is not a multiple of 128 the words are not aligned,
// and they pass through registers.  (16 bytes of a row at a time, four K steps,
// are a quarter of the requests, but LDS then has no room for the output's
// lines: as fast at best.)
//
// 131072 rows of 128 experts, 1536 x 2048: 275 us, 3.0 PFLOP/s (MXFP8 390); one
// 4096 x 4096 weight, 16384 rows: 147 us, 3.7 PFLOP/s.  With 4 waves of 128 x
// 128 in place of 8 of 128 x 64: 290 and 153; a block per tile and two barriers
// a stage: 339 and 171.  What bounds it, in parts of the second: the products
// alone 70 us (the clock falls to 1.9 GHz), the DMA alone 114, of which the
// scales, 4 bytes of a line each, are 26; without output 143.
// ---------------------------------------------------------------------------
template <int N, class F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl<N>(f, std::make_integer_sequence<int, N>{});
}

// The stage's code has no branch that the compiler sees: across blocks it moves products away from their operands'
// reads and runs out of registers.  What depends on the stage branches inside asm statements.  With one wave on a
// SIMD every instruction beside the products counts (an MXFP4 product leaves room for three), so they are few: the
// K offset of a DMA goes through the instruction's scalar offset.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// DMA of W bytes a lane into lds0 + LDS (off outside the buffer: zeros), if go != 0
template <int W, int LDS>
__device__ __forceinline__ void dma_if(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t k, uint32_t lds0, int go) {
  if constexpr (W == 16)
    asm volatile("s_cmp_eq_u32 %4, 0\n\ts_cbranch_scc1 .Lnodma%=\n\ts_add_u32 m0, %3, %5\n\t"
                 "buffer_load_dwordx4 %0, %1, %2 offen lds\n.Lnodma%=:"
                 :: "v"(off), "s"(r), "s"(k), "s"(lds0), "s"(go), "n"(LDS) : "memory", "m0", "scc");
  else
    asm volatile("s_cmp_eq_u32 %4, 0\n\ts_cbranch_scc1 .Lnodma%=\n\ts_add_u32 m0, %3, %5\n\t"
                 "buffer_load_dword %0, %1, %2 offen lds\n.Lnodma%=:"
                 :: "v"(off), "s"(r), "s"(k), "s"(lds0), "s"(go), "n"(LDS) : "memory", "m0", "scc");
}
template <int W, int LDS>
__device__ __forceinline__ void dma_to(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t k, uint32_t lds0) {
  if constexpr (W == 16)
    asm volatile("s_add_u32 m0, %3, %4\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :: "v"(off), "s"(r), "s"(k), "s"(lds0), "n"(LDS) : "memory", "m0", "scc");
  else
    asm volatile("s_add_u32 m0, %3, %4\n\tbuffer_load_dword %0, %1, %2 offen lds"
                 :: "v"(off), "s"(r), "s"(k), "s"(lds0), "n"(LDS) : "memory", "m0", "scc");
}
#pragma clang diagnostic pop
// d = s in place if left == 0, four or one at a time
__device__ __forceinline__ void move4_if(uint32_t* d, const uint32_t* s, int left) {
  asm("s_cmp_lg_u32 %8, 0\n\ts_cbranch_scc1 .Lnomove%=\n\tv_mov_b32 %0, %4\n\tv_mov_b32 %1, %5\n\tv_mov_b32 %2, %6\n\t"
      "v_mov_b32 %3, %7\n.Lnomove%=:"
      : "+v"(d[0]), "+v"(d[1]), "+v"(d[2]), "+v"(d[3]) : "v"(s[0]), "v"(s[1]), "v"(s[2]), "v"(s[3]), "s"(left) : "scc");
}
template <int N>
__device__ __forceinline__ void move_if(uint32_t (&d)[N], const uint32_t (&s)[N], int left) {
#pragma unroll
  for (int i = 0; i + 4 <= N; i += 4) move4_if(d + i, s + i, left);
#pragma unroll
  for (int i = N / 4 * 4; i < N; ++i) d[i] = left == 0 ? s[i] : d[i];
}
// the wait for all vector memory operations, or when kt == 0 for all but the youngest N
template <int N>
__device__ __forceinline__ void vm_wait_if(int kt) {
  asm volatile("s_cmp_eq_u32 %0, 0\n\ts_cbranch_scc1 .Lsome%=\n\ts_waitcnt vmcnt(0)\n.Lsome%=:\n\ts_waitcnt vmcnt(%1)"
               :: "s"(kt), "n"(N) : "memory", "scc");
}

template <bool FP8_, bool SC4_, int BM_, int BN_, int WGM_, int WGN_, int PER_CU_>
struct Mx4Cfg {
  static constexpr bool FP8 = FP8_, SC4 = SC4_;
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_;
  static constexpr int PER_CU = PER_CU_;                 // resident blocks per compute unit
  static constexpr int NW = WGM * WGN, NTHR = 64 * NW;
  static constexpr int WPE = PER_CU * NW / 4;            // waves per SIMD
  static constexpr int WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
  static constexpr int KST = FP8 ? 128 : 256;            // K per stage
  static constexpr int SS = KST / KSTEP;                 // units per stage
  static constexpr int RA = 128, RB = KST / 2;           // code bytes per row and stage
  static constexpr int SB = KST / 32;                    // scale bytes per row and stage
  static constexpr int A_BYTES = BM * RA, B_BYTES = BN * RB;
  static constexpr int DA = A_BYTES / 1024 / NW, DB = B_BYTES / 1024 / NW;   // 1 KiB DMAs per wave and stage
  static constexpr int A_SC = A_BYTES + B_BYTES, B_SC = A_SC + BM * SB;
  static constexpr int STAGE = B_SC + BN * SB;
  static constexpr int SR = (BM + BN) / NTHR;            // scale rows per thread; groups of 64 of them per wave
  static constexpr int DS = SC4 ? SR * SS : 0;           // 256-byte DMAs of scales per wave and stage
  static constexpr int D = DA + DB + DS;
  static constexpr int PB = FM - 3;                      // row of the barrier
  static constexpr int DPR = NW == 8 ? 2 : 3;                // DMAs per row of products
  static constexpr int D_TAIL = (FM - PB) * DPR;         // DMAs of a stage issued before the next one begins
  static constexpr int PB_FIRST = SS == 1 ? PB - 1 : FM; // rows of a stage's first unit that may issue the others
  static constexpr int OUT_ROW = WN * 2, OUT_WAVE = 16 * OUT_ROW;   // bytes of a wave's output in LDS: 16 rows
  // stores of a whole tile by a wave: 16 bytes a lane, twice as many of fp32 (which bf16's number waits for too)
  static constexpr int OUT_STORES = WM * WN * 2 / 1024;
  static constexpr int TILES = 64;                       // tiles listed at a time
  static constexpr int OUT0 = 2 * STAGE, LIST0 = OUT0 + NW * OUT_WAVE, ROWS0 = LIST0 + TILES * 16;
  static constexpr int MAP0 = ROWS0 + 2 * BM * 4;
  static constexpr int LDS = MAP0 + BM * 4;
  static_assert(DA * NW * 1024 == A_BYTES && DB * NW * 1024 == B_BYTES, "whole DMAs per wave");
  static_assert(SR * NTHR == BM + BN && BM == BN && SR <= 2, "scale rows: one of each operand per thread, or of one");
  static_assert(FM % 4 == 0 && FN % 4 == 0, "whole words of scales per lane");
  static_assert(PB >= 1, "ring of four A fragments");
  static_assert(D - D_TAIL <= PB_FIRST * DPR, "the other DMAs fit before the next barrier");
  static_assert(NW * OUT_WAVE >= 1025 * 4, "the prefix sums and first rows fit where the output is staged");
  static_assert(LDS * PER_CU <= 160 * 1024, "LDS of a compute unit");
};

template <class C>
__global__ __launch_bounds__(C::NTHR) __attribute__((amdgpu_waves_per_eu(C::WPE, C::WPE)))
void mx4_tile_kernel(Mx4Args a, int n_tiles) {
  constexpr int BM = C::BM, BN = C::BN, WM = C::WM, WN = C::WN, FM = C::FM, FN = C::FN, NW = C::NW, SS = C::SS;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WGN, wn = wave % C::WGN;
  const int g = lane >> 4, rl = lane & 15;

  // ---------------- this block's tiles: (expert, first row, row limit, column tile), TILES at a time in LDS.
  // Block b runs on XCD b % 8; each XCD takes a contiguous run of the tiles (column tiles fastest), its blocks
  // deal them out in turn, so that those sharing an expert's rows and weights meet in one L2.  The tiles are
  // counted from the offsets, cut to [0, rows] so that no index leaves c.
  int4* const s_list = reinterpret_cast<int4*>(smem + C::LIST0);
  int* const s_pre = reinterpret_cast<int*>(smem + C::OUT0);   // tiles of the experts up to each one
  int* const s_first = s_pre + 512;                            // their first rows, and the last one's end
  auto row_at = [&](int e) { return min(max(a.offsets[e], 0), a.rows); };
  auto list_tiles = [&](int it0) {
    int total;
    __syncthreads();
    if (a.offsets) {
      for (int e = tid; e < 512; e += C::NTHR) {
        int n = 0;
        if (e < a.E) {
          const int first = row_at(e), end = row_at(e + 1);
          n = max(0, end - first + BM - 1) / BM;
          s_first[e] = first;
          if (e == a.E - 1) s_first[a.E] = end;
        }
        s_pre[e] = n;
      }
      __syncthreads();
      if (wave == 0) {   // inclusive prefix sums, 8 experts a lane
        int v[8], sum = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) { sum += s_pre[lane * 8 + q]; v[q] = sum; }
        int inc = sum;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
          const int u = __shfl_up(inc, off);
          if (lane >= off) inc += u;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) s_pre[lane * 8 + q] = v[q] + inc - sum;
      }
      __syncthreads();
      total = s_pre[a.E - 1];
    } else {
      total = (a.rows + BM - 1) / BM;
    }
    const int64_t tiles = (int64_t)total * n_tiles;
    const int64_t per_xcd = (tiles + gg::NXCD - 1) / gg::NXCD;
    const int x = blockIdx.x % gg::NXCD, slot = blockIdx.x / gg::NXCD, slots = gridDim.x / gg::NXCD;
    if (tid < C::TILES) {
      const int64_t j = slot + (int64_t)(it0 + tid) * slots, L = x * per_xcd + j;
      int4 t = make_int4(-1, 0, 0, 0);
      if (j < per_xcd && L < tiles) {
        const int i = (int)(L / n_tiles);
        t.w = (int)(L - (int64_t)i * n_tiles);
        if (a.offsets) {
          int lo = 0, hi = a.E - 1;             // first expert whose prefix passes i
          while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_pre[mid] > i) hi = mid; else lo = mid + 1;
          }
          t.x = lo;
          t.y = s_first[lo] + (i - (lo > 0 ? s_pre[lo - 1] : 0)) * BM;
          t.z = s_first[lo + 1];
        } else {
          t.x = 0;
          t.y = i * BM;
          t.z = a.rows;
        }
      }
      s_list[tid] = t;
    }
    __syncthreads();
  };
  struct Tile { int e, m0, mlim, n0; };
  auto tile_at = [&](int it) -> Tile {
    const int4 t = s_list[it % C::TILES];
    return Tile{__builtin_amdgcn_readfirstlane(t.x), __builtin_amdgcn_readfirstlane(t.y),
                __builtin_amdgcn_readfirstlane(t.z), __builtin_amdgcn_readfirstlane(t.w) * BN};
  };

  // ---------------- operands
  const uint32_t pb = (uint32_t)a.KB * 16, pa = C::FP8 ? (uint32_t)a.K : pb;   // code bytes of a row
  const auto ra = make_rsrc(a.a, (uint32_t)a.a_rows * pa);
  const int nk = max(2, (a.K + C::KST - 1) / C::KST);   // at least two: the DMA runs two stages ahead, into the next tile at most
  // DMA i of wave w fills the 1 KiB block ci = i * NW + w of an operand: lane l writes 16 bytes at 16 l
  const int line = lane >> 3, chunk8 = (lane & 7) ^ line;
  const uint32_t cola = 16u * chunk8;                                          // 8 rows of 128 bytes
  const uint32_t colb = C::RB == 128 ? 16u * chunk8 : 16u * (chunk8 & 3);      // or 16 rows of 64
  const int lineb = C::RB == 128 ? line : 2 * line + (chunk8 >> 2);            // row of B within the block
  // scale rows of this thread: rows R < BM are A's, the others B's (the same side for all lanes of a wave)
  using sc_t = std::conditional_t<C::SB == 8, uint64_t, uint32_t>;
  typedef sc_t scu_t __attribute__((aligned(1)));
  const bool upper = wave * 64 >= BM;
  auto sc_is_b = [&](int q) { return C::SR > 1 ? q > 0 : upper; };
  auto sc_r = [&](int q) { return C::SR > 1 || !upper ? tid : tid - BM; };
  const auto rsa = make_rsrc(a.sa, (uint32_t)a.a_rows * a.KB);

  // The tile being loaded (the loads run up to two stages ahead of the products, into the next tile): the byte
  // offsets of its operand rows, OOB for a row outside.  Those of A come from s_rows, which holds two tiles' row
  // offsets: a tile's row_map entries are fetched three tiles ahead, put there two ahead and turned into offsets
  // one ahead.  A scale word holds four K blocks of one row; in LDS they lie in the order (wave row, r, i) of row
  // 16 i + r of the wave's, so that a lane reads those of its FM fragments side by side.
  struct Source {
    const uint8_t *b, *sb;            // the expert's weights and scales
    int64_t sb_room;                  // bytes from there to the scales' end
    uint32_t oa[C::DA], ob[C::DB], os[C::SR];
  };
  uint32_t* const s_rows = reinterpret_cast<uint32_t*>(smem + C::ROWS0);
  auto put_row = [&](const Tile& t, int it, int v) __attribute__((always_inline)) {   // v: the row's row_map entry
    const int s = a.row_map ? div_by((uint32_t)v, a.div_mul, a.div_shift) : t.m0 + tid;
    const bool ok = t.e >= 0 && t.m0 + tid < t.mlim && (v >= 0 || !a.row_map) && s < a.a_rows;
    if (tid < BM) s_rows[(it & 1) * BM + tid] = ok ? (uint32_t)s * pa : OOB;
  };
  auto map_now = [&](const Tile& t) __attribute__((always_inline)) {
    return a.row_map ? a.row_map[min(t.m0 + tid, max(t.mlim - 1, 0))] : 0;
  };
  // the entries of a later tile, to LDS: a register would have to wait for the operands on their way before it
  const int* const s_map = reinterpret_cast<const int*>(smem + C::MAP0);
  auto fetch_map = [&](const Tile& t) __attribute__((always_inline)) {
    if (a.row_map && wave * 64 < BM)
      dma_to<4, C::MAP0>(make_rsrc(a.row_map + t.m0, __builtin_amdgcn_readfirstlane(min(max(t.mlim - t.m0, 0), BM) * 4)), tid * 4, 0,
                         __builtin_amdgcn_readfirstlane((uint32_t)(size_t)(const __attribute__((address_space(3))) void*)smem + wave * 256));
  };
  auto aim = [&](const Tile& t, int it, Source& o) __attribute__((always_inline)) {
    const uint32_t* rows = s_rows + (it & 1) * BM;
    const int64_t e = max(t.e, 0);
    const int n_left = t.e >= 0 ? a.N - t.n0 : 0;        // (no column of a tile behind the last)
    o.b = a.b + e * a.N * pb;
    o.sb = a.sb + e * a.N * a.KB;
    o.sb_room = ((int64_t)a.E - e) * a.N * a.KB;
#pragma unroll
    for (int i = 0; i < C::DA; ++i) {
      const uint32_t r = rows[8 * (i * NW + wave) + line];
      o.oa[i] = r == OOB ? OOB : r + cola;
    }
#pragma unroll
    for (int i = 0; i < C::DB; ++i) {
      const int n = (C::RB == 128 ? 8 : 16) * (i * NW + wave) + lineb;
      o.ob[i] = n < n_left ? (uint32_t)(t.n0 + n) * pb + colb : OOB;
    }
#pragma unroll
    for (int q = 0; q < C::SR; ++q) {                    // this thread's scale rows
      const int R = sc_r(q);
      const uint32_t r = rows[R & (BM - 1)];
      const uint32_t va = r == OOB ? OOB : r >> (C::FP8 ? 5 : 4), vb = R < n_left ? (uint32_t)(t.n0 + R) * a.KB : OOB;
      o.os[q] = sc_is_b(q) ? vb : va;
    }
  };
  Source src, src_n;
  auto take_source = [&](int left) __attribute__((always_inline)) {   // the next tile's if no stage of this one is left
    src.b = left == 0 ? src_n.b : src.b;
    src.sb = left == 0 ? src_n.sb : src.sb;
    src.sb_room = left == 0 ? src_n.sb_room : src.sb_room;
    move_if(src.oa, src_n.oa, left);
    move_if(src.ob, src_n.ob, left);
    move_if(src.os, src_n.os, left);
  };
  const uint32_t lds0 = (uint32_t)(size_t)(const __attribute__((address_space(3))) void*)smem;
  const uint32_t lds16 = __builtin_amdgcn_readfirstlane(lds0 + wave * 1024);   // where this wave's DMAs start
  const uint32_t lds4 = __builtin_amdgcn_readfirstlane(lds0 + (C::SR == 1 && upper ? C::B_SC - C::A_SC : 0) + (64 * wave & (BM - 1)) * 4);
  // DMA instruction i < D of stage kt: A's codes, B's codes, scales; go == 0 (known only then): not now
  int dma_kt = 0;                     // stage that the DMA now fills
  bool in_a = false, in_b = false;    // whether the lane's codes are inside K there
  auto set_dma = [&](int kt) __attribute__((always_inline)) {
    dma_kt = kt;
    in_a = cola + (uint32_t)kt * C::RA < pa;
    in_b = colb + (uint32_t)kt * C::RB < pb;
  };
  auto dma = [&](auto i_, auto sure_, int st, int go) __attribute__((always_inline)) {
    constexpr int i = i_;
    const uint32_t half = st ? C::STAGE : 0;
    auto to = [&](auto w_, auto at_, __amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t k, uint32_t l) __attribute__((always_inline)) {
      if constexpr (sure_) dma_to<w_, at_>(r, off, k, l); else dma_if<w_, at_>(r, off, k, l, go);
    };
    if constexpr (i < C::DA) {
      to(std::integral_constant<int, 16>{}, std::integral_constant<int, i * NW * 1024>{}, ra, in_a ? src.oa[i] : OOB,
         (uint32_t)dma_kt * C::RA, lds16 + half);
    } else if constexpr (i < C::DA + C::DB) {
      constexpr int q = i - C::DA;
      to(std::integral_constant<int, 16>{}, std::integral_constant<int, C::A_BYTES + q * NW * 1024>{},
         make_rsrc(src.b, (uint32_t)a.N * pb), in_b ? src.ob[q] : OOB, (uint32_t)dma_kt * C::RB, lds16 + half);
    } else {
      constexpr int q = (i - C::DA - C::DB) / SS, s = (i - C::DA - C::DB) % SS;           // row group, MFMA step
      const bool b = sc_is_b(q);
      const uint32_t k = (uint32_t)dma_kt * C::SB + 4 * s;
      to(std::integral_constant<int, 4>{}, std::integral_constant<int, (q > 0 ? C::B_SC : C::A_SC) + s * BM * 4>{},
         b ? make_rsrc(src.sb, (uint32_t)a.N * a.KB) : rsa, k < (uint32_t)a.KB ? src.os[q] : OOB, k, lds4 + half);
    }
  };
  // K not a multiple of 128: the words of a row are not aligned, and its scales pass through a register.  SB bytes
  // of a row for stage kt; those past the row's end, and of a row outside, zero.  The last bytes of the array are
  // read from SB before its end and shifted down.
  sc_t sc[C::SR], sc_mask;
  int sc_fix[C::SR];
  auto load_scales = [&](int kt) __attribute__((always_inline)) {
    const int rem = min(max(a.KB - kt * C::SB, 0), C::SB);
    sc_mask = rem == C::SB ? ~(sc_t)0 : ((sc_t)1 << (8 * rem)) - 1;
#pragma unroll
    for (int q = 0; q < C::SR; ++q) {
      const uint32_t row = src.os[q];
      const uint8_t* base = sc_is_b(q) ? src.sb : a.sa;
      const int64_t lim = (sc_is_b(q) ? src.sb_room : (int64_t)a.a_rows * a.KB) - C::SB;
      // (an expert within SB bytes of the array's end reads from before its own scales: lim < 0)
      const int64_t at = (row == OOB ? 0 : (int64_t)row) + (int64_t)kt * C::SB, from = min(at, lim);
      sc[q] = *reinterpret_cast<const scu_t*>(base + from);
      sc_fix[q] = row == OOB ? 64 : (int)min(at - from, (int64_t)8) * 8;
    }
  };
  auto store_scales = [&](int st) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < C::SR; ++q) {
      const bool b = sc_is_b(q);
      const sc_t v = sc_fix[q] >= 8 * C::SB ? (sc_t)0 : (sc[q] >> sc_fix[q]) & sc_mask;
      uint32_t* p = reinterpret_cast<uint32_t*>(smem + st * C::STAGE + (b ? C::B_SC : C::A_SC)) + sc_r(q);
#pragma unroll
      for (int s = 0; s < SS; ++s) p[s * BM] = (uint32_t)(v >> (32 * (s % SS)));
    }
  };

  // ---------------- fragments
  f32x4_t acc[FM][FN];
  u32x4_t ar[4], ar_h[C::FP8 ? 4 : 1], br[2][FN];     // (kept as the four words that MXFP4 codes take)
  uint32_t xa[2][FM / 4], xb[2][FN / 4];              // scales, as many sets: byte i % 4 of word i / 4
  const int sw = rl & 7;                              // rows of a fragment differ from rl by multiples of 16
  auto read_a = [&](int st, int s, int i, int slot) __attribute__((always_inline)) {
    const uint8_t* p = smem + st * C::STAGE + (wm * WM + 16 * i + rl) * 128;
    ar[slot] = *reinterpret_cast<const u32x4_t*>(p + (((C::FP8 ? g : 4 * s + g) ^ sw) << 4));
    if constexpr (C::FP8) ar_h[slot] = *reinterpret_cast<const u32x4_t*>(p + (((4 + g) ^ sw) << 4));
  };
  auto read_b = [&](int st, int s, int j, int set) __attribute__((always_inline)) {
    const int row = wn * WN + 16 * j + rl;
    const uint8_t* p = smem + st * C::STAGE + C::A_BYTES;
    if constexpr (C::RB == 128) br[set][j] = *reinterpret_cast<const u32x4_t*>(p + row * 128 + (((4 * s + g) ^ sw) << 4));
    else br[set][j] = *reinterpret_cast<const u32x4_t*>(p + (row >> 1) * 128 + ((((rl & 1) * 4 + g) ^ ((rl >> 1) & 7)) << 4));
  };
  // Lane (r, g) fetches the word of row 16 g + r, the four K blocks of fragment g, and needs byte g of the four
  // fragments: a 4 x 4 transpose of bytes over the four lanes of r.
  auto read_scales = [&](int st, int s, int set) __attribute__((always_inline)) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(smem + st * C::STAGE + C::A_SC) + s * BM + wm * WM + lane;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(smem + st * C::STAGE + C::B_SC) + s * BN + wn * WN + lane;
#pragma unroll
    for (int i = 0; i < FM / 4; ++i) xa[set][i] = p[64 * i];
#pragma unroll
    for (int j = 0; j < FN / 4; ++j) xb[set][j] = q[64 * j];
  };
  const uint32_t sel_half = g & 2 ? 0x03020706u : 0x01000504u, sel_byte = g & 1 ? 0x03070105u : 0x02060004u;
  auto turn = [&](uint32_t& x) __attribute__((always_inline)) {
    const auto h = __builtin_amdgcn_permlane32_swap(x, x, false, false);        // words of fragments g % 2 and g % 2 + 2
    const uint32_t w = __builtin_amdgcn_perm(h[0], h[1], sel_half);             // their bytes g / 2 * 2 and the next
    const auto q = __builtin_amdgcn_permlane16_swap(w, w, false, false);        // the same of fragments 0, 2 and 1, 3
    x = __builtin_amdgcn_perm(q[0], q[1], sel_byte);
  };

  // ---------------- state of the walk
  int it = 0;                       // tile of the products, its stage, and the LDS half that holds it
  int kt = 0, st = 0;
  list_tiles(0);
  Tile cur = tile_at(0), nxt = tile_at(1), nxt2 = tile_at(2);
  if (cur.e < 0) return;

  // One unit of products: MFMA step s of the stage in half st.
  auto unit = [&](auto s_) __attribute__((always_inline)) {
    constexpr int s = s_;
    constexpr bool LAST = s == SS - 1;              // of the stage
    constexpr int set = SS == 2 ? s : 0, nset = 1 - set;
    static_for<FM>([&](auto i_) {
      constexpr int i = i_;
      if constexpr (LAST && i == C::PB) {
        vm_wait_if<C::OUT_STORES>(kt);              // the next stage's DMA has arrived (in a tile's first stage the last
                                                    // tile's stores, which are younger, may still be under way)
        if constexpr (!C::SC4) store_scales(st ^ 1);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        // this half is free: the stage after the next goes there, the next tile's at the end of this one (zeros
        // behind the last)
        take_source(nk - (kt + 2));
        set_dma(kt + 2 < nk ? kt + 2 : kt + 2 - nk);
        if constexpr (!C::SC4) load_scales(dma_kt);
      }
      // What a row does beside its products goes between them, one thing after each: the row's other instructions
      // would otherwise hold up the matrix core, which has no second wave to turn to.
      constexpr bool head = LAST && i >= C::PB;
      constexpr int at = head ? i - C::PB : s == 0 && i < C::PB_FIRST ? C::D_TAIL / C::DPR + i : -1;
      constexpr int per_b = !LAST ? (FN + FM - 1) / FM : head ? (FN + FM - C::PB - 1) / (FM - C::PB) : 0;
      constexpr int b0 = (!LAST ? i : i - C::PB) * per_b;
      constexpr bool scales = LAST ? i == C::PB : i == 0;
      constexpr bool turns = i == FM - 1;             // the next unit's scales
      constexpr int acts = 1 + per_b + (at >= 0 ? C::DPR : 0) + (scales ? 1 : 0) + (turns ? FM / 4 + FN / 4 : 0);
      auto act = [&](auto n_) __attribute__((always_inline)) {
        constexpr int n = n_;
        constexpr int m = n - (scales ? 1 : turns ? FM / 4 + FN / 4 : 0);
        if constexpr (scales && n == 0) {
          if constexpr (LAST) read_scales(st ^ 1, 0, nset); else read_scales(st, s + 1, nset);
        } else if constexpr (m < 0) {
          if constexpr (n < FN / 4) turn(xb[nset][n]); else turn(xa[nset][n - FN / 4]);
        } else if constexpr (m == 0) {
          if constexpr (i + 3 < FM) read_a(st, s, i + 3, (i + 3) % 4);
          else if constexpr (!LAST) read_a(st, s + 1, i + 3 - FM, (i + 3) % 4);
          else read_a(st ^ 1, 0, i + 3 - FM, (i + 3) % 4);
        } else if constexpr (m <= per_b) {
          constexpr int jb = b0 + m - 1;
          if constexpr (jb < FN) { if constexpr (LAST) read_b(st ^ 1, 0, jb, nset); else read_b(st, s + 1, jb, nset); }
        } else {
          // the stage's DMAs, DPR a row from the barrier on; the last ones in the next stage's first unit, unless they
          // were sent before the output
          constexpr int d = at * C::DPR + m - 1 - per_b;
          if constexpr (d < C::D) dma(std::integral_constant<int, d>{}, std::bool_constant<head>{}, head ? st : st ^ 1, kt);
        }
      };
      static_for<FN>([&](auto j_) {
        constexpr int j = j_;
        const u32x4_t b = br[set][j], x = ar[i % 4], h = C::FP8 ? ar_h[C::FP8 ? i % 4 : 0] : u32x4_t{0u, 0u, 0u, 0u};
        const i32x8_t fb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
        const i32x8_t fa = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)h[0], (int)h[1], (int)h[2], (int)h[3]};
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, fa, acc[i][j], FMT_FP4,
                                                                     C::FP8 ? FMT_FP8 : FMT_FP4, j % 4,
                                                                     (int)xb[set][j / 4], i % 4, (int)xa[set][i / 4]);
        __builtin_amdgcn_sched_barrier(0);
        static_for<acts>([&](auto n_) { if constexpr (n_ * FN / acts == j) { act(n_); __builtin_amdgcn_sched_barrier(0); } });
      });
    });
  };
  auto stage = [&]() __attribute__((always_inline)) {
    unit(std::integral_constant<int, 0>{});
    if constexpr (SS == 2) {
      unit(std::integral_constant<int, 1>{});
    } else {
#pragma unroll
      for (int j = 0; j < FN; ++j) br[0][j] = br[1][j];
#pragma unroll
      for (int j = 0; j < FN / 4; ++j) xb[0][j] = xb[1][j];
#pragma unroll
      for (int i = 0; i < FM / 4; ++i) xa[0][i] = xa[1][i];
    }
    st ^= 1;
  };

  // ---------------- results: 16 rows at a time through the wave's own LDS, so that the stores run along the rows.
  // A whole tile's rows go one step ahead: the next ones' writes and reads of LDS are under way while a row block's
  // pieces are stored.
  auto copy_out = [&](auto zero, auto whole_) __attribute__((always_inline)) {
    using T = decltype(zero);
    constexpr bool WHOLE = whole_;
    constexpr int VT = 16 / (int)sizeof(T);                 // values per 16-byte piece
    constexpr int COLS = C::OUT_ROW / (int)sizeof(T);       // columns that fit at once
    constexpr int NQ = C::OUT_ROW / 16, RPP = 64 / NQ;      // pieces per row, rows per pass of the wave
    constexpr int NH = WN / COLS, NC = FM * NH, NP = 16 / RPP;
    int lane = tid & 63;
    asm volatile("" : "+v"(lane));   // keeps what follows from it out of the walk, where it would hold registers
    const int g = lane >> 4, rl = lane & 15, prow = lane / NQ, piece = lane % NQ;
    uint8_t* const stg = smem + C::OUT0 + wave * C::OUT_WAVE;
    const int mw = cur.m0 + wm * WM, nw = cur.n0 + wn * WN;
    T* const o0 = static_cast<T*>(a.c) + (int64_t)(mw + prow) * a.ldc + nw + piece * VT;
    auto put = [&](auto c_) __attribute__((always_inline)) {
      constexpr int i = c_ / NH, h = c_ % NH;
#pragma unroll
      for (int jj = 0; jj < COLS / 16; ++jj) {
        const f32x4_t v = acc[i][h * (COLS / 16) + jj];
        const int byte = (16 * jj + 4 * g) * (int)sizeof(T);
        uint8_t* p = stg + rl * C::OUT_ROW + (((byte >> 4) ^ (rl % NQ)) << 4) + (byte & 15);
        if constexpr (sizeof(T) == 2)
          *reinterpret_cast<uint2*>(p) = make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]));
        else
          *reinterpret_cast<f32x4_t*>(p) = v;
      }
    };
    auto at = [&](int q) { return stg + (q * RPP + prow) * C::OUT_ROW + ((piece ^ ((q * RPP + prow) % NQ)) << 4); };
    if constexpr (WHOLE) {
      u32x4v_t v[2][NP];
      auto get = [&](auto c_) __attribute__((always_inline)) {
        put(c_);
#pragma unroll
        for (int q = 0; q < NP; ++q) v[c_ % 2][q] = *reinterpret_cast<const u32x4v_t*>(at(q));
        __builtin_amdgcn_sched_barrier(0);
      };
      get(std::integral_constant<int, 0>{});
      static_for<NC>([&](auto c_) {
        constexpr int c = c_;
        if constexpr (c + 1 < NC) get(std::integral_constant<int, c + 1>{});
#pragma unroll
        for (int q = 0; q < NP; ++q)
          __builtin_nontemporal_store(v[c % 2][q], reinterpret_cast<u32x4u_t*>(o0 + (int64_t)(16 * (c / NH) + q * RPP) * a.ldc + c % NH * COLS));
      });
    } else {
      static_for<NC>([&](auto c_) {
        constexpr int c = c_;
        put(c_);
#pragma nounroll
        for (int q = 0; q < NP; ++q) {
          const T* p = reinterpret_cast<const T*>(at(q));
          T* o = o0 + (int64_t)(16 * (c / NH) + q * RPP) * a.ldc + c % NH * COLS;
          const int cnt = mw + 16 * (c / NH) + q * RPP + prow < cur.mlim ? a.N - nw - piece * VT - c % NH * COLS : 0;
          if (cnt >= VT) {
            *reinterpret_cast<u32x4u_t*>(o) = *reinterpret_cast<const u32x4v_t*>(p);
          } else if (cnt > 0) {
#pragma nounroll
            for (int k = 0; k < cnt; ++k) o[k] = p[k];
          }
        }
      });
    }
  };

  // ---------------- the walk
  auto send = [&](auto from_, int st) __attribute__((always_inline)) {   // the stage's DMAs from that one on
    static_for<C::D>([&](auto i_) {
      if constexpr (i_ >= from_) dma(i_, std::true_type{}, st, 1);
    });
  };
  constexpr std::integral_constant<int, 0> all{};
  constexpr std::integral_constant<int, C::D_TAIL> rest{};
  const int v_cur = map_now(cur), v_nxt = map_now(nxt);
  put_row(cur, 0, v_cur);
  put_row(nxt, 1, v_nxt);
  fetch_map(nxt2);
  __syncthreads();
  aim(cur, 0, src);
  if constexpr (!C::SC4) {
    load_scales(0);
    store_scales(0);
    load_scales(1);
  }
  set_dma(0);
  send(all, 0);
  set_dma(1);
  send(all, 1);
  gg::vm_wait<0>();
  __syncthreads();
  read_scales(0, 0, 0);
#pragma unroll
  for (int i = 0; i < FM / 4; ++i) turn(xa[0][i]);
#pragma unroll
  for (int j = 0; j < FN / 4; ++j) turn(xb[0][j]);
#pragma unroll
  for (int j = 0; j < FN; ++j) read_b(0, 0, j, 0);
  read_a(0, 0, 0, 0);
  read_a(0, 0, 1, 1);
  read_a(0, 0, 2, 2);
  for (;;) {
    if ((it + 3) % C::TILES == 0) list_tiles(it + 3);   // (the waves' staged output has been read by then)
    aim(nxt, it + 1, src_n);
    put_row(nxt2, it + 2, s_map[tid & (BM - 1)]);
    const Tile nxt3 = tile_at(it + 3);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the entries have been read
    fetch_map(nxt3);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma nounroll
    for (kt = 0; kt < nk; ++kt) stage();
    send(rest, st ^ 1);           // the rest of the next tile's second stage, ahead of the stores
    if (cur.m0 + (wm + 1) * WM <= cur.mlim && cur.n0 + (wn + 1) * WN <= a.N) {
      if (a.c_bf16) copy_out(bf16_t{}, std::true_type{});
      else copy_out(float{}, std::true_type{});
    } else {
      if (a.c_bf16) copy_out(bf16_t{}, std::false_type{});
      else copy_out(float{}, std::false_type{});
      gg::vm_wait<0>();           // (fewer stores than the next tile's first wait allows for)
    }
    if (nxt.e < 0) break;
    cur = nxt;
    nxt = nxt2;
    nxt2 = nxt3;
    ++it;
  }
  gg::vm_wait<0>();   // no DMA is under way when the block gives its LDS back
}

// row tiles of height bm at most: every expert with rows ends in a partial one
int64_t max_tiles(const Mx4Args& a, int bm) {
  if (a.offsets == nullptr || a.E == 1) return ((int64_t)a.rows + bm - 1) / bm;
  return (a.E < a.rows ? a.E : a.rows) + (int64_t)a.rows / bm;
}

template <bool FP8, bool SC4, int CF>
hipError_t launch_stream(const Mx4Args& a, hipStream_t s) {
  const int n_groups = (a.N + 16 * CF - 1) / (16 * CF);
  const int64_t grid = max_tiles(a, 16) * n_groups;
  if (grid >= 1 << 24) return hipErrorInvalidValue;   // a launch has fewer than 2^32 threads
  return launch_kernel(mx4_stream_kernel<FP8, SC4, CF>, dim3((unsigned)grid), dim3(256), 0, s, a, n_groups);
}

template <class C>
hipError_t launch_tiles(const Mx4Args& a, hipStream_t s) {
  const int n_tiles = (a.N + C::BN - 1) / C::BN;
  const int64_t tiles = max_tiles(a, C::BM) * n_tiles;
  const int64_t all = (tiles + gg::NXCD - 1) / gg::NXCD * gg::NXCD, resident = resident_blocks(C::PER_CU);
  return launch_kernel(mx4_tile_kernel<C>, dim3((unsigned)(all < resident ? all : resident)), dim3(C::NTHR), 0, s, a,
                       n_tiles);
}

// What the stream kernel and the 128 x 128 tiles take, in us, as fitted to 107 sizes (1 to 8192 rows, 1 to 128 experts,
// N 256 to 4096, K 128 to 4480): good to 20 %, and the choice they give was within 4 % of the better one but for two of
// the sizes (9 and 11 %).
//
// The stream kernel reads the weights once for every 16 rows of an expert, which costs most where all 16 are there.
// Tiles come in rounds of two on every compute unit, each as long as K and a little more.  Both measured, stream and
// tiles: 32 rows on 32 of 128 experts, 1536 x 2048: 13.2 and 17.6; 64 rows on 56: 20.3 and 18.6, 128 rows on 81: 28.7 and
// 25.9; 64 rows of one 4096 x 4096 weight 13.2 and 17.0, 128 rows 24.1 and 16.8; 2048 rows of one 1024 x 256 weight 11.4
// and 8.4, 512 rows of 64 4096 x 128 ones 10.1 and 18.7.
bool few_k(const Mx4Args& a) { return a.K <= 3 * 4 * KSTEP; }   // up to 3 steps for each wave of the stream kernel
double stream_us(const Mx4Args& a) {
  const double tiles = (double)max_tiles(a, 16), fill = a.rows / (16 * tiles);
  return 6 + (few_k(a) ? 0.2 : 0.28) * (0.4 + 0.6 * fill) * tiles * a.N * (a.K + 60.0) / 2 / (1 << 20);
}
double tile_us(const Mx4Args& a) {
  const double tiles = (double)max_tiles(a, 128) * ((a.N + 127) / 128), rounds = tiles / resident_blocks(2);
  const int stage = a.a_fp8 ? 128 : 256, stages = (a.K + stage - 1) / stage;
  return 6 + (rounds < 1 ? 1 : rounds) * (2 + 0.8 * (stages < 2 ? 2 : stages));
}

// 256 x 256 tiles halve the operands' traffic: a round of one on every compute unit takes 1.2 times (K = 4096) to
// 1.45 times (short K) a round of two 128 x 128 tiles there and does twice the work, but more of it is partial tiles and
// the last round's idle units.  Of 40 sizes with 256 rows an expert and more the rule was right or within 8 %.  Large and small
// measured: 1024 rows for each of 128 experts, 1536 x 2048, 275 us and 324, 512 rows 185 and 207, 256 rows 118 and 112;
// 512 rows of 4096 x 1536 393 and 448; one 4096 x 4096 weight, 4096 rows 44 and 57, 2048 rows 38 and 33; 512 rows of 16
// 2048 x 1024 weights 29 and 25.
bool big_tiles(const Mx4Args& a) {
  const int64_t units = resident_blocks(1), big = (max_tiles(a, 256) * ((a.N + 255) / 256) + units - 1) / units;
  const double experts = a.E == 1 ? 0 : a.E < a.rows ? a.E : a.rows;
  const double small = (a.rows / 128.0 + experts / 2) * ((a.N + 127) / 128) / (2 * units);
  return std::min(1.45, 1.1 + 400.0 / a.K) * big < small;
}

// Four fragments of columns to a wave of the stream kernel read A less often, two have more blocks: with a short K 64
// tokens on 48 experts' 1000 x 1120 took 9.1 and 10.0 us, 16 tokens on 8 experts' 4096 x 1536 9.0 and 10.1;
// with 4 the 32 rows above 15.1 and 13.4.  (One fragment: 16.3.)
template <bool FP8, bool SC4>
hipError_t launch_formats(const Mx4Args& a, hipStream_t s) {
  // scales that pass through registers are read 8 bytes at a time: that many in each array
  const bool room = SC4 || ((int64_t)a.a_rows * a.KB >= 8 && (int64_t)a.E * a.N * a.KB >= 8);
  if (!room || stream_us(a) <= tile_us(a))
    return few_k(a) ? launch_stream<FP8, SC4, 4>(a, s) : launch_stream<FP8, SC4, 2>(a, s);
  if constexpr (SC4)
    if (big_tiles(a)) return launch_tiles<Mx4Cfg<FP8, SC4, 256, 256, 2, 4, 1>>(a, s);
  return launch_tiles<Mx4Cfg<FP8, SC4, 128, 128, 2, 2, 2>>(a, s);
}

}  // namespace

hipError_t launch_mx4_product(const Mx4Args& a, hipStream_t s) {
  const bool sc4 = a.KB % 4 == 0;
  if (a.a_fp8) return sc4 ? launch_formats<true, true>(a, s) : launch_formats<true, false>(a, s);
  return sc4 ? launch_formats<false, true>(a, s) : launch_formats<false, false>(a, s);
}

}  // namespace moe
