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

namespace moe {
namespace {

using gg::OOB;
using gg::make_rsrc;
using gg::u32x4_t;
typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));

#ifndef MOE_MX4_BIG
#define MOE_MX4_BIG 256
#endif
#ifndef MOE_MX4_MID
#define MOE_MX4_MID 32
#endif
constexpr int MX4_BIG = MOE_MX4_BIG, MX4_MID = MOE_MX4_MID;
constexpr int KSTEP = 128;   // K of one scaled MFMA
constexpr int FMT_FP8 = 0, FMT_FP4 = 4;   // format fields of the instruction

// Row tile i (of height bm, counted over the experts in order) -> expert and
// rows [m0, mlim).  Every wave finds it by itself: lane l counts the tiles of
// experts l*per .. of the offsets, a prefix sum over the lanes and a ballot
// give the lane that holds tile i.  That takes about 0.5 us of a tile's time
// and saves the launch that would build a table.  Offsets are cut to [0, rows]
// so that no index leaves c.  `pick` gives i from the number of tiles; false
// when that is no tile.
template <class Pick>
__device__ __forceinline__ bool find_tile(const Mx4Args& a, int bm, int lane, Pick&& pick, int& e, int& m0,
                                          int& mlim) {
  if (a.offsets == nullptr) {
    const int total = (a.rows + bm - 1) / bm, i = pick(total);
    if (i >= total) return false;
    e = 0;
    m0 = i * bm;
    mlim = a.rows;
    return true;
  }
  const int per = (a.E + 63) / 64;   // <= 8
  int cnt[8], sum = 0;
  const int e0 = lane * per;
  int o = min(max(a.offsets[min(e0, a.E)], 0), a.rows);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    cnt[q] = 0;
    if (q < per) {
      const int o1 = min(max(a.offsets[min(e0 + q + 1, a.E)], 0), a.rows);
      cnt[q] = max(0, o1 - o + bm - 1) / bm;
      o = o1;
    }
    sum += cnt[q];
  }
  int inc = sum;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int v = __shfl_up(inc, off);
    if (lane >= off) inc += v;
  }
  const int i = pick(__builtin_amdgcn_readlane(inc, 63));
  const uint64_t hit = __ballot(inc > i);
  if (hit == 0) return false;
  const int src = __builtin_ctzll(hit);
  int local = i - __builtin_amdgcn_readlane(inc - sum, src);
  int q = 0;
#pragma unroll
  for (int u = 0; u < 7; ++u) {
    const int c = __builtin_amdgcn_readlane(cnt[u], src);
    if (q == u && local >= c) {
      local -= c;
      q = u + 1;
    }
  }
  e = src * per + q;
  const int first = min(max(a.offsets[e], 0), a.rows);
  m0 = first + local * bm;
  mlim = min(max(a.offsets[e + 1], 0), a.rows);
  return true;
}

// A's row of row r of c, or -1 (reads as zeros)
__device__ __forceinline__ int a_row(const Mx4Args& a, int r) {
  int s = r;
  if (a.row_map) {
    const int f = a.row_map[r];
    s = f < 0 ? -1 : (int)((uint32_t)f / (uint32_t)a.row_div);
  }
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
// Few rows per expert: the weights are read once, straight into registers
// (each byte has one reader, so LDS would only add a stop), by as many waves as
// possible: a wave takes MF x 16 rows and 16 columns.  KS waves of a block
// split K and add their sums in wave order through LDS, for few columns.
// SC4: KB % 4 == 0, a K step's four scale bytes of a row are one aligned word.
// ---------------------------------------------------------------------------
template <bool FP8, bool SC4, int MF, int KS>
__global__ __launch_bounds__(256) void mx4_stream_kernel(Mx4Args a, int n_groups) {
  constexpr int U = 4;                         // K steps whose loads are in flight together
  constexpr int NWV = 4 / KS;                  // waves along the columns
  __shared__ f32x4_t s_acc[KS > 1 ? KS - 1 : 1][KS > 1 ? MF : 1][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, rl = lane & 15;
  const int tile = blockIdx.x / n_groups, ng = blockIdx.x % n_groups;
  int e, m0, mlim;
  if (!find_tile(a, 16 * MF, lane, [&](int) { return tile; }, e, m0, mlim)) return;
  const int wk = KS > 1 ? wave : 0, wn = KS > 1 ? 0 : wave;
  const int n0 = (ng * NWV + wn) * 16;
  const uint32_t pb = (uint32_t)a.KB * 16, pa = FP8 ? (uint32_t)a.K : pb;   // code bytes of a row
  const auto rb = make_rsrc(a.b + (size_t)e * a.N * pb, (uint32_t)a.N * pb);
  const auto rsb = make_rsrc(a.sb + (size_t)e * a.N * a.KB, (uint32_t)a.N * a.KB);
  const auto ra = make_rsrc(a.a, (uint32_t)a.a_rows * pa);
  const auto rsa = make_rsrc(a.sa, (uint32_t)a.a_rows * a.KB);
  const int nb = n0 + rl;
  const bool nok = nb < a.N;
  const uint32_t ob = nok ? (uint32_t)nb * pb : 0, osb = nok ? (uint32_t)nb * a.KB : 0;
  uint32_t oa[MF], osa[MF];
  bool mok[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int m = m0 + 16 * i + rl;
    const int s = m < mlim ? a_row(a, m) : -1;
    mok[i] = s >= 0;
    oa[i] = mok[i] ? (uint32_t)s * pa : 0;
    osa[i] = mok[i] ? (uint32_t)s * a.KB : 0;
  }
  f32x4_t acc[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int nk = (a.K + KSTEP - 1) / KSTEP;
  const int per = (nk + KS - 1) / KS;
  const int k0 = wk * per, k1 = min(nk, k0 + per);
  auto scale = [&](__amdgpu_buffer_rsrc_t r, uint32_t row, bool ok, int kt) -> int {
    if constexpr (SC4) return __builtin_amdgcn_raw_buffer_load_b32(r, ok ? row + 4 * kt : OOB, 0, 0);
    else return __builtin_amdgcn_raw_buffer_load_b8(r, ok && 4 * kt + g < a.KB ? row + 4 * kt + g : OOB, 0, 0);
  };
  for (int kt0 = k0; kt0 < k1; kt0 += U) {
    u32x4_t cb[U], ca[U][MF], cah[U][FP8 ? MF : 1];
    int sb[U], sa[U][MF];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kt = kt0 + u;
      const uint32_t kb = (uint32_t)kt * 64 + 16 * g;
      const bool in = kt < k1;
      cb[u] = __builtin_amdgcn_raw_buffer_load_b128(rb, in && nok && kb < pb ? ob + kb : OOB, 0, 0);
      sb[u] = scale(rsb, osb, in && nok, kt);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kt = kt0 + u;
      const bool in = kt < k1;
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        if constexpr (FP8) {
          const uint32_t ka = (uint32_t)kt * 128 + 16 * g;
          ca[u][i] = __builtin_amdgcn_raw_buffer_load_b128(ra, in && mok[i] && ka < pa ? oa[i] + ka : OOB, 0, 0);
          cah[u][i] = __builtin_amdgcn_raw_buffer_load_b128(ra, in && mok[i] && ka + 64 < pa ? oa[i] + ka + 64 : OOB, 0, 0);
        } else {
          const uint32_t ka = (uint32_t)kt * 64 + 16 * g;
          ca[u][i] = __builtin_amdgcn_raw_buffer_load_b128(ra, in && mok[i] && ka < pa ? oa[i] + ka : OOB, 0, 0);
        }
        sa[u][i] = scale(rsa, osa[i], in && mok[i], kt);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const i32x8_t fb = {(int)cb[u][0], (int)cb[u][1], (int)cb[u][2], (int)cb[u][3], 0, 0, 0, 0};
      const int xb = SC4 ? (int)((uint32_t)sb[u] >> (8 * g)) : sb[u];
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        i32x8_t fa = {(int)ca[u][i][0], (int)ca[u][i][1], (int)ca[u][i][2], (int)ca[u][i][3], 0, 0, 0, 0};
        if constexpr (FP8) {
          fa[4] = (int)cah[u][i][0]; fa[5] = (int)cah[u][i][1]; fa[6] = (int)cah[u][i][2]; fa[7] = (int)cah[u][i][3];
        }
        const int xa = SC4 ? (int)((uint32_t)sa[u][i] >> (8 * g)) : sa[u][i];
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, fa, acc[i], FMT_FP4, FP8 ? FMT_FP8 : FMT_FP4, 0,
                                                                  xb, 0, xa);
      }
    }
  }
  if constexpr (KS > 1) {
    if (wave > 0) {
#pragma unroll
      for (int i = 0; i < MF; ++i) s_acc[wave - 1][i][lane] = acc[i];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 0; w < KS - 1; ++w)
#pragma unroll
      for (int i = 0; i < MF; ++i) acc[i] += s_acc[w][i][lane];
  }
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int m = m0 + 16 * i + rl, n = n0 + 4 * g;
    if (m < mlim && n < a.N) store4(a, m, n, acc[i]);
  }
}

// ---------------------------------------------------------------------------
// Many rows per expert: BM x BN tiles, operands through LDS.
//
// K advances by stages of KST (256 with MXFP4 rows, 128 with MXFP8: either way
// 128 bytes, a whole line, per row of A).  Two stages of LDS: while one is
// multiplied, the other receives the next by buffer-to-LDS DMA (16 bytes a
// lane; lanes outside a row, its K or the tile read zeros through an
// out-of-range offset).  One barrier per stage.  Code rows are cut in 16-byte
// chunks, XOR-swizzled within 128 bytes, so that a fragment's 64 chunks cover
// every bank equally; with MXFP8 rows, B's 64-byte rows lie in pairs.
//
// Scales: thread t owns row t of the stage's BM + BN rows, loads its 8 (4)
// bytes of the next stage into a register and, after the products, writes them
// to LDS in the order the lanes consume them: lane (r, g) of wave row w finds
// the bytes of its FM row blocks and both K steps side by side, so one LDS read
// per operand and stage brings them all, and the instruction's byte select
// picks each one.
// ---------------------------------------------------------------------------
template <int N, class F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl<N>(f, std::make_integer_sequence<int, N>{});
}

template <bool FP8_, int BM_, int BN_, int WGM_, int WGN_>
struct Mx4Cfg {
  static constexpr bool FP8 = FP8_;
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_;
  static constexpr int NW = WGM * WGN, NTHR = 64 * NW;
  static constexpr int WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
  static constexpr int KST = FP8 ? 128 : 256;            // K per stage
  static constexpr int SS = KST / KSTEP;                 // MFMA steps per stage
  static constexpr int RA = 128, RB = KST / 2;           // code bytes per row and stage
  static constexpr int SB = KST / 32;                    // scale bytes per row and stage
  static constexpr int A_BYTES = BM * RA, B_BYTES = BN * RB;
  static constexpr int DA = A_BYTES / 1024 / NW, DB = B_BYTES / 1024 / NW;   // 1 KiB DMAs per wave
  static constexpr int A_SC = A_BYTES + B_BYTES, B_SC = A_SC + BM * SB;
  static constexpr int STAGE = B_SC + BN * SB;
  static constexpr int LDS = 2 * STAGE;
  static_assert(DA * NW * 1024 == A_BYTES && DB * NW * 1024 == B_BYTES, "whole DMAs per wave");
  static_assert(BM + BN == NTHR, "one scale row per thread");
  static_assert(FM * SS % 4 == 0 && FN * SS % 4 == 0, "whole words of scales per lane");
};

template <class C>
__global__ __launch_bounds__(C::NTHR) void mx4_tile_kernel(Mx4Args a, int n_tiles) {
  constexpr int BM = C::BM, BN = C::BN, WM = C::WM, WN = C::WN, FM = C::FM, FN = C::FN, NW = C::NW, SS = C::SS;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WGN, wn = wave % C::WGN;
  const int g = lane >> 4, rl = lane & 15;
  // block b runs on XCD b % 8; each XCD takes a contiguous run of the tiles, column tiles fastest, so that
  // the tiles sharing an expert's rows and weights meet in one L2
  int e, m0, mlim, nt;
  const bool live = find_tile(a, BM, lane, [&](int total) {
    const int64_t tiles = (int64_t)total * n_tiles;
    const int per_xcd = (int)((tiles + gg::NXCD - 1) / gg::NXCD);
    const int x = blockIdx.x % gg::NXCD, j = blockIdx.x / gg::NXCD;
    const int64_t L = (int64_t)x * per_xcd + j;
    if (j >= per_xcd || L >= tiles) return INT32_MAX;
    nt = (int)(L % n_tiles);
    return (int)(L / n_tiles);
  }, e, m0, mlim);
  if (!live) return;
  const int n0 = nt * BN;

  const uint32_t pb = (uint32_t)a.KB * 16, pa = C::FP8 ? (uint32_t)a.K : pb;   // code bytes of a row
  const auto rb = make_rsrc(a.b + (size_t)e * a.N * pb, (uint32_t)a.N * pb);
  const auto ra = make_rsrc(a.a, (uint32_t)a.a_rows * pa);
  const int nk = (a.K + C::KST - 1) / C::KST;

  // DMA i of wave w fills the 1 KiB block ci = i * NW + w of an operand: lane l
  // writes 16 bytes at 16 l, which hold chunk `col` of row `row` of that block
  const int line = lane >> 3, phys = lane & 7, chunk8 = phys ^ line;
  const uint32_t cola = 16u * chunk8;                                          // 8 rows of 128 bytes
  const uint32_t colb = C::RB == 128 ? 16u * chunk8 : 16u * (chunk8 & 3);      // or 16 rows of 64
  uint32_t oa[C::DA], ob[C::DB];
#pragma unroll
  for (int i = 0; i < C::DA; ++i) {
    const int m = m0 + 8 * (i * NW + wave) + line;
    const int s = m < mlim ? a_row(a, m) : -1;
    oa[i] = s >= 0 ? (uint32_t)s * pa + cola : OOB;
  }
#pragma unroll
  for (int i = 0; i < C::DB; ++i) {
    const int ci = i * NW + wave;
    const int n = n0 + (C::RB == 128 ? 8 * ci + line : 16 * ci + 2 * line + (chunk8 >> 2));
    ob[i] = n < a.N ? (uint32_t)n * pb + colb : OOB;
  }
  const uint32_t lds0 = (uint32_t)(size_t)(const __attribute__((address_space(3))) void*)smem;
  auto issue = [&](int kt, int st) __attribute__((always_inline)) {
    const uint32_t base = lds0 + (uint32_t)(st * C::STAGE);
    const uint32_t ka = (uint32_t)kt * C::RA, kb = (uint32_t)kt * C::RB;
    const bool in_a = cola + ka < pa, in_b = colb + kb < pb;
#pragma unroll
    for (int i = 0; i < C::DA; ++i)
      gg::dma16(ra, in_a ? oa[i] + ka : OOB, __builtin_amdgcn_readfirstlane(base + (i * NW + wave) * 1024));
#pragma unroll
    for (int i = 0; i < C::DB; ++i)
      gg::dma16(rb, in_b ? ob[i] + kb : OOB, __builtin_amdgcn_readfirstlane(base + C::A_BYTES + (i * NW + wave) * 1024));
  };

  // this thread's scale row: source, and where its bytes go (stage-relative)
  using sc_t = std::conditional_t<C::SB == 8, uint64_t, uint32_t>;
  typedef sc_t scu_t __attribute__((aligned(1)));
  const bool sc_b = tid >= BM;
  const int R = sc_b ? tid - BM : tid;
  int64_t sc_row = -1, sc_end;
  const uint8_t* sc_base;
  if (sc_b) {
    if (n0 + R < a.N) sc_row = ((int64_t)e * a.N + n0 + R) * a.KB;
    sc_base = a.sb;
    sc_end = (int64_t)a.E * a.N * a.KB;
  } else {
    const int s = m0 + R < mlim ? a_row(a, m0 + R) : -1;
    if (s >= 0) sc_row = (int64_t)s * a.KB;
    sc_base = a.sa;
    sc_end = (int64_t)a.a_rows * a.KB;
  }
  const int WX = sc_b ? WN : WM, FX = sc_b ? FN : FM;
  const int sc_dst = (sc_b ? C::B_SC : C::A_SC) + (((R / WX) * 16 + R % 16) * 4) * (FX * SS) + ((R % WX) / 16) * SS;
  // SB scale bytes of stage kt; those past the row's end zero.  The last bytes of the array are read from SB
  // before its end and shifted down.
  auto load_scales = [&](int kt) __attribute__((always_inline)) -> sc_t {
    sc_t v = 0;
    const int rem = a.KB - kt * C::SB;
    if (sc_row >= 0) {
      const int64_t at = sc_row + (int64_t)kt * C::SB, lim = sc_end - C::SB;
      const int64_t from = at < lim ? at : lim;
      v = *reinterpret_cast<const scu_t*>(sc_base + from) >> (8 * (int)(at - from));
    }
    if (rem < C::SB) v &= ((sc_t)1 << (8 * rem)) - 1;
    return v;
  };
  auto store_scales = [&](sc_t v, int st) __attribute__((always_inline)) {
    uint8_t* p = smem + st * C::STAGE + sc_dst;
#pragma unroll
    for (int q = 0; q < 4; ++q) {   // K block q of the step(s): the lanes with g = q
      if constexpr (SS == 2)
        *reinterpret_cast<uint16_t*>(p + q * (FX * SS)) = (uint16_t)(((v >> (8 * q)) & 0xFF) | ((v >> (32 + 8 * q)) & 0xFF) << 8);
      else
        p[q * FX] = (uint8_t)(v >> (8 * q));
    }
  };

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const bool idle = m0 + wm * WM >= mlim;   // no row of this wave: it only moves data

  auto multiply = [&](int st) __attribute__((always_inline)) {
    const uint8_t* base = smem + st * C::STAGE;
    constexpr int WA = FM * SS / 4, WB = FN * SS / 4;   // words of scales
    uint32_t xa[WA], xb[WB];
    const uint32_t* pxa = reinterpret_cast<const uint32_t*>(base + C::A_SC + ((wm * 16 + rl) * 4 + g) * (FM * SS));
    const uint32_t* pxb = reinterpret_cast<const uint32_t*>(base + C::B_SC + ((wn * 16 + rl) * 4 + g) * (FN * SS));
#pragma unroll
    for (int w = 0; w < WA; ++w) xa[w] = pxa[w];
#pragma unroll
    for (int w = 0; w < WB; ++w) xb[w] = pxb[w];
    static_for<SS>([&](auto s_) {
      constexpr int s = s_;
      i32x8_t fa[FM], fb[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int row = wn * WN + 16 * j + rl;
        int off;
        if constexpr (C::RB == 128) off = row * 128 + (((4 * s + g) ^ (row & 7)) << 4);
        else off = (row >> 1) * 128 + ((((row & 1) * 4 + g) ^ ((row >> 1) & 7)) << 4);
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(base + C::A_BYTES + off);
        fb[j] = i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int row = wm * WM + 16 * i + rl;
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(base + row * 128 + (((C::FP8 ? g : 4 * s + g) ^ (row & 7)) << 4));
        u32x4_t h = {0u, 0u, 0u, 0u};
        if constexpr (C::FP8) h = *reinterpret_cast<const u32x4_t*>(base + row * 128 + (((4 + g) ^ (row & 7)) << 4));
        fa[i] = i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], (int)h[0], (int)h[1], (int)h[2], (int)h[3]};
      }
      static_for<FM>([&](auto i_) {
        static_for<FN>([&](auto j_) {
          constexpr int i = i_, j = j_, ia = i * SS + s, ib = j * SS + s;
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              fb[j], fa[i], acc[i][j], FMT_FP4, C::FP8 ? FMT_FP8 : FMT_FP4, ib % 4, (int)xb[ib / 4], ia % 4,
              (int)xa[ia / 4]);
        });
      });
    });
  };

  sc_t sc = load_scales(0);
  issue(0, 0);
  gg::vm_wait<0>();
  store_scales(sc, 0);
  __syncthreads();
  for (int kt = 0; kt < nk; ++kt) {
    const int st = kt & 1;
    if (kt + 1 < nk) {
      sc = load_scales(kt + 1);
      issue(kt + 1, st ^ 1);
    }
    if (!idle) multiply(st);
    gg::vm_wait<0>();
    if (kt + 1 < nk) store_scales(sc, st ^ 1);
    __syncthreads();
  }

  // the tile leaves through LDS, CH rows at a time, so that the stores run along its rows
  auto copy_out = [&](auto zero) __attribute__((always_inline)) {
    using T = decltype(zero);
    constexpr int VT = 16 / (int)sizeof(T);                 // values per 16-byte piece
    constexpr int NQ = BN / VT, ROWB = BN * (int)sizeof(T);
    constexpr int CH = BM * ROWB <= C::LDS ? BM : BM * ROWB <= 2 * C::LDS ? BM / 2 : BM / 4;
    static_assert(CH * ROWB <= C::LDS && CH % 16 == 0, "row chunk fits");
#pragma unroll
    for (int ch = 0; ch < BM / CH; ++ch) {
      if (ch > 0) __syncthreads();
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if ((wm * WM + 16 * i) / CH != ch) continue;        // a 16-row block lies in one chunk
        const int row = (wm * WM + 16 * i) % CH + rl;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const int byte = (wn * WN + 16 * j + 4 * g) * (int)sizeof(T);
          uint8_t* p = smem + row * ROWB + (((byte >> 4) ^ (row % NQ)) << 4) + (byte & 15);
          const f32x4_t v = acc[i][j];
          if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint2*>(p) = make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]));
          else
            *reinterpret_cast<f32x4_t*>(p) = v;
        }
      }
      __syncthreads();
      T* c = static_cast<T*>(a.c);
      for (int q0 = tid; q0 < CH * NQ; q0 += C::NTHR) {
        const int row = q0 / NQ, q = q0 % NQ;
        const int m = m0 + ch * CH + row, n = n0 + q * VT;
        const int cnt = min(VT, a.N - n);
        if (m < mlim && cnt > 0) {
          const RowVec<T> v = {*reinterpret_cast<const u32x4v_t*>(smem + row * ROWB + ((q ^ (row % NQ)) << 4))};
          v.store(c + (int64_t)m * a.ldc + n, cnt);
        }
      }
    }
  };
  if (a.c_bf16) copy_out(bf16_t{});
  else copy_out(float{});
}

// row tiles of height bm at most: every expert with rows ends in a partial one
int64_t max_tiles(const Mx4Args& a, int bm) {
  if (a.offsets == nullptr) return ((int64_t)a.rows + bm - 1) / bm;
  return (a.E < a.rows ? a.E : a.rows) + (int64_t)a.rows / bm;
}

template <bool FP8, bool SC4, int MF, int KS>
hipError_t launch_stream(const Mx4Args& a, hipStream_t s) {
  const int cols = 16 * (4 / KS);
  const int n_groups = (a.N + cols - 1) / cols;
  const int64_t grid = max_tiles(a, 16 * MF) * n_groups;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  return launch_kernel(mx4_stream_kernel<FP8, SC4, MF, KS>, dim3((unsigned)grid), dim3(256), 0, s, a, n_groups);
}

template <class C>
hipError_t launch_tiles(const Mx4Args& a, hipStream_t s) {
  const int n_tiles = (a.N + C::BN - 1) / C::BN;
  const int64_t tiles = max_tiles(a, C::BM) * n_tiles;
  const int64_t grid = (tiles + gg::NXCD - 1) / gg::NXCD * gg::NXCD;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  return launch_kernel(mx4_tile_kernel<C>, dim3((unsigned)grid), dim3(C::NTHR), 0, s, a, n_tiles);
}

template <bool FP8, bool SC4>
hipError_t launch_formats(const Mx4Args& a, hipStream_t s) {
  // the tile kernel reads scales 8 bytes at a time and needs that many in each array
  const bool room = (int64_t)a.a_rows * a.KB >= 8 && (int64_t)a.E * a.N * a.KB >= 8;
  if (room && a.rows / a.E >= MX4_BIG) return launch_tiles<Mx4Cfg<FP8, 256, 256, 2, 4>>(a, s);
  if (room && a.rows / a.E >= MX4_MID) return launch_tiles<Mx4Cfg<FP8, 128, 128, 2, 2>>(a, s);
  return launch_stream<FP8, SC4, 1, 4>(a, s);
}

}  // namespace

hipError_t launch_mx4_product(const Mx4Args& a, hipStream_t s) {
  const bool sc4 = a.KB % 4 == 0;
  if (a.a_fp8) return sc4 ? launch_formats<true, true>(a, s) : launch_formats<true, false>(a, s);
  return sc4 ? launch_formats<false, true>(a, s) : launch_formats<false, false>(a, s);
}

}  // namespace moe
