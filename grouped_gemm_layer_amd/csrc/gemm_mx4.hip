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

constexpr int KSTEP = 128;   // K of one scaled MFMA
constexpr int FMT_FP8 = 0, FMT_FP4 = 4;   // format fields of the instruction

// Row tile i (of height bm, counted over the experts in order) -> expert and
// rows [m0, mlim).  Every wave finds it by itself: lane l counts the tiles of
// experts l*per .. of the offsets, a prefix sum over the lanes and a ballot
// give the lane that holds tile i.  That takes about 0.5 us of a tile's time
// and saves the launch that would build a table.  Offsets are cut to [0, rows]
// so that no index leaves c.  False behind the last tile.
__device__ __forceinline__ bool find_tile(const Mx4Args& a, int bm, int i, int lane, int& e, int& m0, int& mlim) {
  if (a.offsets == nullptr) {
    e = 0;
    m0 = i * bm;
    mlim = a.rows;
    return m0 < mlim;
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
  if (!find_tile(a, 16 * MF, tile, lane, e, m0, mlim)) return;
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

template <bool FP8, bool SC4>
hipError_t launch_formats(const Mx4Args& a, hipStream_t s) {
  return launch_stream<FP8, SC4, 1, 4>(a, s);
}

}  // namespace

hipError_t launch_mx4_product(const Mx4Args& a, hipStream_t s) {
  const bool sc4 = a.KB % 4 == 0;
  if (a.a_fp8) return sc4 ? launch_formats<true, true>(a, s) : launch_formats<true, false>(a, s);
  return sc4 ? launch_formats<false, true>(a, s) : launch_formats<false, false>(a, s);
}

}  // namespace moe
