// MXFP4 quantisation and its inverse (TE dropless-MoE page, "03 Specialised
// optimisations" quantises to MXFP8; this is the same microscaling with 4-bit
// elements).  A block of 32 consecutive values stores one E8M0 scale 2^X and 32
// E2M1 codes (0, .5, 1, 1.5, 2, 3, 4, 6, sign in bit 3):
//   X    = smallest integer with amax <= 6 * 2^X, clamped to [-127, 127]
//          (-127 for an all-zero block); 255 as scale byte and zero codes when
//          the block holds an infinity or NaN
//   code = v / 2^X to the nearest value, ties to the even code, sign kept.
// The scaling is one exact fp32 product (2^-X is a normal number for every X
// that occurs: -127 .. 126) and the rounding is the hardware conversion, so the
// codes are those of the exact definition.  Both directions are bound by HBM:
// they read and write each byte once.
#include "moe_internal.h"
#include "row_vec.h"

namespace moe {
namespace {

// X + 127 from the bits of the block's largest magnitude (finite): amax = (1 +
// f) 2^(eb-127) and 6 = 1.5 * 2^2, so X = eb - 129 when f <= 0.5, else eb - 128;
// adding 0x3FFFFF carries into the exponent exactly when f > 0.5.  Up to
// 6 * 2^-127 = 0x01400000 (zero among them) the clamp gives X = -127.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax_bits) {
  return amax_bits <= 0x01400000u ? 0u : ((amax_bits + 0x3FFFFFu) >> 23) - 2u;
}
// 2^-X of scale byte s = X + 127 (s <= 253): exponent field 254 - s
__device__ __forceinline__ float mx4_inv_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }
// 2^X of any scale byte; 0 is the subnormal 2^-127, 255 NaN
__device__ __forceinline__ float mx4_scale(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x400000u : s == 255u ? 0x7FC00000u : s << 23);
}
constexpr uint32_t NONFINITE = 0x7F800000u;

// 8 values -> 8 codes in one word (value i in bits 4i .. 4i+3); 4 values -> the low half of one
__device__ __forceinline__ uint32_t mx4_pack(const float (&v)[4], float inv) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * inv, v[1] * inv, 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * inv, v[3] * inv, 1.0f, 1);
  return w;
}
__device__ __forceinline__ uint32_t mx4_pack(const float (&v)[8], float inv) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * inv, v[1] * inv, 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * inv, v[3] * inv, 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * inv, v[5] * inv, 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * inv, v[7] * inv, 1.0f, 3);
  return w;
}

// Along the rows a lane handles 16 bytes of values, 8 of bf16 or 4 of fp32, and
// the codes of those: 4 or 8 lanes a block, so that a wave's loads and stores
// are consecutive bytes on both sides.  (With 8 fp32 values a lane, in two
// pieces, the way back to 131072 x 2048 values took 536 us for 1.2 GB.)
template <typename T>
struct Lanes {
  static constexpr int V = RowVec<T>::N, N = 32 / V, BLOCKS = 256 / N;   // values a lane, lanes a block, blocks
  using codes_t = std::conditional_t<V == 8, uint32_t, uint16_t>;
};

// The block maximum crosses the lanes by swaps within quads and, for eight of
// them, the mirror of eight.  SWIGLU: v = SiLU(g1) * g3 with g1 at column c, g3
// at cols + c.  131072 x 2048: bf16 112 us (6.0 TB/s), fp32 203 (6.0); SwiGLU of
// them 94 (6.4) and 184 (6.2).
template <typename T, bool SWIGLU>
__global__ __launch_bounds__(256) void mx4_rows_kernel(const T* __restrict__ src, int64_t ld, int64_t rows, int cols,
                                                       int kb, uint8_t* __restrict__ codes,
                                                       uint8_t* __restrict__ scales) {
  using L = Lanes<T>;
  constexpr int V = L::V;
  const int q = threadIdx.x % L::N;
  const int64_t total = rows * kb;
  const int64_t step = (int64_t)gridDim.x * L::BLOCKS;
  for (int64_t b = (int64_t)blockIdx.x * L::BLOCKS + threadIdx.x / L::N; b < total; b += step) {   // a block's lanes together
    const int64_t r = b / kb;
    const int c = (int)(b - r * kb) * 32 + V * q;
    const int n = min(V, cols - c);
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.f;
    if (n > 0) {
      RowVec<T>::load_once(src + r * ld + c, n).unpack(v);
      if constexpr (SWIGLU) {
        float g3[V];
        RowVec<T>::load_once(src + r * ld + cols + c, n).unpack(g3);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = i < n ? v[i] * sigmoid_f32(v[i]) * g3[i] : 0.f;
      }
    }
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    amax = max(amax, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)amax, 0xB1, 0xF, 0xF, false));   // quad_perm 1,0,3,2
    amax = max(amax, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)amax, 0x4E, 0xF, 0xF, false));   // quad_perm 2,3,0,1
    if constexpr (L::N == 8)
      amax = max(amax, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)amax, 0x141, 0xF, 0xF, false));   // row_half_mirror
    const bool bad = amax >= NONFINITE;
    const uint32_t s = mx4_scale_byte(bad ? 0u : amax);
    const uint32_t w = mx4_pack(v, mx4_inv_scale(s));
    using codes_t = typename L::codes_t;
    __builtin_nontemporal_store((codes_t)(bad ? 0u : w), reinterpret_cast<codes_t*>(codes) + b * L::N + q);
    if (q == 0) scales[b] = (uint8_t)(bad ? 255u : s);
  }
}

// Blocks down the columns, written transposed.  A tile of TR rows x TF columns
// per thread block: lane l of wave w takes columns 2l, 2l+1 over blocks w, w + 4
// of 32 rows, read row by row (a wave's 256 or 512 consecutive bytes) straight
// into registers; only the codes pass through LDS, to leave as the tile's 128
// bytes of every output row.
constexpr int TR = 256, TF = 128;
constexpr int CODE_LD = TR / 2 + 16;   // bytes between the staged code rows: 16-byte pieces spread over the banks

__device__ __forceinline__ void load_pair(const bf16_t* p, int n, float& a, float& b) {
  typedef uint32_t u32u_t __attribute__((aligned(2)));
  uint32_t w = 0;
  if (n >= 2) w = __builtin_nontemporal_load(reinterpret_cast<const u32u_t*>(p));
  else if (n == 1) w = *p;
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void load_pair(const float* p, int n, float& a, float& b) {
  typedef float f32x2u_t __attribute__((ext_vector_type(2), aligned(4)));
  a = b = 0.f;
  if (n >= 2) {
    const f32x2u_t v = __builtin_nontemporal_load(reinterpret_cast<const f32x2u_t*>(p));
    a = v[0];
    b = v[1];
  } else if (n == 1) {
    a = *p;
  }
}

template <typename T>
__global__ __launch_bounds__(256) void mx4_cols_kernel(const T* __restrict__ src, int64_t ld, int rows, int cols,
                                                       int kb, int n_ft, int n_rt, int64_t tiles,
                                                       uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ __attribute__((aligned(16))) uint8_t s_codes[TF * CODE_LD];
  __shared__ __attribute__((aligned(8))) uint8_t s_scales[TF * (TR / 32)];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t L = blockIdx.x; L < tiles; L += gridDim.x) {
    const int ft = (int)(L % n_ft);
    const int64_t m = L / n_ft;
    const int rt = (int)(m % n_rt);
    const int64_t batch = m / n_rt;
    const int f = ft * TF + 2 * lane;
    const int nf = min(2, cols - f);              // <= 0: no column here
    const T* base = src + batch * rows * ld + f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int blk = wave + 4 * half;
      const int r0 = rt * TR + 32 * blk;
      float v[2][32];
      if (r0 + 32 <= rows) {
#pragma unroll
        for (int i = 0; i < 32; ++i) load_pair(base + (int64_t)(r0 + i) * ld, nf, v[0][i], v[1][i]);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) load_pair(base + (int64_t)(r0 + i) * ld, r0 + i < rows ? nf : 0, v[0][i], v[1][i]);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) amax = max(amax, __float_as_uint(v[c][i]) & 0x7FFFFFFFu);
        const bool bad = amax >= NONFINITE;
        const uint32_t s = mx4_scale_byte(bad ? 0u : amax);
        const float inv = mx4_inv_scale(s);
        u32x4v_t w;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = v[c][8 * g + i];
          w[g] = bad ? 0u : mx4_pack(x, inv);
        }
        *reinterpret_cast<u32x4v_t*>(&s_codes[(2 * lane + c) * CODE_LD + 16 * blk]) = w;
        s_scales[(2 * lane + c) * (TR / 32) + blk] = (uint8_t)(bad ? 255u : s);
      }
    }
    __syncthreads();
    const int b0 = rt * (TR / 32), nb = min(TR / 32, kb - b0);   // the tile's blocks of an output row
    const int64_t row0 = batch * cols + ft * TF;
    const int nc = min(TF, cols - ft * TF);
#pragma unroll
    for (int i = threadIdx.x; i < TF * (TR / 32); i += 256) {
      const int c = i / (TR / 32), b = i % (TR / 32);
      if (c < nc && b < nb)
        *reinterpret_cast<u32x4v_t*>(codes + ((row0 + c) * kb + b0 + b) * 16) =
            *reinterpret_cast<const u32x4v_t*>(&s_codes[c * CODE_LD + 16 * b]);
    }
    if (threadIdx.x < nc) {
      const int c = threadIdx.x;
      uint8_t* o = scales + (row0 + c) * kb + b0;
      const uint64_t w = *reinterpret_cast<const uint64_t*>(&s_scales[c * (TR / 32)]);
      typedef uint64_t u64u_t __attribute__((aligned(1)));
      if (nb == TR / 32) *reinterpret_cast<u64u_t*>(o) = w;
      else
        for (int b = 0; b < nb; ++b) o[b] = (uint8_t)(w >> (8 * b));
    }
    __syncthreads();
  }
}

// The way back, lanes as along the rows.  131072 x 2048: bf16 93 us (7.3 TB/s),
// fp32 160 (7.6).
template <typename T>
__global__ __launch_bounds__(256) void mx4_values_kernel(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, int64_t rows, int cols,
                                                         int kb, T* __restrict__ out, int64_t ld) {
  using L = Lanes<T>;
  constexpr int V = L::V;
  const int q = threadIdx.x % L::N;
  const int64_t total = rows * kb, step = (int64_t)gridDim.x * L::BLOCKS;
  for (int64_t b = (int64_t)blockIdx.x * L::BLOCKS + threadIdx.x / L::N; b < total; b += step) {
    const int64_t r = b / kb;
    const int c = (int)(b - r * kb) * 32 + V * q;
    const int n = min(V, cols - c);
    const uint32_t w = reinterpret_cast<const typename L::codes_t*>(codes)[b * L::N + q];
    const float s = mx4_scale(scales[b]);
    if (n <= 0) continue;
    float v[V];
    const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const auto p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    v[0] = p0[0] * s; v[1] = p0[1] * s; v[2] = p1[0] * s; v[3] = p1[1] * s;
    if constexpr (V == 8) {
      const auto p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
      const auto p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
      v[4] = p2[0] * s; v[5] = p2[1] * s; v[6] = p3[0] * s; v[7] = p3[1] * s;
    }
    RowVec<T>::pack(v).store_once(out + r * ld + c, n);
  }
}

// Grid of a kernel that loops over units: a unit each up to `most` thread blocks, then several each.  Quantising
// 131072 x 2048 fp32 values along the rows took 203 us with 2^16 blocks and 220 with one for every unit, the way back
// 181 and 160.
unsigned stream_grid(int64_t units, int64_t most = 65536) { return (unsigned)(units < most ? units : most); }
constexpr int64_t EVERY_UNIT = 1 << 23;   // a launch has fewer than 2^32 threads

template <typename T>
hipError_t quantize_t(const T* src, int64_t ld, int batch, int rows, int cols, int along, int swiglu, uint8_t* codes,
                      uint8_t* scales, hipStream_t s) {
  if (along == 1) {
    const int kb = (cols + 31) / 32;
    const int64_t n = (int64_t)batch * rows;
    const dim3 grid(stream_grid((n * kb + Lanes<T>::BLOCKS - 1) / Lanes<T>::BLOCKS));
    return swiglu ? launch_kernel(mx4_rows_kernel<T, true>, grid, dim3(256), 0, s, src, ld, n, cols, kb, codes, scales)
                  : launch_kernel(mx4_rows_kernel<T, false>, grid, dim3(256), 0, s, src, ld, n, cols, kb, codes,
                                  scales);
  }
  const int kb = (rows + 31) / 32, n_ft = (cols + TF - 1) / TF, n_rt = (rows + TR - 1) / TR;
  const int64_t tiles = (int64_t)batch * n_ft * n_rt;
  return launch_kernel(mx4_cols_kernel<T>, dim3(stream_grid(tiles)), dim3(256), 0, s, src, ld, rows, cols, kb, n_ft,
                       n_rt, tiles, codes, scales);
}

}  // namespace

hipError_t launch_mx4_quantize(const void* src, int64_t ld, int batch, int rows, int cols, int type, int along,
                               int swiglu, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  return type == 0 ? quantize_t(static_cast<const float*>(src), ld, batch, rows, cols, along, swiglu, codes, scales, s)
                   : quantize_t(static_cast<const bf16_t*>(src), ld, batch, rows, cols, along, swiglu, codes, scales, s);
}

hipError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int rows, int cols, void* out,
                                 int64_t ld, int type, hipStream_t s) {
  auto go = [&](auto zero) {
    using T = decltype(zero);
    const int kb = (cols + 31) / 32;
    const int64_t units = ((int64_t)rows * kb + Lanes<T>::BLOCKS - 1) / Lanes<T>::BLOCKS;
    return launch_kernel(mx4_values_kernel<T>, dim3(stream_grid(units, EVERY_UNIT)), dim3(256), 0, s, codes, scales,
                         (int64_t)rows, cols, kb, static_cast<T*>(out), ld);
  };
  return type == 0 ? go(float{}) : go(bf16_t{});
}

}  // namespace moe
