// C ABI of the operators beside the layer: argument checks and launches (rows
// sorted by expert and back, MXFP4 quantisation and product, gradient norm and
// clipping).  As for the layer: no allocation on the device, no host
// synchronisation, every check before the first launch.
#include "../../include/moe.h"
#include "moe_internal.h"

#include <algorithm>
#include <limits>
#include <new>
#include <vector>

using namespace moe;

namespace {

inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline bool type_ok(int32_t type) { return type == MOE_TYPE_FP32 || type == MOE_TYPE_BF16; }
inline size_t type_size(int32_t type) { return type == MOE_TYPE_FP32 ? 4 : 2; }
inline moe_status launched(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }

// a matrix operand of `rows` rows of `cols` values: pointer, pitch, alignment
moe_status check_matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, int32_t type) {
  if (rows == 0 || cols == 0) return MOE_OK;
  if (!p) return MOE_ERR_NULL;
  if (ld < cols || ld > (int64_t)1 << 40) return MOE_ERR_DIMS;
  return aligned_to(p, type_size(type)) ? MOE_OK : MOE_ERR_ALIGN;
}

moe_status check_rows_call(const RowsArgs& a, int32_t type) {
  if (a.T < 0 || a.H < 0 || a.k <= 0 || a.rows < 0 || (int64_t)a.T * a.k > INT32_MAX) return MOE_ERR_DIMS;
  if (!type_ok(type) || a.k > 32) return MOE_ERR_UNSUPPORTED;
  if (a.T == 0) return MOE_OK;
  if (!a.f2s) return MOE_ERR_NULL;
  if (!aligned_to(a.f2s, 4) || !aligned_to(a.weights, 4) || !aligned_to(a.dweights, 4)) return MOE_ERR_ALIGN;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_sort_workspace_size(int32_t T, int32_t k, int32_t E, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  if (T < 0 || k <= 0 || E <= 0 || (int64_t)T * k > INT32_MAX) return MOE_ERR_DIMS;
  if (E > 512) return MOE_ERR_UNSUPPORTED;
  *bytes = sort_ws_bytes((int64_t)T * k, E);
  return MOE_OK;
}

moe_status moe_sort_tokens(const int32_t* topk_idx, int32_t T, int32_t k, int32_t E, int32_t* counts,
                           int32_t* offsets, int32_t* sorted_to_flat, int32_t* flat_to_sorted, void* ws,
                           size_t ws_bytes, hipStream_t stream) {
  size_t need = 0;
  const moe_status st = moe_sort_workspace_size(T, k, E, &need);
  if (st != MOE_OK) return st;
  if (!counts || !offsets || (T > 0 && (!topk_idx || !sorted_to_flat || !flat_to_sorted)) || (need > 0 && !ws))
    return MOE_ERR_NULL;
  if (!aligned_to(topk_idx, 4) || !aligned_to(counts, 4) || !aligned_to(offsets, 4) ||
      !aligned_to(sorted_to_flat, 4) || !aligned_to(flat_to_sorted, 4) || (need > 0 && !aligned_to(ws, 256)))
    return MOE_ERR_ALIGN;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  return launched(launch_sort(topk_idx, (int64_t)T * k, E, counts, offsets, sorted_to_flat, flat_to_sorted,
                              static_cast<int32_t*>(ws), stream));
}

moe_status moe_permute(const void* x, int64_t ldx, int32_t T, int32_t H, int32_t k, int32_t type,
                       const int32_t* flat_to_sorted, const float* weights, void* xp, int64_t ldp, int32_t rows,
                       hipStream_t stream) {
  RowsArgs a{};
  a.T = T; a.H = H; a.k = k; a.rows = rows; a.f2s = flat_to_sorted; a.weights = weights;
  a.token_in = x; a.ld_token_in = ldx;
  a.rows_out = xp; a.ld_rows_out = ldp;
  moe_status st = check_rows_call(a, type);
  if (st != MOE_OK) return st;
  if ((st = check_matrix(x, ldx, T, H, type)) != MOE_OK || (st = check_matrix(xp, ldp, rows, H, type)) != MOE_OK)
    return st;
  if (T == 0 || H == 0 || rows == 0) return MOE_OK;
  return launched(launch_scatter_rows(a, type, stream));
}

moe_status moe_permute_backward(const void* dxp, int64_t ldp, int32_t rows, int32_t T, int32_t H, int32_t k,
                                int32_t type, const int32_t* flat_to_sorted, const float* weights, const void* x,
                                int64_t ldx, void* dx, int64_t lddx, float* dweights, hipStream_t stream) {
  RowsArgs a{};
  a.T = T; a.H = H; a.k = k; a.rows = rows; a.f2s = flat_to_sorted; a.weights = weights; a.dweights = dweights;
  a.rows_in = dxp; a.ld_rows_in = ldp;
  a.token_in = x; a.ld_token_in = ldx;
  a.token_out = dx; a.ld_token_out = lddx;
  moe_status st = check_rows_call(a, type);
  if (st != MOE_OK) return st;
  if ((st = check_matrix(dxp, ldp, rows, H, type)) != MOE_OK || (st = check_matrix(dx, lddx, T, H, type)) != MOE_OK)
    return st;
  if (dweights && (st = check_matrix(x, ldx, T, H, type)) != MOE_OK) return st;
  if (T == 0 || (H == 0 && !dweights)) return MOE_OK;
  return launched(launch_gather_rows(a, type, stream));
}

moe_status moe_unpermute(const void* o, int64_t ldo, int32_t rows, int32_t T, int32_t H, int32_t k, int32_t type,
                         const int32_t* flat_to_sorted, const float* weights, void* y, int64_t ldy,
                         hipStream_t stream) {
  return moe_permute_backward(o, ldo, rows, T, H, k, type, flat_to_sorted, weights, nullptr, 0, y, ldy, nullptr,
                              stream);
}

moe_status moe_unpermute_backward(const void* dy, int64_t lddy, int32_t T, int32_t H, int32_t k, int32_t type,
                                  const int32_t* flat_to_sorted, const float* weights, const void* o, int64_t ldo,
                                  void* drows, int64_t lddr, int32_t rows, float* dweights, hipStream_t stream) {
  RowsArgs a{};
  a.T = T; a.H = H; a.k = k; a.rows = rows; a.f2s = flat_to_sorted; a.weights = weights; a.dweights = dweights;
  a.token_in = dy; a.ld_token_in = lddy;
  a.rows_in = o; a.ld_rows_in = ldo;
  a.rows_out = drows; a.ld_rows_out = lddr;
  moe_status st = check_rows_call(a, type);
  if (st != MOE_OK) return st;
  if ((st = check_matrix(dy, lddy, T, H, type)) != MOE_OK || (st = check_matrix(drows, lddr, rows, H, type)) != MOE_OK)
    return st;
  if (dweights && (st = check_matrix(o, ldo, rows, H, type)) != MOE_OK) return st;
  if (T == 0 || ((H == 0 || rows == 0) && !dweights)) return MOE_OK;
  return launched(launch_scatter_rows(a, type, stream));
}

moe_status moe_mxfp4_quantize(const void* src, int64_t ld, int32_t batch, int32_t rows, int32_t cols, int32_t type,
                              int32_t along, int32_t swiglu, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  if (batch < 0 || rows < 0 || cols < 0 || (along != 0 && along != 1)) return MOE_ERR_DIMS;
  if (!type_ok(type) || (swiglu && along == 0)) return MOE_ERR_UNSUPPORTED;
  const int64_t width = swiglu ? 2 * (int64_t)cols : cols;
  if (width > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (batch == 0 || rows == 0 || cols == 0) return MOE_OK;
  if (!codes || !scales) return MOE_ERR_NULL;
  const moe_status st = check_matrix(src, ld, (int64_t)batch * rows, width, type);
  if (st != MOE_OK) return st;
  if (!aligned_to(codes, 256) || !aligned_to(scales, 256)) return MOE_ERR_ALIGN;
  return launched(launch_mx4_quantize(src, ld, batch, rows, cols, type, along, swiglu != 0, codes, scales, stream));
}

moe_status moe_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int32_t rows, int32_t cols, void* out,
                                int64_t ld, int32_t type, hipStream_t stream) {
  if (rows < 0 || cols < 0) return MOE_ERR_DIMS;
  if (!type_ok(type)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return MOE_OK;
  if (!codes || !scales) return MOE_ERR_NULL;
  const moe_status st = check_matrix(out, ld, rows, cols, type);
  if (st != MOE_OK) return st;
  if (!aligned_to(codes, 256) || !aligned_to(scales, 256)) return MOE_ERR_ALIGN;
  return launched(launch_mx4_dequantize(codes, scales, rows, cols, out, ld, type, stream));
}

moe_status moe_mxfp4_product(const uint8_t* a_codes, const uint8_t* a_scales, int32_t a_rows, int32_t a_format,
                             const uint8_t* b_codes, const uint8_t* b_scales, int32_t E, int32_t N, int32_t K,
                             const int32_t* offsets, const int32_t* row_map, int32_t row_div, void* c, int64_t ldc,
                             int32_t rows, int32_t c_type, hipStream_t stream) {
  if (a_rows < 0 || E <= 0 || N < 0 || K <= 0 || rows < 0 || row_div <= 0) return MOE_ERR_DIMS;
  if (!offsets && E != 1) return MOE_ERR_NULL;
  if ((a_format != MOE_MX_FP4 && a_format != MOE_MX_FP8) || !type_ok(c_type) || E > 512) return MOE_ERR_UNSUPPORTED;
  if (a_format == MOE_MX_FP8 && K % 32 != 0) return MOE_ERR_UNSUPPORTED;
  const int64_t kb = ((int64_t)K + 31) / 32, limit = (int64_t)1 << 31;
  if (N * kb * 16 >= limit || a_rows * (a_format == MOE_MX_FP8 ? (int64_t)K : kb * 16) >= limit)
    return MOE_ERR_UNSUPPORTED;
  if ((int64_t)rows > INT32_MAX - 4096) return MOE_ERR_UNSUPPORTED;   // row indices with a tile's height added
  if (rows == 0 || N == 0) return MOE_OK;
  if (!b_codes || !b_scales || (a_rows > 0 && (!a_codes || !a_scales))) return MOE_ERR_NULL;
  const moe_status st = check_matrix(c, ldc, rows, N, c_type);
  if (st != MOE_OK) return st;
  if (!aligned_to(a_codes, 256) || !aligned_to(a_scales, 256) || !aligned_to(b_codes, 256) ||
      !aligned_to(b_scales, 256) || !aligned_to(offsets, 4) || !aligned_to(row_map, 4))
    return MOE_ERR_ALIGN;
  Mx4Args a{};
  a.a = a_codes; a.sa = a_scales; a.b = b_codes; a.sb = b_scales;
  a.offsets = offsets; a.row_map = row_map;
  // 2^(31+s) / row_div rounded up, 2^s >= row_div: the quotients of 31-bit numbers are exact
  int s = 0;
  while (((int64_t)1 << s) < row_div) ++s;
  a.div_shift = 31 + s;
  a.div_mul = (uint32_t)((((uint64_t)1 << (31 + s)) + (uint64_t)row_div - 1) / (uint64_t)row_div);
  a.c = c; a.ldc = ldc; a.c_bf16 = c_type == MOE_TYPE_BF16;
  a.a_rows = a_rows; a.a_fp8 = a_format == MOE_MX_FP8;
  a.E = E; a.N = N; a.K = K; a.KB = (int)kb; a.rows = rows;
  return launched(launch_mx4_product(a, stream));
}

}  // extern "C"

namespace {

static_assert(sizeof(moe_tensor) == sizeof(GradTensor) && offsetof(moe_tensor, out) == offsetof(GradTensor, out) &&
                  offsetof(moe_tensor, n) == offsetof(GradTensor, n) &&
                  offsetof(moe_tensor, type) == offsetof(GradTensor, type),
              "the kernels' view of moe_tensor");

// `written`: the call writes `out` (in place where it is NULL or data), so no
// byte of an output may belong to another output or to another gradient, and
// no gradient may be there twice; without it the gradients are only read.
moe_status check_tensors(const moe_tensor* t, int32_t count, bool written) {
  if (count < 0) return MOE_ERR_DIMS;
  if (count > 0 && !t) return MOE_ERR_NULL;
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].n < 0 || t[i].n > ((int64_t)1 << 40)) return MOE_ERR_DIMS;
    total += t[i].n;
    if (total > ((int64_t)1 << 40)) return MOE_ERR_DIMS;   // (the kernels count chunks of them in 32 bits)
    if (!type_ok(t[i].type)) return MOE_ERR_UNSUPPORTED;
    if (t[i].n == 0) continue;
    if (!t[i].data) return MOE_ERR_NULL;
    if (!aligned_to(t[i].data, type_size(t[i].type)) || !aligned_to(t[i].out, type_size(t[i].type)))
      return MOE_ERR_ALIGN;
  }
  if (!written) return MOE_OK;
  // byte ranges of the gradients, and of outputs elsewhere: no two may overlap
  struct Range { uintptr_t lo, hi; };
  try {
    std::vector<Range> r;
    r.reserve(2 * (size_t)count);
    for (int32_t i = 0; i < count; ++i) {
      const uintptr_t bytes = (uintptr_t)t[i].n * type_size(t[i].type);
      if (bytes == 0) continue;
      const uintptr_t d = reinterpret_cast<uintptr_t>(t[i].data), o = reinterpret_cast<uintptr_t>(t[i].out);
      r.push_back({d, d + bytes});
      if (o && o != d) r.push_back({o, o + bytes});
    }
    auto less = [](const Range& a, const Range& b) { return a.lo < b.lo; };
    if (!std::is_sorted(r.begin(), r.end(), less)) std::sort(r.begin(), r.end(), less);
    for (size_t i = 1; i < r.size(); ++i)
      if (r[i].lo < r[i - 1].hi) return MOE_ERR_UNSUPPORTED;
  } catch (const std::bad_alloc&) {
    return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_grad_workspace_size(int32_t count, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  if (count < 0) return MOE_ERR_DIMS;
  *bytes = grad_ws_bytes(count);
  return MOE_OK;
}

moe_status moe_grad_norm(const moe_tensor* tensors, int32_t count, double* sumsq, void* ws, size_t ws_bytes,
                         hipStream_t stream) {
  const moe_status st = check_tensors(tensors, count, false);
  if (st != MOE_OK) return st;
  if (!sumsq || (count > 0 && !ws)) return MOE_ERR_NULL;
  if (!aligned_to(sumsq, 8) || !aligned_to(ws, 256)) return MOE_ERR_ALIGN;
  if (ws_bytes < grad_ws_bytes(count)) return MOE_ERR_WORKSPACE;
  return launched(launch_grad_sumsq(reinterpret_cast<const GradTensor*>(tensors), count, sumsq,
                                    static_cast<double*>(ws), stream));
}

moe_status moe_grad_clip(const moe_tensor* tensors, int32_t count, const double* sumsq, float max_norm,
                         float* norm_out, hipStream_t stream) {
  const moe_status st = check_tensors(tensors, count, true);
  if (st != MOE_OK) return st;
  if (!sumsq) return MOE_ERR_NULL;
  if (!(max_norm >= 0.f)) return MOE_ERR_DIMS;   // NaN among them
  if (!aligned_to(sumsq, 8) || !aligned_to(norm_out, 4)) return MOE_ERR_ALIGN;
  return launched(launch_grad_clip(reinterpret_cast<const GradTensor*>(tensors), count, sumsq, max_norm, norm_out,
                                   stream));
}

}  // extern "C"
