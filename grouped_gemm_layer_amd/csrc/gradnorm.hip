// Norm of many gradient tensors and clipping by it, for the step's end (the
// fp32 main gradients of the accumulating backward and whatever else the step
// trains).
//   sumsq = sum over all tensors of g^2,  out = g * min(1, max_norm / sqrt(sumsq))
// Bound by HBM: one read for the norm, one read and one write for the clipping.
// The tensors' addresses travel in the kernel arguments, TENSORS_PER_LAUNCH a
// launch, cut into chunks of GRAD_CHUNK values.  Squares are summed in fp64: no
// square of an fp32 value overflows or vanishes there, and the vector units'
// fp64 rate is still several times what HBM delivers.  Every sum has a fixed
// order (no atomics).
//
// 604 million fp32 values in six tensors: 353 us for the norm (6.8 TB/s), 787
// for the clipping (6.1 TB/s of reads and writes).  Both pass the caches by:
// with plain loads the norm took 400 us.  The clipping has a thread block for
// every chunk, 4096 values, the fastest of what was tried: 2048 blocks that take
// chunks in turn 882 us, 8192 blocks 850; chunks of 8192 values 880, of 2048
// the same for fp32 but 5% slower in the norm, which sums per block and so has
// blocks that take several.
#include "moe_internal.h"
#include "row_vec.h"

namespace moe {
namespace {

constexpr int TENSORS_PER_LAUNCH = 128;     // 3.6 KB of kernel arguments
constexpr int GRAD_CHUNK = 4096;            // values per chunk
constexpr int NORM_BLOCKS = 4096;           // thread blocks of the norm's launch at most, one partial sum each
constexpr int CLIP_BLOCKS = 1 << 23;        // of the clipping's: a launch has fewer than 2^32 threads

struct TensorTable {
  const void* data[TENSORS_PER_LAUNCH];
  void* out[TENSORS_PER_LAUNCH];
  int64_t n[TENSORS_PER_LAUNCH];            // values; ~values for a bf16 tensor
  uint32_t chunk0[TENSORS_PER_LAUNCH];      // first chunk of the tensor
  int count;
  uint32_t chunks;                          // the host checks that all values give fewer than 2^31
};
static_assert(sizeof(TensorTable) <= 3800, "kernel arguments stay below 4 KB");

__device__ __forceinline__ int find_tensor(const TensorTable& t, uint32_t chunk) {   // uniform over the block
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.chunk0[mid] <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ double chunk_sumsq(const T* p, int64_t n) {
  constexpr int V = RowVec<T>::N, U = 4;
  double s[U] = {0.0, 0.0, 0.0, 0.0};
  for (int64_t i0 = (int64_t)threadIdx.x * V; i0 < n; i0 += 256 * V * U) {
    RowVec<T> v[U];
    int m[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + (int64_t)u * 256 * V;
      m[u] = (int)min((int64_t)V, n - i);
      if (m[u] > 0) v[u] = RowVec<T>::load_once(p + i, m[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (m[u] > 0) {
        float f[V];
        v[u].unpack(f);
#pragma unroll
        for (int i = 0; i < V; ++i) s[u] = fma((double)f[i], (double)f[i], s[u]);
      }
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// sum over the block's 256 threads, in thread 0
__device__ __forceinline__ double block_sum(double v, double* s_w) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  if ((threadIdx.x & 63) == 0) s_w[threadIdx.x >> 6] = v;
  __syncthreads();
  return (s_w[0] + s_w[1]) + (s_w[2] + s_w[3]);
}

__global__ __launch_bounds__(256) void grad_sumsq_kernel(TensorTable t, double* __restrict__ partials) {
  __shared__ double s_w[4];
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int k = find_tensor(t, c);
    const bool bf16 = t.n[k] < 0;
    const int64_t i0 = (int64_t)(c - t.chunk0[k]) * GRAD_CHUNK;
    const int64_t n = min((int64_t)GRAD_CHUNK, (bf16 ? ~t.n[k] : t.n[k]) - i0);
    s += bf16 ? chunk_sumsq(static_cast<const bf16_t*>(t.data[k]) + i0, n)
              : chunk_sumsq(static_cast<const float*>(t.data[k]) + i0, n);
  }
  s = block_sum(s, s_w);
  if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

__global__ __launch_bounds__(256) void grad_total_kernel(const double* __restrict__ partials, int n,
                                                         double* __restrict__ sumsq) {
  __shared__ double s_w[4];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 256) s += partials[i];
  s = block_sum(s, s_w);
  if (threadIdx.x == 0) *sumsq = s;
}

// out = f * g, or g as it is when the factor is 1 (in place: nothing to do)
template <typename T>
__device__ __forceinline__ void chunk_scale(const T* p, T* o, int64_t n, float f, bool scale) {
  constexpr int V = RowVec<T>::N, U = 4;
  for (int64_t i0 = (int64_t)threadIdx.x * V; i0 < n; i0 += 256 * V * U) {
    RowVec<T> v[U];
    int m[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + (int64_t)u * 256 * V;
      m[u] = (int)min((int64_t)V, n - i);
      if (m[u] > 0) v[u] = RowVec<T>::load_once(p + i, m[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (m[u] > 0) {
        if (scale) {
          float x[V];
          v[u].unpack(x);
#pragma unroll
          for (int i = 0; i < V; ++i) x[i] *= f;
          v[u] = RowVec<T>::pack(x);
        }
        v[u].store_once(o + i0 + (int64_t)u * 256 * V, m[u]);
      }
  }
}

__global__ __launch_bounds__(256) void grad_clip_kernel(TensorTable t, const double* __restrict__ sumsq,
                                                        float max_norm, float* __restrict__ norm_out) {
  const double norm = sqrt(*sumsq);
  const bool scale = norm > (double)max_norm && norm <= 1.7976931348623157e308;   // a norm that is not finite clips nothing
  const float f = scale ? (float)((double)max_norm / norm) : 1.f;
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int k = find_tensor(t, c);
    if (!scale && t.out[k] == t.data[k]) continue;
    const bool bf16 = t.n[k] < 0;
    const int64_t i0 = (int64_t)(c - t.chunk0[k]) * GRAD_CHUNK;
    const int64_t n = min((int64_t)GRAD_CHUNK, (bf16 ? ~t.n[k] : t.n[k]) - i0);
    if (bf16)
      chunk_scale(static_cast<const bf16_t*>(t.data[k]) + i0, static_cast<bf16_t*>(t.out[k]) + i0, n, f, scale);
    else
      chunk_scale(static_cast<const float*>(t.data[k]) + i0, static_cast<float*>(t.out[k]) + i0, n, f, scale);
  }
}

// The next launch's tensors from position `at` on (empty ones left out).
TensorTable next_table(const GradTensor* tensors, int count, int& at) {
  TensorTable t{};
  while (at < count && t.count < TENSORS_PER_LAUNCH) {
    const GradTensor& g = tensors[at++];
    if (g.n == 0) continue;
    const int k = t.count++;
    t.data[k] = g.data;
    t.out[k] = g.out ? g.out : const_cast<void*>(g.data);
    t.n[k] = g.type == 1 ? ~g.n : g.n;
    t.chunk0[k] = t.chunks;
    t.chunks += (uint32_t)((g.n + GRAD_CHUNK - 1) / GRAD_CHUNK);
  }
  return t;
}
int table_grid(const TensorTable& t, uint32_t most) { return (int)(t.chunks < most ? t.chunks : most); }

}  // namespace

size_t grad_ws_bytes(int count) {
  const int64_t launches = ((int64_t)count + TENSORS_PER_LAUNCH - 1) / TENSORS_PER_LAUNCH;
  return (size_t)launches * NORM_BLOCKS * sizeof(double);
}

hipError_t launch_grad_sumsq(const GradTensor* tensors, int count, double* sumsq, double* ws, hipStream_t s) {
  int n = 0;
  for (int at = 0; at < count;) {
    const TensorTable t = next_table(tensors, count, at);
    if (t.count == 0) break;
    const int grid = table_grid(t, NORM_BLOCKS);
    const hipError_t e = launch_kernel(grad_sumsq_kernel, dim3(grid), dim3(256), 0, s, t, ws + n);
    if (e != hipSuccess) return e;
    n += grid;
  }
  return launch_kernel(grad_total_kernel, dim3(1), dim3(256), 0, s, (const double*)ws, n, sumsq);
}

hipError_t launch_grad_clip(const GradTensor* tensors, int count, const double* sumsq, float max_norm,
                            float* norm_out, hipStream_t s) {
  int at = 0;
  do {   // at least one launch, which writes the norm
    const TensorTable t = next_table(tensors, count, at);
    if (t.count == 0 && norm_out == nullptr) break;
    const int grid = t.chunks > 0 ? table_grid(t, CLIP_BLOCKS) : 1;
    const hipError_t e =
        launch_kernel(grad_clip_kernel, dim3(grid), dim3(256), 0, s, t, sumsq, max_norm, norm_out);
    if (e != hipSuccess) return e;
    norm_out = nullptr;
  } while (at < count);
  return hipSuccess;
}

}  // namespace moe
