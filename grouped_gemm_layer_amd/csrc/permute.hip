// Tokens sorted by expert, and token rows to the experts and back, with
// weights and gradients, as calls of their own (TE dropless-MoE page, "03":
// permute and unpermute around the experts; inside the layer they are folded
// into the GEMMs).
//
//   sort:     stable sort of the flat slots t*k+j by expert, slots without an
//             expert behind the last
//   scatter:  dst[r] = w src[t]           (permute; unpermute's row gradient)
//   gather:   out[t] = sum_j w rows[r]    (unpermute; permute's gradient)
// with r = f2s[t*k+j], and optionally the dots <token row, expert row> that
// are the weights' gradient, taken while the rows pass.  Both walk the
// tokens: a token's row is read or written once and its k expert rows once,
// which is the least traffic, and only f2s is needed.  All are bound by HBM:
// 16384 tokens, top-8 of 128 experts, H = 2048, bf16: sort 10 us (the rows
// kernels move 40 times its bytes), permute 104 us (5.8 TB/s), its gradient
// and unpermute 106 (5.7), unpermute's gradient with the dots 207 (5.5).
// Rows of the experts pass the caches by, token rows do not (with non-temporal
// loads of these the permute took 240 us with its gradient, not 221; with plain
// loads of those 245).
#include "moe_internal.h"
#include "row_vec.h"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------
// Buckets: the E experts, then bucket E for the slots without one, so that
// every slot has a place and the same code serves both.
constexpr int SORT_MAX_E = 512;
constexpr int SORT_NB = SORT_MAX_E + 1;
constexpr int SORT_THREADS = 1024;
constexpr int SORT_WAVES = SORT_THREADS / 64;
constexpr int SORT_ONE = 4096;       // slots up to which one block does everything
constexpr int SORT_MAX_BLOCKS = 256; // every block reads all blocks' counts: their number stays bounded

__device__ __forceinline__ int sort_key(int e, int E) { return (uint32_t)e < (uint32_t)E ? e : E; }

// Bucket counts of the block's chunk of slots (LDS atomics only count).
__device__ __forceinline__ void chunk_counts(const int32_t* idx, int64_t f0, int64_t f1, int E, int* s_hist) {
  for (int e = threadIdx.x; e <= E; e += SORT_THREADS) s_hist[e] = 0;
  __syncthreads();
  for (int64_t f = f0 + threadIdx.x; f < f1; f += SORT_THREADS) atomicAdd(&s_hist[sort_key(idx[f], E)], 1);
  __syncthreads();
}

__global__ __launch_bounds__(SORT_THREADS) void sort_count_kernel(const int32_t* __restrict__ idx, int64_t M, int E,
                                                                  int64_t chunk, int32_t* __restrict__ partials) {
  __shared__ int s_hist[SORT_NB];
  const int64_t f0 = blockIdx.x * chunk;
  chunk_counts(idx, f0, min(M, f0 + chunk), E, s_hist);
  for (int e = threadIdx.x; e <= E; e += SORT_THREADS) partials[(size_t)blockIdx.x * (E + 1) + e] = s_hist[e];
}

// Places of the chunk's slots.  A slot's row = first row of its bucket + the
// bucket's slots in earlier chunks + its rank among the chunk's earlier slots,
// which comes from wave ballots over the bucket's bits (equal keys in lower
// lanes) and the counts of the waves before.  ONE: a single block, which
// counts its slots itself; else the counts of all blocks are in `partials`
// and every block sums them (bucket totals and its own prefix), which costs
// less than a launch in between (blocks <= 256: 132 KB from L2 at E = 128).
template <bool ONE>
__global__ __launch_bounds__(SORT_THREADS) void sort_place_kernel(const int32_t* __restrict__ idx, int64_t M, int E,
                                                                  int ebits, int64_t chunk,
                                                                  const int32_t* __restrict__ partials,
                                                                  int32_t* __restrict__ counts,
                                                                  int32_t* __restrict__ offsets,
                                                                  int32_t* __restrict__ s2f,
                                                                  int32_t* __restrict__ f2s) {
  __shared__ int s_run[SORT_NB];               // next row of each bucket
  __shared__ int s_wc[SORT_WAVES][SORT_NB];    // a round's slots of each wave and bucket
  __shared__ int s_sum[SORT_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int NB = E + 1;
  const int64_t f0 = blockIdx.x * chunk, f1 = min(M, f0 + chunk);
  int total = 0, before = 0;                   // of bucket `tid`: all slots, those of earlier chunks
  if constexpr (ONE) {
    chunk_counts(idx, f0, f1, E, s_run);
    if (tid < NB) total = s_run[tid];
  } else {
    // the blocks' counts by up to 8 groups of NB threads, 16 loads at a time: 128 blocks of 128 experts take 2 rounds
    // of loads, not the 8 of one group (131072 slots with the counting 12.2 -> 9.7 us, 262144 slots 18.0 -> 11.7)
    constexpr int U = 16, GROUPS = SORT_WAVES / 2;
    const int nblk = gridDim.x, me = blockIdx.x;
    const int groups = nblk <= U ? 1 : min(GROUPS, SORT_THREADS / NB), group = tid / NB, e = tid - group * NB;
    auto add_up = [&](auto first, auto step) __attribute__((always_inline)) {   // constants for one group: a scalar loop
      for (int b0 = first; b0 < nblk; b0 += step * U) {
        int c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) c[u] = b0 + u * step < nblk ? partials[(b0 + u * step) * NB + e] : 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          total += c[u];
          if (b0 + u * step < me) before += c[u];
        }
      }
    };
    if (group < groups) {
      if (groups == 1) add_up(std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{});
      else add_up(group, groups);
    }
    if (groups > 1) {
      if (group < groups) {
        s_wc[group][e] = total;
        s_wc[GROUPS + group][e] = before;
      }
      __syncthreads();
      total = before = 0;
      if (tid < NB)
        for (int i = 0; i < groups; ++i) {
          total += s_wc[i][tid];
          before += s_wc[GROUPS + i][tid];
        }
      __syncthreads();                         // (s_wc is cleared below)
    }
  }
  // exclusive prefix of the totals over the buckets: within waves, then over the waves
  int inc = total;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(inc, off);
    if (lane >= off) inc += o;
  }
  if (lane == 63) s_sum[wave] = inc;
  for (int i = tid; i < SORT_WAVES * NB; i += SORT_THREADS) s_wc[i / NB][i % NB] = 0;
  __syncthreads();
  int first = inc - total;
  for (int w = 0; w < wave; ++w) first += s_sum[w];
  if (tid < NB) {
    s_run[tid] = first + before;
    if (blockIdx.x == 0) {
      offsets[tid] = first;                    // offsets[E] = rows with an expert
      if (tid < E) counts[tid] = total;
    }
  }
  __syncthreads();
  const uint64_t lt_mask = (1ull << lane) - 1;
  for (int64_t fr = f0; fr < f1; fr += SORT_THREADS) {
    const int64_t f = fr + tid;
    const bool valid = f < f1;
    const int e = valid ? sort_key(idx[f], E) : 0;
    uint64_t same = __ballot(valid);
    for (int b = 0; b < ebits; ++b) {
      const bool bit = (e >> b) & 1;
      const uint64_t ones = __ballot(bit);
      same &= bit ? ones : ~ones;
    }
    const int rank = __popcll(same & lt_mask);
    if (valid && rank == 0) s_wc[wave][e] = __popcll(same);
    __syncthreads();
    if (valid) {
      int pos = s_run[e] + rank;
      for (int w = 0; w < wave; ++w) pos += s_wc[w][e];
      s2f[pos] = e < E ? (int32_t)f : -1;
      f2s[f] = e < E ? pos : -1;
    }
    if (fr + SORT_THREADS >= f1) break;        // uniform over the block
    __syncthreads();
    for (int b = tid; b < NB; b += SORT_THREADS) {
      int sum = 0;
#pragma unroll
      for (int w = 0; w < SORT_WAVES; ++w) {
        sum += s_wc[w][b];
        s_wc[w][b] = 0;
      }
      s_run[b] += sum;
    }
    __syncthreads();
  }
}

// slots per block: whole rounds of a block, at most SORT_MAX_BLOCKS blocks
int64_t sort_chunk(int64_t M) {
  if (M <= SORT_ONE) return SORT_ONE;
  const int64_t per = (M + SORT_MAX_BLOCKS - 1) / SORT_MAX_BLOCKS;
  return (per + SORT_THREADS - 1) / SORT_THREADS * SORT_THREADS;
}

// ---------------------------------------------------------------------------
// Rows
// ---------------------------------------------------------------------------
constexpr int JG = 8;   // slots handled together (one batch of row loads)

// Sums of v[0..JG) over the waves of a token (WPT of them), every lane of the
// first wave gets them.  s: [4][JG] floats of LDS.
template <int WPT>
__device__ __forceinline__ void token_sums(float (&v)[JG], float (*s)[JG], int lane, int wave) {
#pragma unroll
  for (int j = 0; j < JG; ++j) v[j] = wave_sum(v[j]);
  if constexpr (WPT > 1) {
    __syncthreads();                           // the previous group's sums have been read
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < JG; ++j) s[wave][j] = v[j];
    }
    __syncthreads();
    const int w0 = wave / WPT * WPT;
#pragma unroll
    for (int j = 0; j < JG; ++j) {
      v[j] = s[w0][j];
#pragma unroll
      for (int w = 1; w < WPT; ++w) v[j] += s[w0 + w][j];
    }
  }
}

// rows and weights of slots j0 .. j0+JG-1 of token t (wave-uniform): row -1 and
// weight 0 for a slot without a row
__device__ __forceinline__ void load_slots(const int32_t* f2s, const float* weights, int64_t t, int k, int j0,
                                           int rows, bool live, int (&r)[JG], float (&w)[JG]) {
#pragma unroll
  for (int j = 0; j < JG; ++j) {
    const bool in = live && j0 + j < k;
    const int row = in ? f2s[t * k + j0 + j] : -1;
    r[j] = (uint32_t)row < (uint32_t)rows ? row : -1;
    w[j] = r[j] < 0 ? 0.f : weights ? weights[t * k + j0 + j] : 1.f;
  }
}

template <int WPT>
__device__ __forceinline__ void store_dots(float (&d)[JG], float* dweights, int64_t t, int k, int j0, bool live,
                                           int tl) {
#pragma unroll
  for (int j = 0; j < JG; ++j)
    if (live && tl == j && j0 + j < k) dweights[t * k + j0 + j] = d[j];
}

// WPT waves per token, 4 / WPT tokens per block; grid.y pieces of the row
// (pieces > 1 only without dots).  WEIGHTED = false copies bits.
template <typename T, int WPT, bool WEIGHTED, bool DOT>
__global__ __launch_bounds__(256) void scatter_rows_kernel(const T* __restrict__ src, int64_t lds, int T_, int H,
                                                           int k, const int32_t* __restrict__ f2s,
                                                           const float* __restrict__ weights,
                                                           const T* __restrict__ other, int64_t ldo,
                                                           T* __restrict__ dst, int64_t ldd, int rows,
                                                           float* __restrict__ dweights) {
  constexpr int V = RowVec<T>::N;
  __shared__ float s_dot[4][JG];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * (4 / WPT) + wave / WPT;
  const bool live = t < T_;
  const int tl = (wave % WPT) * 64 + lane;
  const T* row = src + (live ? t : 0) * lds;
  for (int j0 = 0; j0 < k; j0 += JG) {
    int r[JG];
    float w[JG], d[JG];
    load_slots(f2s, weights, t, k, j0, rows, live, r, w);
#pragma unroll
    for (int j = 0; j < JG; ++j) d[j] = 0.f;
    if (live) {
      for (int64_t h = ((int64_t)blockIdx.y * WPT * 64 + tl) * V; h < H; h += (int64_t)gridDim.y * WPT * 64 * V) {
        const int n = (int)min((int64_t)V, H - h);
        const RowVec<T> x = RowVec<T>::load(row + h, n);
        float xf[V];
        if constexpr (WEIGHTED || DOT) x.unpack(xf);
        if constexpr (DOT) {
          RowVec<T> o[JG];
#pragma unroll
          for (int j = 0; j < JG; ++j)
            if (r[j] >= 0) o[j] = RowVec<T>::load_once(other + (int64_t)r[j] * ldo + h, n);
#pragma unroll
          for (int j = 0; j < JG; ++j)
            if (r[j] >= 0) {
              float of[V];
              o[j].unpack(of);
#pragma unroll
              for (int i = 0; i < V; ++i) d[j] += xf[i] * of[i];
            }
        }
#pragma unroll
        for (int j = 0; j < JG; ++j) {
          if (r[j] < 0) continue;
          T* p = dst + (int64_t)r[j] * ldd + h;
          if constexpr (WEIGHTED) {
            float y[V];
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] = w[j] * xf[i];
            RowVec<T>::pack(y).store_once(p, n);
          } else {
            x.store_once(p, n);
          }
        }
      }
    }
    if constexpr (DOT) {
      token_sums<WPT>(d, s_dot, lane, wave);
      store_dots<WPT>(d, dweights, t, k, j0, live, tl);
    }
  }
}

// As above.  Up to JG slots the rows pass once for sum and dots together;
// with more the dots take a pass of their own, from the caches.
template <typename T, int WPT, bool DOT>
__global__ __launch_bounds__(256) void gather_rows_kernel(const T* __restrict__ src, int64_t lds, int rows, int T_,
                                                          int H, int k, const int32_t* __restrict__ f2s,
                                                          const float* __restrict__ weights,
                                                          const T* __restrict__ x, int64_t ldx, T* __restrict__ out,
                                                          int64_t ldo, float* __restrict__ dweights) {
  constexpr int V = RowVec<T>::N;
  __shared__ float s_dot[4][JG];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * (4 / WPT) + wave / WPT;
  const bool live = t < T_;
  const int tl = (wave % WPT) * 64 + lane;
  const int64_t h0 = ((int64_t)blockIdx.y * WPT * 64 + tl) * V, step = (int64_t)gridDim.y * WPT * 64 * V;
  float d[JG];
#pragma unroll
  for (int j = 0; j < JG; ++j) d[j] = 0.f;
  int r[JG];
  float w[JG];
  load_slots(f2s, weights, t, k, 0, rows, live, r, w);
  if (live) {
    for (int64_t h = h0; h < H; h += step) {
      const int n = (int)min((int64_t)V, H - h);
      float acc[V], xf[V];
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = 0.f;
      if constexpr (DOT) RowVec<T>::load(x + t * ldx + h, n).unpack(xf);
      for (int j0 = 0; j0 < k; j0 += JG) {
        if (k > JG) load_slots(f2s, weights, t, k, j0, rows, live, r, w);
        RowVec<T> o[JG];
#pragma unroll
        for (int j = 0; j < JG; ++j)
          if (r[j] >= 0) o[j] = RowVec<T>::load_once(src + (int64_t)r[j] * lds + h, n);
#pragma unroll
        for (int j = 0; j < JG; ++j)
          if (r[j] >= 0) {
            float of[V];
            o[j].unpack(of);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += w[j] * of[i];
            if constexpr (DOT) {
              if (k <= JG) {
#pragma unroll
                for (int i = 0; i < V; ++i) d[j] += xf[i] * of[i];
              }
            }
          }
      }
      RowVec<T>::pack(acc).store_once(out + t * ldo + h, n);
    }
  }
  if constexpr (DOT) {
    if (k <= JG) {
      token_sums<WPT>(d, s_dot, lane, wave);
      store_dots<WPT>(d, dweights, t, k, 0, live, tl);
      return;
    }
    for (int j0 = 0; j0 < k; j0 += JG) {
      load_slots(f2s, weights, t, k, j0, rows, live, r, w);
#pragma unroll
      for (int j = 0; j < JG; ++j) d[j] = 0.f;
      if (live) {
        for (int64_t h = h0; h < H; h += step) {
          const int n = (int)min((int64_t)V, H - h);
          float xf[V];
          RowVec<T>::load(x + t * ldx + h, n).unpack(xf);
#pragma unroll
          for (int j = 0; j < JG; ++j)
            if (r[j] >= 0) {
              float of[V];
              RowVec<T>::load(src + (int64_t)r[j] * lds + h, n).unpack(of);
#pragma unroll
              for (int i = 0; i < V; ++i) d[j] += xf[i] * of[i];
            }
        }
      }
      token_sums<WPT>(d, s_dot, lane, wave);
      store_dots<WPT>(d, dweights, t, k, j0, live, tl);
    }
  }
}

// Waves per token: as many as the row has 64-lane vectors, up to a block.
// Without dots the rest of a long row goes to further blocks (grid.y), so that
// a few tokens still fill more than a few compute units.
struct RowGrid { int wpt; dim3 grid; };
RowGrid row_grid(int T, int H, int V, bool dot) {
  const int64_t nv = ((int64_t)H + V - 1) / V;
  RowGrid g;
  g.wpt = nv <= 64 ? 1 : nv <= 128 ? 2 : 4;
  const int64_t pieces = dot ? 1 : (nv + 255) / 256;
  g.grid = dim3((unsigned)(((int64_t)T + 4 / g.wpt - 1) / (4 / g.wpt)), (unsigned)(pieces > 16 ? 16 : pieces));
  return g;
}

template <typename T, int WPT>
hipError_t scatter_wpt(const RowsArgs& a, dim3 grid, hipStream_t s) {
  auto go = [&](auto kernel) {
    return launch_kernel(kernel, grid, dim3(256), 0, s, static_cast<const T*>(a.token_in), a.ld_token_in, a.T, a.H,
                         a.k, a.f2s, a.weights, static_cast<const T*>(a.rows_in), a.ld_rows_in,
                         static_cast<T*>(a.rows_out), a.ld_rows_out, a.rows, a.dweights);
  };
  if (a.dweights) return a.weights ? go(scatter_rows_kernel<T, WPT, true, true>)
                                   : go(scatter_rows_kernel<T, WPT, false, true>);
  return a.weights ? go(scatter_rows_kernel<T, WPT, true, false>) : go(scatter_rows_kernel<T, WPT, false, false>);
}

template <typename T, int WPT>
hipError_t gather_wpt(const RowsArgs& a, dim3 grid, hipStream_t s) {
  auto go = [&](auto kernel) {
    return launch_kernel(kernel, grid, dim3(256), 0, s, static_cast<const T*>(a.rows_in), a.ld_rows_in, a.rows, a.T,
                         a.H, a.k, a.f2s, a.weights, static_cast<const T*>(a.token_in), a.ld_token_in,
                         static_cast<T*>(a.token_out), a.ld_token_out, a.dweights);
  };
  return a.dweights ? go(gather_rows_kernel<T, WPT, true>) : go(gather_rows_kernel<T, WPT, false>);
}

template <typename T>
hipError_t launch_rows(const RowsArgs& all, bool scatter, hipStream_t s) {
  constexpr int PART = 1 << 22;   // tokens per launch, which has fewer than 2^32 threads
  for (int64_t t0 = 0; t0 < all.T; t0 += PART) {
    RowsArgs a = all;
    a.T = (int)(all.T - t0 < PART ? all.T - t0 : PART);
    a.f2s += t0 * a.k;
    if (a.weights) a.weights += t0 * a.k;
    if (a.dweights) a.dweights += t0 * a.k;
    if (a.token_in) a.token_in = static_cast<const T*>(a.token_in) + t0 * a.ld_token_in;
    if (a.token_out) a.token_out = static_cast<T*>(a.token_out) + t0 * a.ld_token_out;
    const RowGrid g = row_grid(a.T, a.H, RowVec<T>::N, a.dweights != nullptr);
    const hipError_t e = scatter ? (g.wpt == 1   ? scatter_wpt<T, 1>(a, g.grid, s)
                                    : g.wpt == 2 ? scatter_wpt<T, 2>(a, g.grid, s)
                                                 : scatter_wpt<T, 4>(a, g.grid, s))
                                 : (g.wpt == 1   ? gather_wpt<T, 1>(a, g.grid, s)
                                    : g.wpt == 2 ? gather_wpt<T, 2>(a, g.grid, s)
                                                 : gather_wpt<T, 4>(a, g.grid, s));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t sort_ws_bytes(int64_t M, int E) {
  if (M <= SORT_ONE) return 0;
  const int64_t chunk = sort_chunk(M);
  return (size_t)((M + chunk - 1) / chunk) * (E + 1) * 4;
}

hipError_t launch_sort(const int32_t* idx, int64_t M, int E, int32_t* counts, int32_t* offsets, int32_t* s2f,
                       int32_t* f2s, int32_t* ws, hipStream_t s) {
  int ebits = 0;
  while ((1 << ebits) < E + 1) ++ebits;
  const int64_t chunk = sort_chunk(M);
  if (M <= SORT_ONE)
    return launch_kernel(sort_place_kernel<true>, dim3(1), dim3(SORT_THREADS), 0, s, idx, M, E, ebits, chunk, nullptr,
                         counts, offsets, s2f, f2s);
  const int nblk = (int)((M + chunk - 1) / chunk);
  const hipError_t e =
      launch_kernel(sort_count_kernel, dim3(nblk), dim3(SORT_THREADS), 0, s, idx, M, E, chunk, ws);
  if (e != hipSuccess) return e;
  return launch_kernel(sort_place_kernel<false>, dim3(nblk), dim3(SORT_THREADS), 0, s, idx, M, E, ebits, chunk,
                       (const int32_t*)ws, counts, offsets, s2f, f2s);
}

hipError_t launch_scatter_rows(const RowsArgs& a, int type, hipStream_t s) {
  return type == 0 ? launch_rows<float>(a, true, s) : launch_rows<bf16_t>(a, true, s);
}
hipError_t launch_gather_rows(const RowsArgs& a, int type, hipStream_t s) {
  return type == 0 ? launch_rows<float>(a, false, s) : launch_rows<bf16_t>(a, false, s);
}

}  // namespace moe
