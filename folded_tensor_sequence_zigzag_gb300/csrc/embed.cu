// embed.cu -- token embedding into the zigzag rank-major order, and the
// gradient of its table.
//
//   forward   x[row(p)] = round(scale * E[id[p]])
//   backward  dE[v] (+)= scale * sum over the positions p with id[p] == v of dx[row(p)]
//
// row(p) is the zigzag row of global position p (common.cuh); with D = 1 the
// order is the global one and S may be odd.  An id below 0 is padding: its row
// is zero and it has no gradient.  An id >= V is treated the same way and
// recorded as TSP_ERR_RANGE.  Both directions are bound by HBM: the forward
// reads the distinct table rows and writes S rows, the backward reads S rows
// and writes V.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace tsp {

namespace {

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

__device__ __forceinline__ int64_t load_id(const void* ids, int id_bytes, int64_t p) {
  return id_bytes == 8 ? (int64_t)reinterpret_cast<const long long*>(ids)[p]
                       : (int64_t)reinterpret_cast<const int*>(ids)[p];
}
// c = S / (2D); D == 1 is the identity for every S
__device__ __forceinline__ int row_of(int p, int c, int D) {
  return D == 1 ? p : zz_row_of_pos32(p, c, D);
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------

// One unit of a row scaled in fp32 and rounded once to the table's type.
template <typename T>
__device__ __forceinline__ T scaled(T v, float s) {
  return from_f<T>(to_f<T>(v) * s);
}
template <typename T, typename V>
__device__ __forceinline__ V scale_unit(V u, float s) {
  constexpr int N = sizeof(V) / sizeof(T);
  T e[N];
  memcpy(e, &u, sizeof(V));
#pragma unroll
  for (int i = 0; i < N; ++i) e[i] = scaled<T>(e[i], s);
  memcpy(&u, e, sizeof(V));
  return u;
}

// One warp per (position, segment of 128 units of V bytes): four loads in
// flight a lane.
template <typename T, typename V>
__global__ void __launch_bounds__(256) embed_fwd_kernel(const void* __restrict__ ids, int id_bytes,
                                                        const V* __restrict__ table,
                                                        V* __restrict__ x, int S, int c, int D,
                                                        int64_t vocab, int upr, int nseg,
                                                        float scale, int* __restrict__ status) {
  const int lane = threadIdx.x & 31;
  const int64_t items = (int64_t)S * nseg, stride = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t it = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items;
       it += stride) {
    const int p = (int)(it / nseg), seg = (int)(it - (int64_t)p * nseg);
    const int64_t id = load_id(ids, id_bytes, p);
    const int row = row_of(p, c, D);
    if (!TSP_INB(row >= 0 && row < S, status)) continue;
    if (id >= vocab && lane == 0) report_status(status, (int)TSP_ERR_RANGE);
    const bool there = id >= 0 && id < vocab;
    const V* src = table + (there ? id : 0) * upr;
    V* dst = x + (int64_t)row * upr;
    V v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = seg * 128 + k * 32 + lane;
      v[k] = V{};
      if (there && u < upr) v[k] = src[u];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = seg * 128 + k * 32 + lane;
      if (u < upr) dst[u] = scale == 1.f ? v[k] : scale_unit<T, V>(v[k], scale);
    }
  }
}

template <typename T, typename V>
tsp_status embed_fwd_t(const void* ids, int id_bytes, const void* table, void* x, int64_t S, int D,
                       int64_t vocab, int d, float scale, cudaStream_t st) {
  const int upr = (int)((int64_t)d * sizeof(T) / sizeof(V));
  const int nseg = (upr + 127) / 128;
  const int64_t ctas = (S * nseg + 7) / 8;
  const int grid = (int)std::min<int64_t>(ctas, (int64_t)num_sms() * 8);
  Prof prof("embed_fwd", st);
  embed_fwd_kernel<T, V><<<grid, 256, 0, st>>>(ids, id_bytes, (const V*)table, (V*)x, (int)S,
                                               (int)(S / (2 * D)), D, vocab, upr, nseg, scale,
                                               status_word());
  TSP_CUDA_TRY(cudaGetLastError());
  return TSP_OK;
}

// ---------------------------------------------------------------------------
// Backward, step 1: the positions sorted by token, and the rows of absent tokens
// ---------------------------------------------------------------------------
// The first cluster of the grid sorts (token, zigzag row) by a stable
// least-significant-digit radix sort: every CTA of it owns a contiguous range of
// the positions, every warp a contiguous part of that.  A pass counts digits per
// warp in shared memory, turns the counts into places (over warps, then over the
// cluster's CTAs through distributed shared memory, then over digits) and
// scatters.  Equal tokens keep the order of their positions, so the sums of
// step 2 have one fixed order.  Ids outside the table sort to the end as token
// `vocab`.  The sort is a few microseconds of latency on eight multiprocessors;
// meanwhile the CTAs of the other clusters write the zero rows: each owns the
// tokens v with v % zero_ctas equal to its number, and marks those that occur in
// a bitmap of its own by reading all ids (from L2).
constexpr int kBits = 9, kBins = 1 << kBits, kSortWarps = 32, kMaxCluster = 8;
constexpr int kSortSmem = kSortWarps * kBins * 4;
constexpr int kBatch = 8;   // positions a lane loads before it uses the first

struct SortArgs {
  const void* ids;
  int id_bytes;
  int S, c, D, vocab, d;
  int passes, bits;
  int *key[2], *row[2];   // the last pass writes key[passes & 1], row[passes & 1]
  float* table;
  int zero_shift;         // log2 of the CTAs that write zeros, -1: none
  int* status;
};

template <bool VEC>
__device__ void zero_absent_rows(const SortArgs& a, int me, int* bitmap) {
  const int shift = a.zero_shift, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int mine = (int)(((int64_t)a.vocab - me + (1 << shift) - 1) >> shift);   // my tokens
  constexpr int kCap = kSortSmem * 8;                                            // marked at a time
  for (int first = 0; first < mine; first += kCap) {
    const int count = min(kCap, mine - first);
    for (int i = t; i < (count + 31) / 32; i += blockDim.x) bitmap[i] = 0;
    __syncthreads();
    for (int p = t; p < a.S; p += kBatch * blockDim.x) {
      int64_t id[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int q = p + k * (int)blockDim.x;
        id[k] = q < a.S ? load_id(a.ids, a.id_bytes, q) : -1;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (id[k] < 0 || id[k] >= a.vocab || ((int)id[k] & ((1 << shift) - 1)) != me) continue;
        const int i = ((int)id[k] >> shift) - first;
        if (i >= 0 && i < count) atomicOr(bitmap + (i >> 5), 1 << (i & 31));
      }
    }
    __syncthreads();
    for (int i = warp; i < count; i += kSortWarps) {
      if (bitmap[i >> 5] >> (i & 31) & 1) continue;
      float* row = a.table + (((int64_t)(first + i) << shift) + me) * a.d;
      if constexpr (VEC) {
        for (int c = lane * 4; c < a.d; c += 128)
          *reinterpret_cast<float4*>(row + c) = make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
        for (int c = lane; c < a.d; c += 32) row[c] = 0.f;
      }
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kSortWarps * 32) embed_sort_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ int hist[];                   // [kSortWarps][bins]
  __shared__ int total[kBins], wsum[kSortWarps];
  cg::cluster_group cl = cg::this_cluster();
  const int me = (int)cl.block_rank(), nc = (int)cl.num_blocks();
  if ((int)blockIdx.x >= nc) {
    const int z = (int)blockIdx.x - nc;
    if (z >> a.zero_shift) return;   // (the grid is whole clusters)
    if (a.d % 4 == 0) zero_absent_rows<true>(a, z, hist);
    else zero_absent_rows<false>(a, z, hist);
    return;
  }
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, bins = 1 << a.bits;
  // this warp's positions, in whole groups of 32
  const int64_t groups = ((int64_t)a.S + 31) / 32;
  const int64_t gw = (int64_t)me * kSortWarps + warp, nw = (int64_t)nc * kSortWarps;
  const int g0 = (int)(groups * gw / nw), g1 = (int)(groups * (gw + 1) / nw);
  int* const mine = hist + warp * bins;

  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    const int* key_in = a.key[pass & 1];
    const int* row_in = a.row[pass & 1];
    int* key_out = a.key[(pass & 1) ^ 1];
    int* row_out = a.row[(pass & 1) ^ 1];
    int key[kBatch], row[kBatch];
    auto load_keys = [&](int g) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int p = (g + u) * 32 + lane;
        key[u] = 0;
        if (g + u >= g1 || p >= a.S) continue;
        if (pass > 0) {
          key[u] = __ldcg(key_in + p);
        } else {
          const int64_t id = load_id(a.ids, a.id_bytes, p);
          key[u] = id < 0 ? a.vocab : (int)min(id, (int64_t)a.vocab);
          if (id >= a.vocab) report_status(a.status, (int)TSP_ERR_RANGE);
        }
      }
    };
    // the digit of batch position u, `bins` where there is none
    auto digit_of = [&](int g, int u) {
      return g + u < g1 && (g + u) * 32 + lane < a.S ? (key[u] >> shift) & (bins - 1) : bins;
    };
    for (int i = t; i < kSortWarps * bins; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    for (int g = g0; g < g1; g += kBatch) {
      load_keys(g);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int digit = digit_of(g, u);
        const unsigned same = __match_any_sync(0xffffffffu, digit);
        if (digit < bins && lane == __ffs(same) - 1) mine[digit] += __popc(same);
        __syncwarp();
      }
    }
    __syncthreads();
    int sum = 0;
    if (t < bins) {
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const int n = hist[w * bins + t];
        hist[w * bins + t] = sum;
        sum += n;
      }
      total[t] = sum;
    }
    cl.sync();
    // this digit's count over the cluster, and over the CTAs before this one
    int all = 0, before = 0;
    if (t < bins) {
      for (int j = 0; j < nc; ++j) {
        const int n = cl.map_shared_rank(total, j)[t];
        all += n;
        if (j < me) before += n;
      }
    }
    int inc = all;   // inclusive scan over the digits
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += n;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    if (t < bins) {
      int base = inc - all + before;
      for (int w = 0; w < warp; ++w) base += wsum[w];
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) hist[w * bins + t] += base;
    }
    __syncthreads();
    for (int g = g0; g < g1; g += kBatch) {
      // (one batch a warp: the keys are still there)
      if (g1 - g0 > kBatch) load_keys(g);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int p = (g + u) * 32 + lane;
        row[u] = 0;
        if (g + u < g1 && p < a.S) row[u] = pass > 0 ? __ldcg(row_in + p) : row_of(p, a.c, a.D);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int digit = digit_of(g, u);
        const unsigned same = __match_any_sync(0xffffffffu, digit);
        int at = -1;
        if (digit < bins) at = mine[digit] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (digit < bins && lane == __ffs(same) - 1) mine[digit] += __popc(same);
        __syncwarp();
        if (digit < bins && TSP_INB(at >= 0 && at < a.S, a.status)) {
          __stcg(key_out + at, key[u]);
          __stcg(row_out + at, row[u]);
        }
      }
    }
    cl.sync();   // the pass is written, and no CTA reads `total` any more
  }
}

// ---------------------------------------------------------------------------
// Backward, step 2: rows summed along the sorted order
// ---------------------------------------------------------------------------
// A warp takes a chunk of the sorted positions and a slab of 256 columns (8 a
// lane) and walks the chunk's rows, four loads ahead; places and tokens come 32
// at a time.  A token whose positions lie inside the chunk is written (or added)
// to its table row at once; one that came in from the chunk before leaves its
// part in slot 2*chunk, one that starts here and goes on in slot 2*chunk + 1.
// Step 3 adds those up.
constexpr int kSlab = 256;

template <typename T, bool VEC>
__device__ __forceinline__ void load_cols(const T* row, int c0, int lane, int d, float (&v)[8]) {
  if constexpr (VEC) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 + h * 128 + lane * 4;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < d) {
        if constexpr (sizeof(T) == 4) {
          f = __ldcs(reinterpret_cast<const float4*>(row + c));
        } else {
          const uint2 u = __ldcs(reinterpret_cast<const uint2*>(row + c));
          f = make_float4(lo2<T>(u.x), hi2<T>(u.x), lo2<T>(u.y), hi2<T>(u.y));
        }
      }
      v[4 * h] = f.x; v[4 * h + 1] = f.y; v[4 * h + 2] = f.z; v[4 * h + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = c0 + e * 32 + lane;
      v[e] = c < d ? to_f<T>(row[c]) : 0.f;
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void store_cols(float* row, int c0, int lane, int d, const float (&v)[8],
                                           float s, bool add) {
  if constexpr (VEC) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 + h * 128 + lane * 4;
      if (c >= d) continue;
      float4* p = reinterpret_cast<float4*>(row + c);
      float4 o = make_float4(v[4 * h] * s, v[4 * h + 1] * s, v[4 * h + 2] * s, v[4 * h + 3] * s);
      if (add) {
        const float4 q = *p;
        o = make_float4(q.x + o.x, q.y + o.y, q.z + o.z, q.w + o.w);
      }
      *p = o;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = c0 + e * 32 + lane;
      if (c < d) row[c] = (add ? row[c] : 0.f) + v[e] * s;
    }
  }
}

struct SumArgs {
  const int *key, *row;
  float *table, *part;
  int S, vocab, d, chunk, nchunks, nslabs;
  float scale;
  bool add;   // to the table rows instead of overwriting them
  int* status;
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) embed_sum_kernel(const T* __restrict__ dx,
                                                        const __grid_constant__ SumArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t task = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (task >= (int64_t)a.nchunks * a.nslabs) return;
  const int ch = (int)(task / a.nslabs), c0 = (int)(task - (int64_t)ch * a.nslabs) * kSlab;
  const int j0 = ch * a.chunk, j1 = (int)min((int64_t)a.S, (int64_t)j0 + a.chunk);
  int cur = a.key[j0];
  if (cur >= a.vocab) return;
  bool opened = j0 == 0 || a.key[j0 - 1] != cur;   // the current token's positions start here
  const bool goes_on = j1 < a.S && a.key[j1] == a.key[j1 - 1];
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto leave = [&](bool on) {
    if (opened && !on)
      store_cols<VEC>(a.table + (int64_t)cur * a.d, c0, lane, a.d, acc, a.scale, a.add);
    else
      store_cols<VEC>(a.part + ((int64_t)2 * ch + (opened ? 1 : 0)) * a.d, c0, lane, a.d, acc, 1.f,
                      false);
  };
  for (int j = j0; j < j1; j += 32) {
    const bool in = j + lane < j1;
    const int keys = in ? a.key[j + lane] : a.vocab, rows = in ? a.row[j + lane] : 0;
    for (int k = 0; k < 32 && j + k < j1; k += 4) {
      float v[4][8];
      int key[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        key[u] = __shfl_sync(0xffffffffu, keys, k + u);
        const int r = __shfl_sync(0xffffffffu, rows, k + u);
        if (key[u] < a.vocab && TSP_INB(r >= 0 && r < a.S, a.status)) {
          load_cols<T, VEC>(dx + (int64_t)r * a.d, c0, lane, a.d, v[u]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[u][e] = 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (j + k + u >= j1) break;
        if (key[u] != cur) {
          leave(false);
          cur = key[u];
          opened = true;
          if (cur >= a.vocab) return;   // padding to the end
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += v[u][e];
      }
    }
  }
  leave(goes_on);
}

// Step 3: a token that starts in one chunk and ends in a later one.  A CTA a
// chunk and slab (nearly all see at once that no token starts there and goes
// on); the warps add up every eighth part each, then the eight sums in order.
template <bool VEC>
__global__ void __launch_bounds__(256) embed_join_kernel(const __grid_constant__ SumArgs a) {
  __shared__ float sums[8][kSlab];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ch = (int)(blockIdx.x / a.nslabs), c0 = (int)(blockIdx.x - ch * a.nslabs) * kSlab;
  const int end = (ch + 1) * a.chunk;   // < S: there is a chunk after this one
  const int tok = a.key[end - 1];
  if (tok >= a.vocab || a.key[end] != tok) return;
  const int j0 = ch * a.chunk;
  if (j0 > 0 && a.key[j0] == tok && a.key[j0 - 1] == tok) return;   // it started before this chunk
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (warp == 0) load_cols<float, VEC>(a.part + ((int64_t)2 * ch + 1) * a.d, c0, lane, a.d, acc);
  for (int k = ch + 1 + warp; k < a.nchunks; k += 32) {
    float v[4][8];
    bool in[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int q = k + u * 8;
      in[u] = q < a.nchunks && a.key[q * a.chunk] == tok;
      if (in[u]) load_cols<float, VEC>(a.part + (int64_t)2 * q * a.d, c0, lane, a.d, v[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (!in[u]) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += v[u][e];
    }
    if (!in[3]) break;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[warp][e * 32 + lane] = acc[e];
  __syncthreads();
  if (warp != 0) return;
  for (int w = 1; w < 8; ++w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += sums[w][e * 32 + lane];
  }
  store_cols<VEC>(a.table + (int64_t)tok * a.d, c0, lane, a.d, acc, a.scale, a.add);
}

// Positions per chunk: the smallest power of two, 16 to 64, with which the
// chunks' warps fit the GPU at once (64 a multiprocessor).
int chunk_of(int64_t S, int d) {
  const int64_t slabs = (d + kSlab - 1) / kSlab, warps = 152 * 64;
  int c = 16;
  while (c < 64 && ((S + c - 1) / c) * slabs > warps) c *= 2;
  return c;
}

struct BwdLayout {
  int *key[2], *row[2];
  float* part;
  size_t bytes;
};
BwdLayout bwd_layout(int64_t S, int d, uint8_t* base) {
  BwdLayout L;
  size_t off = 0;
  auto take = [&](size_t n) {
    uint8_t* p = base ? base + off : nullptr;
    off += up256(n);
    return p;
  };
  for (int k = 0; k < 2; ++k) {
    L.key[k] = (int*)take((size_t)S * 4);
    L.row[k] = (int*)take((size_t)S * 4);
  }
  const int c = chunk_of(S, d);
  L.part = (float*)take((size_t)((S + c - 1) / c) * 2 * d * 4);
  L.bytes = off;
  return L;
}

template <typename T, bool VEC>
tsp_status embed_sum_t(const void* dx, const SumArgs& a, cudaStream_t st) {
  const int64_t tasks = (int64_t)a.nchunks * a.nslabs;
  Prof prof("embed_bwd_sum", st, a.nchunks > 1 ? 2 : 1);
  embed_sum_kernel<T, VEC><<<(unsigned)((tasks + 7) / 8), 256, 0, st>>>((const T*)dx, a);
  TSP_CUDA_TRY(cudaGetLastError());
  if (a.nchunks > 1) {
    embed_join_kernel<VEC><<<(unsigned)((a.nchunks - 1) * (int64_t)a.nslabs), 256, 0, st>>>(a);
    TSP_CUDA_TRY(cudaGetLastError());
  }
  return TSP_OK;
}

}  // namespace

tsp_status launch_embed_fwd(const void* ids, int id_bytes, const void* table, void* x, int64_t S,
                            int D, int64_t vocab, int d, float scale, int dtype, cudaStream_t st) {
  const int64_t row_bytes = (int64_t)d * (dtype == TSP_BF16 ? 2 : 4);
  if (dtype == TSP_BF16) {
    typedef __nv_bfloat16 bf;
    if (row_bytes % 16 == 0)
      return embed_fwd_t<bf, uint4>(ids, id_bytes, table, x, S, D, vocab, d, scale, st);
    if (row_bytes % 4 == 0)
      return embed_fwd_t<bf, uint32_t>(ids, id_bytes, table, x, S, D, vocab, d, scale, st);
    return embed_fwd_t<bf, uint16_t>(ids, id_bytes, table, x, S, D, vocab, d, scale, st);
  }
  if (row_bytes % 16 == 0)
    return embed_fwd_t<float, uint4>(ids, id_bytes, table, x, S, D, vocab, d, scale, st);
  return embed_fwd_t<float, uint32_t>(ids, id_bytes, table, x, S, D, vocab, d, scale, st);
}

size_t embed_bwd_ws_bytes(int64_t S, int d) {
  return bwd_layout(S, d, nullptr).bytes;
}

tsp_status launch_embed_bwd(const void* ids, int id_bytes, const void* dx, int dx_dtype,
                            float* dtable, int64_t S, int D, int64_t vocab, int d, float scale,
                            bool accumulate, void* ws, cudaStream_t st) {
  const BwdLayout L = bwd_layout(S, d, (uint8_t*)ws);
  SortArgs s;
  s.ids = ids;
  s.id_bytes = id_bytes;
  s.S = (int)S;
  s.c = (int)(S / (2 * D));
  s.D = D;
  s.vocab = (int)vocab;
  int nb = 1;   // bits of the largest key, `vocab` itself
  while (((int64_t)vocab >> nb) != 0) ++nb;
  s.passes = (nb + kBits - 1) / kBits;
  s.bits = (nb + s.passes - 1) / s.passes;
  for (int k = 0; k < 2; ++k) {
    s.key[k] = L.key[k];
    s.row[k] = L.row[k];
  }
  s.table = dtable;
  s.d = d;
  s.status = status_word();
  // a CTA for every 256 KB of the table writes its absent rows, 128 at most
  s.zero_shift = -1;
  if (!accumulate) {
    s.zero_shift = 0;
    while (s.zero_shift < 7 && ((int64_t)vocab * d * 4 >> s.zero_shift) > 256 * 1024) ++s.zero_shift;
  }
  {
    Prof prof("embed_bwd_sort", st);
    static bool ready[kMaxDevices] = {false};
    const int dev = current_device();
    if (!ready[dev]) {
      TSP_CUDA_TRY(cudaFuncSetAttribute(embed_sort_kernel,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem));
      ready[dev] = true;
    }
    int nc = 1;   // CTAs of the cluster: 4096 positions each before another joins
    while (nc < kMaxCluster && (int64_t)nc * 4096 < S) nc *= 2;
    cudaLaunchConfig_t cfg = {};
    const int zero = s.zero_shift < 0 ? 0 : 1 << s.zero_shift;
    cfg.gridDim = dim3(nc + (zero + nc - 1) / nc * nc);
    cfg.blockDim = dim3(kSortWarps * 32);
    cfg.dynamicSmemBytes = kSortSmem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = nc;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    TSP_CUDA_TRY(cudaLaunchKernelEx(&cfg, embed_sort_kernel, s));
  }
  SumArgs a;
  a.key = L.key[s.passes & 1];
  a.row = L.row[s.passes & 1];
  a.add = accumulate;
  a.table = dtable;
  a.part = L.part;
  a.S = (int)S;
  a.vocab = (int)vocab;
  a.d = d;
  a.chunk = chunk_of(S, d);
  a.nchunks = (int)((S + a.chunk - 1) / a.chunk);
  a.nslabs = (d + kSlab - 1) / kSlab;
  a.scale = scale;
  a.status = s.status;
  const bool vec = d % 4 == 0;
  if (dx_dtype == TSP_BF16)
    return vec ? embed_sum_t<__nv_bfloat16, true>(dx, a, st)
               : embed_sum_t<__nv_bfloat16, false>(dx, a, st);
  return vec ? embed_sum_t<float, true>(dx, a, st) : embed_sum_t<float, false>(dx, a, st);
}

}  // namespace tsp
