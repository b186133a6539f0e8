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
#include "common.cuh"
#include "kernels.h"

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
template <typename T, typename V>
__device__ __forceinline__ V scale_unit(V u, float s) {
  if constexpr (sizeof(T) == 2 && sizeof(V) > 2) {
    uint32_t w[sizeof(V) / 4];
    memcpy(w, &u, sizeof(V));
#pragma unroll
    for (int i = 0; i < (int)(sizeof(V) / 4); ++i) w[i] = pack2<T>(lo2<T>(w[i]) * s, hi2<T>(w[i]) * s);
    memcpy(&u, w, sizeof(V));
  } else {
    T e[sizeof(V) / sizeof(T)];
    memcpy(e, &u, sizeof(V));
#pragma unroll
    for (int i = 0; i < (int)(sizeof(V) / sizeof(T)); ++i) e[i] = from_f<T>(to_f<T>(e[i]) * s);
    memcpy(&u, e, sizeof(V));
  }
  return u;
}

// A warp a position, a segment of 32 * LOADS units of sizeof(V) bytes at a time
// (stride gridDim.y), LOADS loads in flight a lane.  Not a persistent grid: CTAs
// started in order keep the rows written at a time next to each other (131072 x
// 4096 bf16 out of 32000 rows: 207 us, 1.32 GB of DRAM traffic at 6.4 TB/s; 232 us
// with 4 resident CTAs a multiprocessor walking the positions).
template <typename T, typename V, int LOADS>
__global__ void __launch_bounds__(256) embed_fwd_kernel(const void* __restrict__ ids, int id_bytes,
                                                        const V* __restrict__ table,
                                                        V* __restrict__ x, int S, int c, int D,
                                                        int64_t vocab, int upr, float scale,
                                                        int* __restrict__ status) {
  const int lane = threadIdx.x & 31, p = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (p >= S) return;
  const int64_t id = load_id(ids, id_bytes, p);
  const int row = row_of(p, c, D);
  if (!TSP_INB(row >= 0 && row < S, status)) return;
  if (id >= vocab && lane == 0) report_status(status, (int)TSP_ERR_RANGE);
  const bool there = id >= 0 && id < vocab;
  const V* src = table + (there ? id : 0) * upr;
  V* dst = x + (int64_t)row * upr;
  for (int u0 = blockIdx.y * 32 * LOADS + lane; u0 < upr; u0 += gridDim.y * 32 * LOADS) {
    V v[LOADS];
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
      v[k] = V{};
      if (there && u0 + k * 32 < upr) v[k] = src[u0 + k * 32];
    }
#pragma unroll
    for (int k = 0; k < LOADS; ++k)
      if (u0 + k * 32 < upr)   // the rows are not read here again: table rows stay in L2
        __stcs(dst + u0 + k * 32, scale == 1.f ? v[k] : scale_unit<T, V>(v[k], scale));
  }
}

// Rows of at most 16 units: 2^lanes lanes a row, and four positions a thread, whose
// ids and then rows are loaded together.
template <typename T, typename V>
__global__ void __launch_bounds__(256) embed_fwd_short_kernel(const void* __restrict__ ids, int id_bytes,
                                                              const V* __restrict__ table,
                                                              V* __restrict__ x, int S, int c, int D,
                                                              int64_t vocab, int upr, int lanes,
                                                              float scale, int* __restrict__ status) {
  constexpr int K = 4;
  const int unit = threadIdx.x & ((1 << lanes) - 1), rows = 256 >> lanes;
  const int64_t p0 = (int64_t)blockIdx.x * K * rows + (threadIdx.x >> lanes);
  int64_t id[K];
  V v[K];
#pragma unroll
  for (int k = 0; k < K; ++k) id[k] = p0 + k * rows < S ? load_id(ids, id_bytes, p0 + k * rows) : -1;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    v[k] = V{};
    if (id[k] >= vocab) report_status(status, (int)TSP_ERR_RANGE);
    else if (id[k] >= 0 && unit < upr) v[k] = table[id[k] * upr + unit];
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (p0 + k * rows >= S || unit >= upr) continue;
    const int row = row_of((int)(p0 + k * rows), c, D);
    if (TSP_INB(row >= 0 && row < S, status))
      x[(int64_t)row * upr + unit] = scale == 1.f ? v[k] : scale_unit<T, V>(v[k], scale);
  }
}

template <typename T, typename V>
tsp_status embed_fwd_t(const void* ids, int id_bytes, const void* table, void* x, int64_t S, int D,
                       int64_t vocab, int d, float scale, cudaStream_t st) {
  const int upr = (int)((int64_t)d * sizeof(T) / sizeof(V));
  const unsigned gx = (unsigned)((S + 7) / 8);
  const int64_t full = (int64_t)num_sms() * 4;   // CTAs the GPU holds at 64 registers a thread
  Prof prof("embed_fwd", st);
  if (upr <= 16) {   // (131072 x 64 bf16: 5.3 us, 27 with a warp a row)
    int lanes = 0;
    while (1 << lanes < upr) ++lanes;
    const int64_t rows = 4 * (256 >> lanes);
    embed_fwd_short_kernel<T, V><<<(unsigned)((S + rows - 1) / rows), 256, 0, st>>>(
        ids, id_bytes, (const V*)table, (V*)x, (int)S, (int)(S / (2 * D)), D, vocab, upr, lanes, scale,
        status_word());
  } else if (gx < full) {   // few positions: short segments, on CTAs of their own
    const int gy = (int)std::min<int64_t>((upr + 63) / 64, full / gx);
    embed_fwd_kernel<T, V, 2><<<dim3(gx, gy), 256, 0, st>>>(
        ids, id_bytes, (const V*)table, (V*)x, (int)S, (int)(S / (2 * D)), D, vocab, upr, scale,
        status_word());
  } else {
    embed_fwd_kernel<T, V, 8><<<gx, 256, 0, st>>>(
        ids, id_bytes, (const V*)table, (V*)x, (int)S, (int)(S / (2 * D)), D, vocab, upr, scale,
        status_word());
  }
  TSP_CUDA_TRY(cudaGetLastError());
  return TSP_OK;
}

// ---------------------------------------------------------------------------
// Backward, step 1: the positions sorted by token
// ---------------------------------------------------------------------------
// (token, zigzag row) pairs in the order of (token, position), so that the sums
// of step 2 have one fixed order.  Ids outside the table sort to the end as token
// `vocab`.  The data are small (8 bytes a position, in L2 throughout): what counts
// is the number of dependent steps.
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;

struct SortArgs {
  const void* ids;
  int id_bytes;
  int S, c, D, vocab;
  int2* pair[2];          // (token, row): a pass reads one and writes the other
  int* count;             // [runs][bins] of the pass
  int run, runs;          // positions of a run, runs
  int shift, bits;
  int pass;               // 0: from the ids
  int* starts;            // [2], set to zero for step 2
  int* status;
};

__device__ __forceinline__ int token_of(const SortArgs& a, int p, bool* past) {
  const int64_t id = load_id(a.ids, a.id_bytes, p);
  *past |= id >= a.vocab;
  return id < 0 ? a.vocab : (int)min(id, (int64_t)a.vocab);
}

// Up to kRankMax positions: the place of each is the number of positions with a
// smaller (token, position), both in one 32-bit word.  A CTA takes 32 positions, a
// warp of it a sixteenth of the comparisons.  As long as there is a multiprocessor for
// every CTA this is quicker than two passes of the sort below (64 columns added up,
// 32000 tokens: 14.5 us at 4800 positions, 17.7 sorted; 17.9 and 17.5 at 5200).
constexpr int kRankMax = 152 * 32;

__global__ void __launch_bounds__(kSortThreads) embed_rank_kernel(const __grid_constant__ SortArgs a,
                                                                  int pos_bits) {
  __shared__ __align__(16) unsigned word[kRankMax];
  __shared__ int place[32];
  constexpr int kBatch = 8;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int padded = (a.S + 63) / 64 * 64;   // each warp's part is whole 4's
  bool past = false;
  for (int p = t; p < padded; p += kBatch * kSortThreads) {
    int key[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int q = p + k * kSortThreads;
      key[k] = q < a.S ? token_of(a, q, &past) : 0;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int q = p + k * kSortThreads;
      if (q < padded) word[q] = q < a.S ? (unsigned)key[k] << pos_bits | q : 0xffffffffu;
    }
  }
  if (past) report_status(a.status, (int)TSP_ERR_RANGE);
  if (t < 32) place[t] = 0;
  if (blockIdx.x == 0 && t < 2) a.starts[t] = 0;
  __syncthreads();
  const int i = blockIdx.x * 32 + lane;
  const unsigned me = i < a.S ? word[i] : 0u;
  const int part = padded / kSortWarps;
  const uint4* w4 = reinterpret_cast<const uint4*>(word + warp * part);
  int below = 0;
#pragma unroll 4
  for (int j = 0; j < part / 4; ++j) {
    const uint4 w = w4[j];
    below += (w.x < me) + (w.y < me) + (w.z < me) + (w.w < me);
  }
  atomicAdd(place + lane, below);   // (integers: the order does not matter)
  __syncthreads();
  if (warp == 0 && i < a.S && TSP_INB(place[lane] < a.S, a.status))
    a.pair[0][place[lane]] = make_int2((int)(me >> pos_bits), row_of(i, a.c, a.D));
}

// More positions: a stable least-significant-digit radix sort, two launches a
// pass.  A CTA a run of kTile positions (of several, beyond kMaxRuns of them)
// counts its digits; then every CTA sums the runs' counts to the places of its
// own digits and scatters, the positions of a warp in order by votes on the
// digit's bits.  (One cluster with its counts in distributed shared memory needs
// one launch but has eight multiprocessors' throughput: 28 us at 16384 positions,
// 88 at 131072.)
constexpr int kTile = 1024, kGroups = kTile / kSortThreads;   // groups of 32 a warp
constexpr int kBits = 9, kBins = 1 << kBits, kMaxRuns = 512;

__global__ void __launch_bounds__(kSortThreads) embed_count_kernel(const __grid_constant__ SortArgs a) {
  __shared__ int hist[kBins];
  const int t = threadIdx.x, bins = 1 << a.bits;
  after_previous_kernel();   // (pass 0: launched in the ordinary way)
  if (t < bins) hist[t] = 0;
  if (blockIdx.x == 0 && t < 2) a.starts[t] = 0;
  __syncthreads();
  bool past = false;
  const int end = min(a.S, (int)(blockIdx.x + 1) * a.run);
#pragma unroll 2
  for (int p = blockIdx.x * a.run + t; p < end; p += kSortThreads) {
    const int key = a.pass == 0 ? token_of(a, p, &past) : a.pair[a.pass & 1][p].x;
    atomicAdd(hist + ((key >> a.shift) & (bins - 1)), 1);
  }
  if (past) report_status(a.status, (int)TSP_ERR_RANGE);
  __syncthreads();
  if (t < bins) a.count[((int64_t)blockIdx.x << a.bits) + t] = hist[t];
}

__global__ void __launch_bounds__(kSortThreads) embed_scatter_kernel(const __grid_constant__ SortArgs a) {
  __shared__ int hist[kSortWarps][kBins];
  __shared__ int sum_all[kSortThreads], sum_before[kSortThreads], wsum[kSortWarps];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, bins = 1 << a.bits;
  after_previous_kernel();
  // the digits' counts over all runs and over those before this one: thread
  // (part, digit) sums every parts-th run
  const int parts = kSortThreads >> a.bits, part = t >> a.bits;
  int all = 0, before = 0;
#pragma unroll 8
  for (int i = part; i < a.runs; i += parts) {
    const int n = a.count[((int64_t)i << a.bits) + (t & (bins - 1))];
    all += n;
    before += i < (int)blockIdx.x ? n : 0;
  }
  sum_all[t] = all;
  sum_before[t] = before;
  __syncthreads();
  all = before = 0;
  if (t < bins) {
    for (int q = 0; q < parts; ++q) {
      all += sum_all[q * bins + t];
      before += sum_before[q * bins + t];
    }
  }
  int inc = all;   // over the digits
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += n;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int pre = lane < warp ? wsum[lane < kSortWarps ? lane : 0] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) pre += __shfl_xor_sync(0xffffffffu, pre, o);
  int at_digit = inc - all + before + pre;   // where this CTA's next position of digit t goes

  bool past = false;
  const int end = min(a.S, (int)(blockIdx.x + 1) * a.run);
  for (int p0 = blockIdx.x * a.run; p0 < end; p0 += kTile) {
    // this lane's positions: group k of the warp, in position order
    int2 pair[kGroups];
    unsigned same[kGroups];
    int digit[kGroups], was[kGroups];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const int p = p0 + (warp * kGroups + k) * 32 + lane;
      pair[k] = make_int2(0, 0);
      if (p < end)
        pair[k] = a.pass == 0 ? make_int2(token_of(a, p, &past), row_of(p, a.c, a.D)) : a.pair[a.pass & 1][p];
      digit[k] = p < end ? (pair[k].x >> a.shift) & (bins - 1) : bins;
    }
    for (int i = lane; i < bins; i += 32) hist[warp][i] = 0;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      same[k] = 0xffffffffu;   // the lanes with this lane's digit
#pragma unroll
      for (int b = 0; b <= kBits; ++b) {
        const bool one = digit[k] >> b & 1;
        const unsigned votes = __ballot_sync(0xffffffffu, one);
        same[k] &= one ? votes : ~votes;
      }
    }
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {   // was: of the digit in the warp's groups before
      was[k] = digit[k] < bins ? hist[warp][digit[k]] : 0;
      __syncwarp();
      if (digit[k] < bins && lane == __ffs(same[k]) - 1) hist[warp][digit[k]] = was[k] + __popc(same[k]);
      __syncwarp();
    }
    __syncthreads();
    if (t < bins) {   // places of the warps' digits
      int n[kSortWarps];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) n[w] = hist[w][t];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        hist[w][t] = at_digit;
        at_digit += n[w];
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      if (digit[k] == bins) continue;
      const int at = hist[warp][digit[k]] + was[k] + __popc(same[k] & ((1u << lane) - 1));
      if (TSP_INB(at >= 0 && at < a.S, a.status)) a.pair[(a.pass & 1) ^ 1][at] = pair[k];
    }
    __syncwarp();
  }
}

// Positions of a run.
int run_of(int64_t S) {
  const int64_t tiles = (S + kTile - 1) / kTile;
  return (int)((tiles + kMaxRuns - 1) / kMaxRuns * kTile);
}

// ---------------------------------------------------------------------------
// Backward, step 2: rows summed along the sorted order
// ---------------------------------------------------------------------------
// A warp takes a chunk of the sorted positions and a slab of 256 columns (8 a
// lane) and walks the chunk's rows, four or (16-bit) eight of them on their way;
// places and tokens come 32 at a time.  A token whose positions lie inside
// the chunk is written (or added) to its table row at once; one that came in from
// the chunk before leaves its part in slot 2*chunk, one that starts here and goes on
// in slot 2*chunk + 1.  Step 3 adds those up.  So a frequent token is split over as
// many warps as it has chunks, and every sum has one order.  The first warps of the
// grid write the zero rows of absent tokens, eight rows each, which they look up in
// the sorted tokens: plain stores next to the other warps' loads.  HBM-bound where
// rows are long (32768 x 4096 fp32 into 32000 rows: 1.01 GB in 162 us of the call's
// 181), by the latency of a warp's few loads where they are short.
constexpr int kSlab = 256, kZeroRows = 8, kLong = 12;

// A lane's eight columns of a row: two groups of four next to each other (VEC), or
// eight single ones 32 apart; as they are stored, until they are added up.
template <typename T, bool VEC>
struct Cols {
  T e[8];
  __device__ __forceinline__ void load(const T* row, int c0, int lane, int d) {
    if constexpr (VEC) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = c0 + h * 128 + lane * 4;
        if constexpr (sizeof(T) == 4)
          reinterpret_cast<float4*>(e)[h] = c < d ? __ldcs(reinterpret_cast<const float4*>(row + c)) : float4{};
        else
          reinterpret_cast<uint2*>(e)[h] = c < d ? __ldcs(reinterpret_cast<const uint2*>(row + c)) : uint2{};
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + i * 32 + lane;
        e[i] = c < d ? row[c] : from_f<T>(0.f);
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f<T>(0.f);
  }
  __device__ __forceinline__ void add_to(float (&acc)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += to_f<T>(e[i]);
  }
} __attribute__((aligned(16)));

// row = v * s, or row += v * s.  The addition is the memory's (nothing waits for the
// old value); it is the only one the element gets in a call, so no order matters.
template <bool VEC>
__device__ __forceinline__ void store_cols(float* row, int c0, int lane, int d, const float (&v)[8],
                                           float s, bool add) {
  if constexpr (VEC) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 + h * 128 + lane * 4;
      if (c >= d) continue;
      float4* p = reinterpret_cast<float4*>(row + c);
      const float4 o = make_float4(v[4 * h] * s, v[4 * h + 1] * s, v[4 * h + 2] * s, v[4 * h + 3] * s);
      if (add) atomicAdd(p, o);
      else *p = o;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = c0 + e * 32 + lane;
      if (c >= d) continue;
      if (add) atomicAdd(row + c, v[e] * s);
      else row[c] = v[e] * s;
    }
  }
}

struct SumArgs {
  const int2* pair;   // sorted (token, row)
  float *table, *part;
  // chunks where a token starts that goes on, for at most kLong chunks and for
  // more: how many [2], which [2][nchunks]
  int *starts, *start;
  int S, vocab, d, chunk, nchunks, nslabs;
  int zero_tasks;   // 0: add to the table rows instead of overwriting them
  float scale;
  int* status;
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) embed_sum_kernel(const T* __restrict__ dx,
                                                        const __grid_constant__ SumArgs a) {
  constexpr int kAhead = VEC && sizeof(T) == 2 ? 8 : 4;
  const int lane = threadIdx.x & 31;
  int64_t task = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const bool adds = a.zero_tasks == 0;
  after_previous_kernel();
  if (task < a.zero_tasks) {
    const int v0 = (int)task * kZeroRows, v = v0 + lane % kZeroRows;
    int lo = 0, hi = a.S;   // the first place with a token >= v
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.pair[mid].x < v) lo = mid + 1; else hi = mid;
    }
    const bool absent = v < a.vocab && (lo == a.S || a.pair[lo].x != v);
    const unsigned rows = __ballot_sync(0xffffffffu, absent);
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int r = 0; r < kZeroRows; ++r) {
      if (!(rows >> r & 1)) continue;
      for (int s = 0; s < a.nslabs; ++s)
        store_cols<VEC>(a.table + (int64_t)(v0 + r) * a.d, s * kSlab, lane, a.d, zero, 1.f, false);
    }
    return;
  }
  task -= a.zero_tasks;
  if (task >= (int64_t)a.nchunks * a.nslabs) return;
  const int ch = (int)(task / a.nslabs), c0 = (int)(task - (int64_t)ch * a.nslabs) * kSlab;
  const int j0 = ch * a.chunk, j1 = (int)min((int64_t)a.S, (int64_t)j0 + a.chunk);
  int cur = a.pair[j0].x;
  if (cur >= a.vocab) return;
  bool opened = j0 == 0 || a.pair[j0 - 1].x != cur;   // the current token's positions start here
  const bool goes_on = j1 < a.S && a.pair[j1].x == a.pair[j1 - 1].x;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto leave = [&](bool on) {
    if (opened && !on)
      store_cols<VEC>(a.table + (int64_t)cur * a.d, c0, lane, a.d, acc, a.scale, adds);
    else
      store_cols<VEC>(a.part + ((int64_t)2 * ch + (opened ? 1 : 0)) * a.d, c0, lane, a.d, acc, 1.f,
                      false);
  };
  auto pairs = [&](int j) { return j + lane < j1 ? a.pair[j + lane] : make_int2(a.vocab, 0); };
  auto load = [&](Cols<T, VEC>& to, int key, int r) {
    if (key < a.vocab && TSP_INB(r >= 0 && r < a.S, a.status)) to.load(dx + (int64_t)r * a.d, c0, lane, a.d);
    else to.clear();
  };
  // true if the row of this token was added, false at the padding behind the last one
  auto add = [&](const Cols<T, VEC>& row, int key) {
    if (key != cur) {
      leave(false);
      cur = key;
      opened = true;
      if (cur >= a.vocab) return false;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    }
    row.add_to(acc);
    return true;
  };
  Cols<T, VEC> v[kAhead];
  if constexpr (sizeof(T) == 2) {
    // the place of the row just added takes the one kAhead further on (131072 x 1024
    // into 32000 rows: 104 us; 122 with eight loaded, then eight added)
    int2 mine = pairs(j0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      load(v[u], __shfl_sync(0xffffffffu, mine.x, u), __shfl_sync(0xffffffffu, mine.y, u));
    for (int j = j0; j < j1; j += 32) {
      const int2 next = pairs(j + 32);
      for (int k = 0; k < 32 && j + k < j1; k += kAhead) {
        const int2 from = k + kAhead < 32 ? mine : next;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int at = (k + u + kAhead) & 31;
          if (j + k + u < j1 && !add(v[u], __shfl_sync(0xffffffffu, mine.x, k + u))) return;
          load(v[u], __shfl_sync(0xffffffffu, from.x, at), __shfl_sync(0xffffffffu, from.y, at));
        }
      }
      mine = next;
    }
  } else {
    // four loaded, then four added: the warps of a row stay together (131072 x 1024:
    // 131 us, 141 in the other way)
    for (int j = j0; j < j1; j += 32) {
      const int2 mine = pairs(j);
      for (int k = 0; k < 32 && j + k < j1; k += kAhead) {
        int key[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          key[u] = __shfl_sync(0xffffffffu, mine.x, k + u);
          load(v[u], key[u], __shfl_sync(0xffffffffu, mine.y, k + u));
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (j + k + u >= j1) break;
          if (!add(v[u], key[u])) return;
        }
      }
    }
  }
  leave(goes_on);
  // (the list's order is that of arrival; its entries are joined each by itself)
  if (opened && goes_on && c0 == 0 && lane == 0) {
    const int64_t far = (int64_t)j0 + (int64_t)kLong * a.chunk;
    const int is_long = far < a.S && a.pair[far].x == cur;
    a.start[is_long * a.nchunks + atomicAdd(a.starts + is_long, 1)] = ch;
  }
}

// acc += the part of the token that starts in chunk ch and goes on
template <bool VEC>
__device__ __forceinline__ void first_part(const SumArgs& a, int ch, int c0, int lane, float (&acc)[8]) {
  Cols<float, VEC> v;
  v.load(a.part + ((int64_t)2 * ch + 1) * a.d, c0, lane, a.d);
  v.add_to(acc);
}
// The first token of chunk k + lane * step (-1 past the last chunk).
__device__ __forceinline__ int head_of(const SumArgs& a, int k, int step, int lane) {
  const int64_t q = k + (int64_t)lane * step;
  return q < a.nchunks ? a.pair[q * a.chunk].x : -1;
}
// acc += the parts of token `tok` in chunks k, k + step, ...; head: head_of these.  The
// chunks that go on with the token are the first ones, so one vote says how many.
template <bool VEC>
__device__ __forceinline__ void add_parts(const SumArgs& a, int head, int tok, int k, int step, int c0,
                                          int lane, float (&acc)[8]) {
  constexpr int kBatch = 8;
  for (;;) {
    const int n = __popc(__ballot_sync(0xffffffffu, head == tok));
    for (int u0 = 0; u0 < n; u0 += kBatch) {
      Cols<float, VEC> v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (u0 + u < n) v[u].load(a.part + (2 * k + 2 * (int64_t)(u0 + u) * step) * a.d, c0, lane, a.d);
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (u0 + u < n) v[u].add_to(acc);
    }
    if (n < 32) return;
    k += 32 * step;
    head = head_of(a, k, step, lane);
  }
}

// Step 3: a token that starts in one chunk and ends in a later one (step 2 has
// listed the chunks where one starts): its parts added in chunk order, a warp a
// token and slab.  The few tokens of more than kLong chunks get a CTA a slab, whose
// warps add up every eighth part each, then the eight sums in order.  Bound by the
// latency of its four dependent loads: the heads of up to 32 chunks are one of them
// (47028 x 768 bf16 into 1086 rows: 39 us, 42 with heads and parts by turns in fours).
template <bool VEC>
__global__ void __launch_bounds__(256) embed_join_kernel(const __grid_constant__ SumArgs a) {
  __shared__ float sums[8][kSlab];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  after_previous_kernel();
  const int64_t n_short = (int64_t)a.starts[0] * a.nslabs, n_long = (int64_t)a.starts[1] * a.nslabs;
  for (int64_t task = blockIdx.x; task < n_long; task += gridDim.x) {
    const int ch = a.start[a.nchunks + task / a.nslabs], c0 = (int)(task % a.nslabs) * kSlab;
    const int tok = a.pair[(ch + 1) * a.chunk].x, head = head_of(a, ch + 1 + warp, 8, lane);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (warp == 0) first_part<VEC>(a, ch, c0, lane, acc);
    add_parts<VEC>(a, head, tok, ch + 1 + warp, 8, c0, lane, acc);
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[warp][e * 32 + lane] = acc[e];
    __syncthreads();
    if (warp == 0) {
      for (int w = 1; w < 8; ++w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += sums[w][e * 32 + lane];
      }
      store_cols<VEC>(a.table + (int64_t)tok * a.d, c0, lane, a.d, acc, a.scale, a.zero_tasks == 0);
    }
    __syncthreads();
  }
  for (int64_t task = (int64_t)blockIdx.x * 8 + warp; task < n_short; task += (int64_t)gridDim.x * 8) {
    const int ch = a.start[task / a.nslabs], c0 = (int)(task % a.nslabs) * kSlab;
    const int head = head_of(a, ch + 1, 1, lane), tok = __shfl_sync(0xffffffffu, head, 0);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    first_part<VEC>(a, ch, c0, lane, acc);
    add_parts<VEC>(a, head, tok, ch + 1, 1, c0, lane, acc);
    store_cols<VEC>(a.table + (int64_t)tok * a.d, c0, lane, a.d, acc, a.scale, a.zero_tasks == 0);
  }
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
  int2* pair[2];
  int *count, *start;
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
  for (int k = 0; k < 2; ++k) L.pair[k] = (int2*)take((size_t)S * 8);
  L.count = (int*)take((size_t)((S + run_of(S) - 1) / run_of(S)) * kBins * 4);
  const int64_t chunks = (S + chunk_of(S, d) - 1) / chunk_of(S, d);
  L.start = (int*)take((size_t)(2 + 2 * chunks) * 4);
  L.part = (float*)take((size_t)chunks * 2 * d * 4);
  L.bytes = off;
  return L;
}

template <typename T, bool VEC>
tsp_status embed_sum_t(const void* dx, const SumArgs& a, cudaStream_t st) {
  const int64_t tasks = (int64_t)a.nchunks * a.nslabs + a.zero_tasks;
  Prof prof("embed_bwd_sum", st, a.nchunks > 1 ? 2 : 1);
  const tsp_status r =
      launch_after(embed_sum_kernel<T, VEC>, dim3((unsigned)((tasks + 7) / 8)), 256, 0, st, (const T*)dx, a);
  if (r != TSP_OK) return r;
  if (a.nchunks > 1) {
    const int64_t most = (int64_t)(a.nchunks - 1) * a.nslabs;   // (a CTA each if all were long)
    return launch_after(embed_join_kernel<VEC>, dim3((unsigned)std::min<int64_t>(most, num_sms() * 4)),
                        256, 0, st, a);
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
  for (int k = 0; k < 2; ++k) s.pair[k] = L.pair[k];
  s.count = L.count;
  s.starts = L.start;
  s.status = status_word();
  s.pass = s.shift = 0;
  int nb = 1;   // bits of the largest token, `vocab` itself
  while ((vocab >> nb) != 0) ++nb;
  int pos_bits = 1;
  while ((S - 1) >> pos_bits != 0) ++pos_bits;
  if (S <= kRankMax && nb + pos_bits <= 32) {
    Prof prof("embed_bwd_sort", st);
    embed_rank_kernel<<<(unsigned)((S + 31) / 32), kSortThreads, 0, st>>>(s, pos_bits);
    TSP_CUDA_TRY(cudaGetLastError());
  } else {
    const int passes = (nb + kBits - 1) / kBits;
    s.bits = std::max(5, (nb + passes - 1) / passes);   // whole warps of digits
    s.run = run_of(S);
    s.runs = (int)((S + s.run - 1) / s.run);
    Prof prof("embed_bwd_sort", st, 2 * passes);
    for (; s.pass < passes; ++s.pass, s.shift += s.bits) {
      tsp_status r = TSP_OK;
      if (s.pass == 0) {
        embed_count_kernel<<<s.runs, kSortThreads, 0, st>>>(s);
        TSP_CUDA_TRY(cudaGetLastError());
      } else {
        r = launch_after(embed_count_kernel, dim3(s.runs), kSortThreads, 0, st, s);
      }
      if (r == TSP_OK) r = launch_after(embed_scatter_kernel, dim3(s.runs), kSortThreads, 0, st, s);
      if (r != TSP_OK) return r;
    }
  }
  SumArgs a;
  a.pair = L.pair[s.pass & 1];
  a.zero_tasks = accumulate ? 0 : (int)((vocab + kZeroRows - 1) / kZeroRows);
  a.table = dtable;
  a.part = L.part;
  a.starts = L.start;
  a.start = L.start + 2;
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
