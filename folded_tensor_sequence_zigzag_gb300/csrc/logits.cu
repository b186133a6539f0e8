// logits.cu -- behind the stack: log probabilities, entropy and top alternatives
// of rows of logits, the token losses, and the gradients of both.
//
// With x the row of a position, m its largest logit, c the scale:
//   l = log sum_j exp(c (x_j - m)),   log p_j = c (x_j - m) - l,
//   H = -sum_j p_j log p_j = l - sum_j p_j c (x_j - m)
//   loss = w_ce (-log p_t) + w_kd sum_k q_k (log q_k - log p_{id_k}),  q = softmax_k(t_scale * teacher)
//   dx_j = p_j (A + B log p_j) + what the listed tokens add at j
// (A, B and the additions in grad_kernel).  Everything is bound by HBM: the
// forward reads the rows once, the gradient reads and writes them once.
//
// A row starts at any element: it is taken as 16-byte units, the few elements in
// front of the first and behind the last one are read by themselves.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "common.cuh"
#include "kernels.h"

namespace tsp {

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Exponents (of 2) below this are 0 in fp32 by far; a clamp to it keeps 0 * -inf away.
constexpr float kLeast = -1024.f;
// A running reference is renewed once a logit is this far (in powers of 2) above it:
// sums then stay below V * 2^8, and renewals are rare.
constexpr float kSlack = 8.f;

__device__ __forceinline__ int64_t load_id(const void* ids, int id_bytes, int64_t p) {
  return id_bytes == 8 ? (int64_t)reinterpret_cast<const long long*>(ids)[p]
                       : (int64_t)reinterpret_cast<const int*>(ids)[p];
}

__device__ __forceinline__ int pos_of(int row, int c, int D) {
  return D == 1 ? row : (int)zz_pos_of_row(row, c, D);
}

template <typename T> __device__ __forceinline__ float lowest();
template <> __device__ __forceinline__ float lowest<float>() { return -3.4028234663852886e38f; }
template <> __device__ __forceinline__ float lowest<__nv_bfloat16>() { return -3.3895313892515355e38f; }

// A row as 16-byte units: `head` elements in front of the first, `units` of them,
// and the elements from `tail` on behind the last.
template <typename T>
struct RowUnits {
  static constexpr int E = 16 / sizeof(T);
  const T* row;
  int head, units, tail, V;
  __device__ RowUnits(const void* base, int64_t ld, int64_t r, int v) {
    row = reinterpret_cast<const T*>(base) + r * ld;
    V = v;
    head = min(v, (int)((16 - ((uintptr_t)row & 15)) & 15) / (int)sizeof(T));
    units = (v - head) / E;
    tail = head + units * E;
  }
  __device__ const uint4* first() const { return reinterpret_cast<const uint4*>(row + head); }
  // the n-th element outside the units, -1 behind the last of them
  __device__ int loose(int n) const { return n < head ? n : (tail + n - head < V ? tail + n - head : -1); }
};

template <typename T> __device__ __forceinline__ float2 pair(uint4 u, int i);
template <> __device__ __forceinline__ float2 pair<__nv_bfloat16>(uint4 u, int i) {
  const uint32_t w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
  return make_float2(bf16_lo(w), bf16_hi(w));
}
template <> __device__ __forceinline__ float2 pair<float>(uint4 u, int i) {
  return i == 0 ? make_float2(__uint_as_float(u.x), __uint_as_float(u.y))
                : make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
}
template <typename T> __device__ __forceinline__ uint4 no_unit();   // -inf throughout
template <> __device__ __forceinline__ uint4 no_unit<__nv_bfloat16>() {
  return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
}
template <> __device__ __forceinline__ uint4 no_unit<float>() {
  return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The largest of N units; NaN does not count.
template <typename T, int N> __device__ __forceinline__ float largest(const uint4 (&u)[N]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t m = 0xff80ff80u;
#pragma unroll
    for (int k = 0; k < N; ++k)
      m = max_bf16x2(m, max_bf16x2(max_bf16x2(u[k].x, u[k].y), max_bf16x2(u[k].z, u[k].w)));
    return fmaxf(bf16_lo(m), bf16_hi(m));
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < N; ++k)
      m = fmax3f(fmax3f(m, __uint_as_float(u[k].x), __uint_as_float(u[k].y)), __uint_as_float(u[k].z),
                 __uint_as_float(u[k].w));
    return m;
  }
}
__device__ __forceinline__ uint4 load_unit(const uint4* p) {
  uint4 u;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p)
               : "memory");
  return u;
}

// A thread's sums over its logits, relative to a reference m that is a logit it has
// seen (the type's lowest value at first): s = sum 2^u and a = sum 2^u u with
// u = c2 (x - m), c2 = c log2(e).  The difference is exact or rounded once, so that
// large logits cost no accuracy.
template <bool ENT>
struct Sums {
  float m, top;      // reference, largest logit so far
  float2 s, a;
  __device__ explicit Sums(float low)
      : m(low), top(-INFINITY), s(make_float2(0.f, 0.f)), a(make_float2(0.f, 0.f)) {}

  __device__ __forceinline__ void see(float largest, float c2, float slack) {
    top = fmaxf(top, largest);
    if (largest > m + slack) {
      const float d = fmaxf((m - largest) * c2, kLeast), f = ex2_approx(d);
      if (ENT) a = make_float2((a.x + d * s.x) * f, (a.y + d * s.y) * f);
      s = make_float2(s.x * f, s.y * f);
      m = largest;
    }
  }
  __device__ __forceinline__ void add(float2 x, float c2) {
    const float2 u = fmul2(fadd2(x, make_float2(-m, -m)), make_float2(c2, c2));
    const float2 e = make_float2(ex2_approx(u.x), ex2_approx(u.y));
    s = fadd2(s, e);
    if (ENT) a = ffma2(e, make_float2(fmaxf(u.x, kLeast), fmaxf(u.y, kLeast)), a);
  }
};

// What the threads of a CTA have together.
struct Row {
  float m, l;        // largest logit, log of the sum: -inf where no logit is above -inf
  float entropy;
};

constexpr int kThreads = 512, kWarps = kThreads / 32;

// The CTA's largest logit and its sums relative to that, in every thread; a fixed order.
template <bool ENT>
__device__ __forceinline__ void join_sums(const Sums<ENT>& t, float low, float c2, float (*part)[4],
                                          float* m_out, float* s_out, float* a_out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  auto onto = [&](float m, float from, float& s, float& a) {   // sums relative to `from`, now to m
    const float d = fmaxf((from - m) * c2, kLeast), f = ex2_approx(d);
    if (ENT) a = (a + d * s) * f;
    s *= f;
  };
  float s = t.s.x + t.s.y, a = ENT ? t.a.x + t.a.y : 0.f;
  const float mw = fmaxf(warp_max(t.top), low);
  onto(mw, t.m, s, a);
  s = warp_sum(s);
  if (ENT) a = warp_sum(a);
  if (lane == 0) {
    part[warp][0] = mw;
    part[warp][1] = s;
    part[warp][2] = a;
  }
  __syncthreads();
  const bool one = lane < warps;   // a lane a warp
  const float from = one ? part[lane][0] : low;
  const float m = warp_max(from);
  s = one ? part[lane][1] : 0.f;
  a = ENT && one ? part[lane][2] : 0.f;
  onto(m, from, s, a);
  *m_out = m;
  *s_out = warp_sum(s);
  if (ENT) *a_out = warp_sum(a);
}
template <bool ENT>
__device__ __forceinline__ Row join(const Sums<ENT>& t, float low, float c2, float (*part)[4]) {
  float m, s, a = 0.f;
  join_sums<ENT>(t, low, c2, part, &m, &s, &a);
  Row r;
  const bool none = s == 0.f;
  r.m = none ? 0.f : m;
  r.l = none ? -INFINITY : logf(s);
  r.entropy = none ? 0.f : r.l - a / s * kLn2;
  if (r.entropy < 0.f) r.entropy = 0.f;
  return r;
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
struct Rows {
  const void* logits;
  int64_t ld;
  const void* ids;     // may be NULL
  int id_bytes, S, c, D, V;
  float scale;
  int* status;
};
struct Teacher {
  const int* ids;      // [S, K]
  const void* logits;  // [S, K]
  int f32, K;
  float scale, w_ce, w_kd;
};
struct FwdArgs {
  Rows r;
  float *logp, *entropy, *stats, *top_logp;
  int* top_ids;
  int top;
  Teacher t;
  float* loss;
};

// A logit and its token as one key: the larger logit first, the lower token of equal
// ones (-0 and 0 are equal).
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, int j) {
  return (uint64_t)order_of(x) << 32 | (uint32_t)~j;
}
constexpr uint32_t kOrderNone = 0x007fffffu;   // order_of(-inf)

constexpr int kCandidates = 1024;
struct TopSmem {
  float best[kThreads];        // largest logit of each group of threads
  int sel[kThreads];
  uint64_t key[kCandidates], above;
  int n, n_sel;
};

// The number of keys above mine among the n.
__device__ __forceinline__ int rank_in(const uint64_t* key, int n, uint64_t mine) {
  int r = 0;
  for (int i = 0; i < n; ++i) r += key[i] > mine;
  return r;
}

// The largest `top` of the row's logits, in order, into smem keys: a bound from the
// threads' own largest values (top of them are logits of the row, so the smallest of
// the best `top` is one), then the logits of the threads that reach it once more,
// out of L2.  Returns how many keys there are (sorted ranks are found by the caller).
template <typename T>
__device__ int candidates(const RowUnits<T>& row, int top, float mine, TopSmem& sm) {
  const int t = threadIdx.x, threads = blockDim.x;
  int g = 1;   // threads a group: some four groups for each alternative
  while (g < 32 && threads / (2 * g) >= 4 * top) g *= 2;
  float b = mine;
  for (int o = 1; o < g; o *= 2) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
  const int groups = threads / g, i = t / g;
  if (t % g == 0) sm.best[i] = b;
  if (t == 0) {
    sm.n = sm.n_sel = 0;
    sm.above = (uint64_t)(kOrderNone + 1) << 32;
  }
  __syncthreads();
  int rank = 0;
  for (int j = t % g; j < groups; j += g) rank += sm.best[j] > b || (sm.best[j] == b && j < i);
  for (int o = 1; o < g; o *= 2) rank += __shfl_xor_sync(0xffffffffu, rank, o);
  if (rank == top - 1 && t % g == 0 && b > -INFINITY) sm.above = (uint64_t)order_of(b) << 32;
  __syncthreads();
  if (t % g == 0 && b > -INFINITY && order_of(b) >= (uint32_t)(sm.above >> 32))
    sm.sel[atomicAdd(&sm.n_sel, 1)] = i;
  __syncthreads();
  const int n_sel = sm.n_sel, rounds = (row.units + threads - 1) / threads;
  const int per = n_sel * g;
  for (;;) {
    const uint64_t above = sm.above;
    auto take = [&](float x, int j) {
      const uint64_t k = key_of(x, j);
      if (k < above) return;
      const int n = atomicAdd(&sm.n, 1);
      if (n < kCandidates) sm.key[n] = k;
    };
    const int j0 = row.loose(t);
    if (t < 2 * RowUnits<T>::E && j0 >= 0) take(to_f<T>(row.row[j0]), j0);
    for (int w = t; w < per * rounds; w += threads) {
      const int round = w / per, in = w - round * per;
      const int u = sm.sel[in / g] * g + in % g + round * threads;
      if (u >= row.units) continue;
      const uint4 v = load_unit(row.first() + u);
      uint4 one[1] = {v};
      if (order_of(largest<T, 1>(one)) < (uint32_t)(above >> 32)) continue;
#pragma unroll
      for (int e = 0; e < RowUnits<T>::E / 2; ++e) {
        const float2 x = pair<T>(v, e);
        take(x.x, row.head + u * RowUnits<T>::E + 2 * e);
        take(x.y, row.head + u * RowUnits<T>::E + 2 * e + 1);
      }
    }
    __syncthreads();
    const int n = sm.n;
    if (n <= kCandidates) return n;
    // More than there is room for (many equal logits, or a few threads hold most of the
    // large ones): the top-th of those stored is a better bound, since as many reach it.
    __syncthreads();
    for (int k = t; k < kCandidates; k += threads)
      if (rank_in(sm.key, kCandidates, sm.key[k]) == top - 1) sm.above = sm.key[k];
    if (t == 0) sm.n = 0;
    __syncthreads();
  }
}

// The teacher's and the given token's part of a row's loss.
__device__ __forceinline__ float teacher_value(const Teacher& t, int64_t i) {
  return t.f32 ? reinterpret_cast<const float*>(t.logits)[i]
               : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(t.logits)[i]);
}
// An entry of the teacher's list: its token (-1: none) and logit.
__device__ __forceinline__ int teacher_entry(const Teacher& t, const Rows& r, int p, int k, float* y) {
  const int64_t i = (int64_t)p * t.K + k;
  const int id = t.ids[i];
  *y = teacher_value(t, i);
  if (id >= r.V) report_status(r.status, (int)TSP_ERR_RANGE);
  return id >= 0 && id < r.V && !(*y == -INFINITY) ? id : -1;
}

// sum_k q_k (log q_k - log p_k) and whether there is an entry, for all threads: entry
// k is thread k's, y the teacher's logit, c its scale, logp the model's.
__device__ __forceinline__ float2 divergence(bool there, float y, float c, float logp,
                                             float (*part)[4]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const bool nan = there && !(y < INFINITY);
  const float mw = warp_max(there && !nan ? y : -INFINITY);
  float e = 0.f, x = 0.f;
  if (there) {
    e = nan ? NAN : expf(c * (y - mw));
    if (!(e == 0.f)) x = e * (c * (y - mw) - logp);
  }
  e = warp_sum(e);
  x = warp_sum(x);
  __syncthreads();
  if (lane == 0) {
    part[warp][0] = mw;
    part[warp][1] = e;
    part[warp][2] = x;
  }
  __syncthreads();
  float m = -INFINITY, se = 0.f, sx = 0.f;
  for (int w = 0; w < warps; ++w) m = fmaxf(m, part[w][0]);
  for (int w = 0; w < warps; ++w) {
    if (part[w][1] == 0.f) continue;
    const float d = c * (part[w][0] - m), f = expf(d);
    if (f == 0.f) continue;
    se += part[w][1] * f;
    sx += (part[w][2] + d * part[w][1]) * f;
  }
  return make_float2(sx / se - logf(se), se == 0.f ? 0.f : 1.f);
}

template <typename T, bool ENT>
__global__ void __launch_bounds__(kThreads, 2) fwd_kernel(const __grid_constant__ FwdArgs a) {
  constexpr int U = 4;
  __shared__ float part[kWarps][4];
  __shared__ TopSmem sm;
  const int t = threadIdx.x, threads = blockDim.x, r = blockIdx.x;
  const int p = pos_of(r, a.r.c, a.r.D);
  if (!TSP_INB(p >= 0 && p < a.r.S, a.r.status)) return;
  int64_t id = -1;
  bool live = true;
  if (a.r.ids) {
    id = load_id(a.r.ids, a.r.id_bytes, p);
    if (id >= a.r.V) {
      if (t == 0) report_status(a.r.status, (int)TSP_ERR_RANGE);
      id = -1;
    }
    live = id >= 0;
  }
  if (!live) {   // padding: the row is not looked at
    if (t == 0) {
      if (a.logp) a.logp[p] = 0.f;
      if (a.entropy) a.entropy[p] = 0.f;
      if (a.loss) a.loss[p] = 0.f;
      if (a.stats) {
        a.stats[2 * (int64_t)p] = 0.f;
        a.stats[2 * (int64_t)p + 1] = -INFINITY;
      }
    }
    for (int k = t; k < a.top; k += threads) {
      a.top_ids[(int64_t)p * a.top + k] = -1;
      a.top_logp[(int64_t)p * a.top + k] = -INFINITY;
    }
    return;
  }
  const RowUnits<T> row(a.r.logits, a.r.ld, r, a.r.V);
  const float c2 = a.r.scale * kLog2e, slack = kSlack / c2, low = lowest<T>();
  Sums<ENT> sums(low);
  const int j0 = t < 2 * RowUnits<T>::E ? row.loose(t) : -1;
  if (j0 >= 0) {
    const float x = to_f<T>(row.row[j0]);
    sums.see(x, c2, slack);
    sums.add(make_float2(x, -INFINITY), c2);
    sums.top = fmaxf(sums.top, x);
  }
  float mine = -INFINITY;   // of the units
  for (int u0 = t; u0 < row.units; u0 += U * threads) {
    uint4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      v[k] = u0 + k * threads < row.units ? load_unit(row.first() + u0 + k * threads) : no_unit<T>();
    const float b = largest<T, U>(v);
    mine = fmaxf(mine, b);
    sums.see(b, c2, slack);
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int e = 0; e < RowUnits<T>::E / 2; ++e) sums.add(pair<T>(v[k], e), c2);
  }
  const float target = id >= 0 && (a.logp || a.t.w_ce != 0.f) ? to_f<T>(row.row[id]) : 0.f;
  const Row x = join<ENT>(sums, low, c2, part);
  const float logp = x.l == -INFINITY ? -INFINITY : a.r.scale * (target - x.m) - x.l;
  if (t == 0) {
    if (a.logp) a.logp[p] = logp;
    if (a.entropy) a.entropy[p] = x.entropy;
    if (a.stats) {
      a.stats[2 * (int64_t)p] = x.m;
      a.stats[2 * (int64_t)p + 1] = x.l;
    }
  }
  if (a.loss) {
    float loss = a.t.w_ce != 0.f ? -a.t.w_ce * logp : 0.f;
    if (a.t.K > 0 && a.t.w_kd != 0.f) {
      float y = 0.f, lp = 0.f;
      int kid = -1;
      if (t < a.t.K) {
        kid = teacher_entry(a.t, a.r, p, t, &y);
        if (kid >= 0)
          lp = x.l == -INFINITY ? -INFINITY : a.r.scale * (to_f<T>(row.row[kid]) - x.m) - x.l;
      }
      const float2 kd = divergence(kid >= 0, y, a.t.scale, lp, part);
      if (kd.y != 0.f) loss += a.t.w_kd * kd.x;
    }
    if (t == 0) a.loss[p] = loss;
  }
  if (a.top > 0) {
    const int64_t at = (int64_t)p * a.top;
    int n = 0;
    if (!isnan(x.l)) n = candidates<T>(row, a.top, mine, sm);
    for (int k = t; k < n; k += threads) {
      const uint64_t key = sm.key[k];
      const int rank = rank_in(sm.key, n, key);
      if (rank < a.top) {
        a.top_ids[at + rank] = (int)~(uint32_t)key;
        a.top_logp[at + rank] = a.r.scale * (logit_of((uint32_t)(key >> 32)) - x.m) - x.l;
      }
    }
    for (int k = n + t; k < a.top; k += threads) {
      a.top_ids[at + k] = -1;
      a.top_logp[at + k] = isnan(x.l) ? x.l : -INFINITY;
    }
  }
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------
struct GradArgs {
  Rows r;
  void* out;
  int64_t ld_out;
  const float *stats, *entropy, *up, *up_entropy;   // up: dlogp, or dloss (NULL: 1)
  Teacher t;
  bool loss;
};

// What the listed tokens add: entry k < K the teacher's, entry K the given token.
struct Adds {
  alignas(16) int id[TSP_TOP_MAX + 4];   // (-1 up to the next multiple of four)
  float add[TSP_TOP_MAX + 1];
};
__device__ __forceinline__ void end_adds(Adds& adds, int n, int t) {
  if (t < 3) adds.id[n + t] = -1;
}
// An entry's token (-1: none of this part's, or not the first entry of its token) and
// what all entries of the token add, in the order of the list.
__device__ __forceinline__ int added(const Adds& adds, int n, int k, float* sum) {
  const int j = adds.id[k];
  *sum = 0.f;
  if (j < 0) return -1;
  int same = 0;
  for (int q = 0; q < n; q += 4) {
    const int4 o = *reinterpret_cast<const int4*>(adds.id + q);
    same += (o.x == j) + (o.y == j) + (o.z == j) + (o.w == j);
  }
  if (same == 1) {
    *sum = adds.add[k];
    return j;
  }
  bool first = true;
  for (int q = 0; q < n; ++q)
    if (adds.id[q] == j) {
      *sum += adds.add[q];
      first &= q >= k;
    }
  return first ? j : -1;
}

// A part of a row a CTA: dx_j = p_j (A + B log p_j), then the listed tokens' values
// once more with what they add (the same token twice adds twice; the first of its
// entries writes the value).
template <typename T, bool ENT, int E>
__global__ void __launch_bounds__(kThreads, 2) grad_kernel(const __grid_constant__ GradArgs a) {
  constexpr int U = 4;
  typedef typename std::conditional<E == 1, T, uint4>::type Unit;
  __shared__ float part[kWarps][4];
  __shared__ Adds adds;
  const int t = threadIdx.x, threads = blockDim.x, r = blockIdx.x;
  const int p = pos_of(r, a.r.c, a.r.D);
  if (!TSP_INB(p >= 0 && p < a.r.S, a.r.status)) return;
  int64_t id = -1;
  if (a.r.ids) id = load_id(a.r.ids, a.r.id_bytes, p);
  if (id >= a.r.V) {
    if (t == 0) report_status(a.r.status, (int)TSP_ERR_RANGE);
    id = -1;
  }
  const float m = a.stats[2 * (int64_t)p], l = a.stats[2 * (int64_t)p + 1];
  const bool live = !(a.r.ids && id < 0) && l != -INFINITY;
  const T* x = reinterpret_cast<const T*>(a.r.logits) + (int64_t)r * a.r.ld;
  T* out = reinterpret_cast<T*>(a.out) + (int64_t)r * a.ld_out;
  const int head = E == 1 ? 0 : min(a.r.V, (int)((16 - ((uintptr_t)x & 15)) & 15) / (int)sizeof(T));
  const int units = (a.r.V - head) / E, tail = head + units * E;
  const Unit* xu = reinterpret_cast<const Unit*>(x + head);
  Unit* ou = reinterpret_cast<Unit*>(out + head);
  // the part of this CTA: units [u_lo, u_hi), and the loose elements with the first part
  const int per = (units + gridDim.y - 1) / gridDim.y;
  const int u_lo = min(units, (int)blockIdx.y * per), u_hi = min(units, u_lo + per);
  const int lo = blockIdx.y == 0 ? 0 : head + u_lo * E;
  const int hi = blockIdx.y == gridDim.y - 1 ? a.r.V : head + u_hi * E;
  float A = 0.f, B = 0.f;
  int n = 0;
  const float c = a.r.scale, c2 = c * kLog2e, l2 = l * kLog2e;
  float at_list[2] = {0.f, 0.f};   // logits of the listed tokens, read before they may be overwritten
  if (live) {
    const float up = a.up ? a.up[p] : 1.f;
    if (a.loss) {
      float w = a.t.w_ce;
      if (a.t.K > 0 && a.t.w_kd != 0.f) {
        float y = 0.f;
        int kid = -1;
        if (t < a.t.K) kid = teacher_entry(a.t, a.r, p, t, &y);
        const int lane = t & 31, warp = t >> 5;
        const float mw = warp_max(kid >= 0 ? y : -INFINITY);
        if (lane == 0) part[warp][0] = mw;
        __syncthreads();
        float mt = -INFINITY;
        for (int k = 0; k < threads / 32; ++k) mt = fmaxf(mt, part[k][0]);
        const float e = kid >= 0 ? expf(a.t.scale * (y - mt)) : 0.f;
        const float sw = warp_sum(e);
        if (lane == 0) part[warp][1] = sw;
        __syncthreads();
        float se = 0.f;
        for (int k = 0; k < threads / 32; ++k) se += part[k][1];
        if (t < a.t.K) {
          adds.id[t] = kid >= lo && kid < hi ? kid : -1;
          adds.add[t] = -up * c * a.t.w_kd * (e / se);
        }
        n = a.t.K;
        if (se != 0.f) w += a.t.w_kd;
      }
      A = up * c * w;
      if (t == 0) {
        adds.id[n] = id >= lo && id < hi && a.t.w_ce != 0.f ? (int)id : -1;
        adds.add[n] = -up * c * a.t.w_ce;
      }
    } else {
      const float de = ENT ? a.up_entropy[p] : 0.f;
      A = a.up ? -c * up : 0.f;
      if (ENT) {
        A -= c * de * a.entropy[p];
        B = -c * de * kLn2;
      }
      if (t == 0) {
        adds.id[0] = a.up && id >= lo && id < hi ? (int)id : -1;
        adds.add[0] = c * up;
      }
    }
    ++n;
    end_adds(adds, n, t);
    __syncthreads();
    for (int k = t, i = 0; k < n; k += threads, ++i)
      if (adds.id[k] >= 0) at_list[i] = to_f<T>(x[adds.id[k]]);
    __syncthreads();
  }
  auto grad = [&](float2 v) {
    if (!live) return make_float2(0.f, 0.f);
    const float2 u = ffma2(fadd2(v, make_float2(-m, -m)), make_float2(c2, c2), make_float2(-l2, -l2));
    const float2 q = make_float2(ex2_approx(u.x), ex2_approx(u.y));
    float2 w = make_float2(A, A);
    if (ENT) w = ffma2(make_float2(fmaxf(u.x, kLeast), fmaxf(u.y, kLeast)), make_float2(B, B), w);
    return fmul2(q, w);
  };
  if (E > 1 && t < 2 * E) {
    const int j = t < head ? t : tail + t - head;
    if (j < a.r.V && (j < head ? blockIdx.y == 0 : blockIdx.y == gridDim.y - 1))
      out[j] = from_f<T>(grad(make_float2(live ? to_f<T>(x[j]) : 0.f, 0.f)).x);
  }
  for (int u0 = u_lo + t; u0 < u_hi; u0 += U * threads) {
    Unit v[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (live && u0 + k * threads < u_hi) {
        if constexpr (E == 1) v[k] = xu[u0 + k * threads];
        else v[k] = load_unit(xu + u0 + k * threads);
      }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (u0 + k * threads >= u_hi) continue;
      if constexpr (E == 1) {
        ou[u0 + k * threads] = from_f<T>(grad(make_float2(live ? to_f<T>(v[k]) : 0.f, 0.f)).x);
      } else if (!live) {
        ou[u0 + k * threads] = make_uint4(0, 0, 0, 0);
      } else if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 g = grad(pair<T>(v[k], e));
          w[e] = pack2<T>(g.x, g.y);
        }
        __stcs(ou + u0 + k * threads, make_uint4(w[0], w[1], w[2], w[3]));
      } else {
        const float2 g = grad(pair<T>(v[k], 0)), h = grad(pair<T>(v[k], 1));
        __stcs(ou + u0 + k * threads, make_uint4(__float_as_uint(g.x), __float_as_uint(g.y),
                                                 __float_as_uint(h.x), __float_as_uint(h.y)));
      }
    }
  }
  if (!live) return;
  __syncthreads();
  for (int k = t, i = 0; k < n; k += threads, ++i) {
    float sum;
    const int j = added(adds, n, k, &sum);
    if (j >= 0) out[j] = from_f<T>(grad(make_float2(at_list[i], 0.f)).x + sum);
  }
}

// ---------------------------------------------------------------------------
// Loss and gradient in one pass
// ---------------------------------------------------------------------------
// A row stays in shared memory between its sum and its gradient, so that it is read
// once and written once.  A CTA, or for long rows a cluster whose CTAs hold a part
// each, takes one row after the other; its threads copy the next row's units into the
// places whose gradient they have just written, so that reading goes on while the
// sums are joined.  A thread copies what it will itself read: the data need no barrier.
// Between the CTAs of a cluster go, through distributed shared memory, their sums and
// the logits of the listed tokens.
constexpr int kOneThreads = 256, kOneCtas = 3;
constexpr int kOnePassPart = 66 * 1024;    // bytes of a row a CTA: three CTAs a multiprocessor
constexpr int kOnePassMost = 200 * 1024;   // ... of the longest rows: one

__device__ __forceinline__ void copy_unit(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_sent() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_left_c() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// until at most n (or eight) of the groups sent last are on their way
__device__ __forceinline__ void copies_left(int n) {
  switch (n) {
    case 0: copies_left_c<0>(); break;
    case 1: copies_left_c<1>(); break;
    case 2: copies_left_c<2>(); break;
    case 3: copies_left_c<3>(); break;
    case 4: copies_left_c<4>(); break;
    case 5: copies_left_c<5>(); break;
    case 6: copies_left_c<6>(); break;
    case 7: copies_left_c<7>(); break;
    default: copies_left_c<8>();
  }
}

struct OnePassArgs {
  GradArgs g;
  float *loss, *stats;
};
// What the CTAs of a cluster write into each other: of two rows, since one of them may
// be a row ahead.
struct Exchange {
  float2 share[8];               // (largest logit, sum) of each part
  float target, z[TSP_TOP_MAX];  // (in the first CTA) logits of the given and the teacher's tokens
};
struct OnePassSmem {
  float part[kOneThreads / 32][4], teach[kOneThreads / 32][2];
  Exchange ex[2];
  Adds adds;                     // of this part
  float z[TSP_TOP_MAX + 1];      // the listed tokens' logits
  float q[TSP_TOP_MAX], logq[TSP_TOP_MAX];
  float loose[16];
};

template <typename T, bool CLUSTER>
__global__ void __launch_bounds__(kOneThreads, kOneCtas) one_pass_kernel(const __grid_constant__ OnePassArgs o) {
  constexpr int E = 16 / sizeof(T), U = 4;
  extern __shared__ uint4 seg[];
  __shared__ OnePassSmem sm;
  const GradArgs& a = o.g;
  const int t = threadIdx.x, threads = blockDim.x, lane = t & 31, warp = t >> 5;
  const auto cluster = cooperative_groups::this_cluster();
  const int rank = CLUSTER ? (int)cluster.block_rank() : 0;
  const int parts = CLUSTER ? (int)cluster.num_blocks() : 1;
  const int stride = gridDim.x / parts;
  const float c = a.r.scale, c2 = c * kLog2e, low = lowest<T>(), slack = kSlack / c2;
  const int K = a.t.w_kd != 0.f ? a.t.K : 0;
  // the units of a row that are this part's
  struct Part {
    const uint4* src;
    int u_lo, n;
  };
  auto part_of = [&](const RowUnits<T>& row) {
    const int per = (row.units + parts - 1) / parts, u_lo = min(row.units, rank * per);
    return Part{row.first() + u_lo, u_lo, min(row.units, u_lo + per) - u_lo};
  };
  auto given = [&](int r) {   // a row's token: -1 for padding, -2 without tokens
    if (r >= a.r.S || !a.r.ids) return -2;
    const int64_t id = load_id(a.r.ids, a.r.id_bytes, pos_of(r, a.r.c, a.r.D));
    if (id >= a.r.V && t == 0) report_status(a.r.status, (int)TSP_ERR_RANGE);
    return id >= 0 && id < a.r.V ? (int)id : -1;
  };
  // the copies of a row's units i + k * threads, k < U
  auto send = [&](const Part& x, int i) {
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (i + k * threads < x.n) copy_unit(seg + i + k * threads, x.src + i + k * threads);
    copies_sent();
  };
  const int most = (a.r.V / E + parts - 1) / parts;      // units of a part at most
  const int groups = (most + U * threads - 1) / (U * threads);
  int r = CLUSTER ? blockIdx.x / parts : blockIdx.x;
  int id = given(r);
  // (the CTAs of a cluster have started before one writes into another's memory)
  if (CLUSTER) cluster.sync();
  bool there = false;   // this row's copies have been sent
  for (int turn = 0; r < a.r.S; r += stride) {
    const int p = pos_of(r, a.r.c, a.r.D);
    if (!TSP_INB(p >= 0 && p < a.r.S, a.r.status)) return;
    const bool live = id != -1;
    const RowUnits<T> row(a.r.logits, a.r.ld, r, a.r.V);
    const Part x = part_of(row);
    const int lo = rank == 0 ? 0 : row.head + x.u_lo * E;
    const int hi = rank == parts - 1 ? a.r.V : row.head + (x.u_lo + x.n) * E;
    T* out = reinterpret_cast<T*>(a.out) + (int64_t)r * a.ld_out;
    uint4* dst = reinterpret_cast<uint4*>(out + row.head) + x.u_lo;
    const int j0 = t < 2 * E ? row.loose(t) : -1;
    const bool mine = j0 >= lo && j0 < hi;   // a loose element of this part
    const int id_next = given(r + stride);
    Exchange& ex = sm.ex[turn];
    float m = 0.f, l = -INFINITY, A = 0.f, x0 = -INFINITY;
    int n = 0;
    if (live) {
      if (!there)
        for (int g = 0; g < groups; ++g) send(x, t + U * g * threads);
      if (mine) x0 = to_f<T>(row.row[j0]);
      float y = 0.f;
      int kid = -1;
      if (t < K) kid = teacher_entry(a.t, a.r, p, t, &y);
      const float up = a.up ? a.up[p] : 1.f;
      Sums<false> sums(low);
      for (int g = 0; g < groups; ++g) {
        copies_left(groups - 1 - g);
        const int i = t + U * g * threads;
        if (i + (U - 1) * threads < x.n) {
          uint4 v[U];
#pragma unroll
          for (int k = 0; k < U; ++k) v[k] = seg[i + k * threads];
          sums.see(largest<T, U>(v), c2, slack);
#pragma unroll
          for (int k = 0; k < U; ++k)
#pragma unroll
            for (int e = 0; e < E / 2; ++e) sums.add(pair<T>(v[k], e), c2);
        } else {
          for (int k = i; k < x.n; k += threads) {
            const uint4 v[1] = {seg[k]};
            sums.see(largest<T, 1>(v), c2, slack);
#pragma unroll
            for (int e = 0; e < E / 2; ++e) sums.add(pair<T>(v[0], e), c2);
          }
        }
      }
      sums.see(x0, c2, slack);
      sums.add(make_float2(x0, -INFINITY), c2);
      if (mine) sm.loose[t] = x0;
      if (K > 0) {
        const float mw = warp_max(kid >= 0 ? y : -INFINITY);
        const float sw = warp_sum(kid >= 0 ? expf(a.t.scale * (y - mw)) : 0.f);
        if (lane == 0) {
          sm.teach[warp][0] = mw;
          sm.teach[warp][1] = sw;
        }
      }
      float s;
      join_sums<false>(sums, low, c2, sm.part, &m, &s, nullptr);
      // every logit of this part is in shared memory: hand on the listed ones
      auto logit = [&](int j) {
        return j < row.head    ? sm.loose[j]
               : j >= row.tail ? sm.loose[row.head + j - row.tail]
                               : to_f<T>(reinterpret_cast<const T*>(seg)[j - row.head - x.u_lo * E]);
      };
      Exchange* first = CLUSTER ? cluster.map_shared_rank(&ex, 0) : &ex;
      const bool here = kid >= lo && kid < hi, given_here = id >= lo && id < hi;
      if (here) first->z[t] = sm.z[t] = logit(kid);
      if (t == 0 && given_here) first->target = sm.z[K] = logit(id);
      if (CLUSTER) {
        if (t < parts) cluster.map_shared_rank(&ex, t)->share[rank] = make_float2(m, s);
        cluster.sync();
        m = low;
        for (int k = 0; k < parts; ++k) m = fmaxf(m, ex.share[k].x);
        s = 0.f;
        for (int k = 0; k < parts; ++k)
          s += ex.share[k].y * ex2_approx(fmaxf((ex.share[k].x - m) * c2, kLeast));
      }
      if (s == 0.f) m = 0.f;
      l = s == 0.f ? -INFINITY : logf(s);
      float w = a.t.w_ce;
      if (K > 0) {
        const float from = lane < threads / 32 ? sm.teach[lane][0] : -INFINITY, mt = warp_max(from);
        float se = lane < threads / 32 ? sm.teach[lane][1] : 0.f;
        if (se != 0.f) se *= expf(a.t.scale * (from - mt));
        se = warp_sum(se);
        if (t < K) {
          const float logq = a.t.scale * (y - mt) - logf(se), q = kid >= 0 ? expf(a.t.scale * (y - mt)) / se : 0.f;
          sm.q[t] = q;
          sm.logq[t] = logq;
          sm.adds.id[t] = here ? kid : -1;
          sm.adds.add[t] = -up * c * a.t.w_kd * q;
        }
        if (se != 0.f) w += a.t.w_kd;
      }
      if (t == 0) {
        sm.adds.id[K] = given_here && a.t.w_ce != 0.f ? id : -1;
        sm.adds.add[K] = -up * c * a.t.w_ce;
      }
      end_adds(sm.adds, K + 1, t);
      A = up * c * w;
      n = l == -INFINITY ? 0 : K + 1;
      if (!CLUSTER) __syncthreads();   // (the listed logits are read before the next row comes in)
    }
    const bool flat = !live || l == -INFINITY;   // a zero gradient
    const float l2 = l * kLog2e;
    auto grad = [&](float2 v) {
      const float2 u = ffma2(fadd2(v, make_float2(-m, -m)), make_float2(c2, c2), make_float2(-l2, -l2));
      return fmul2(make_float2(ex2_approx(u.x), ex2_approx(u.y)), make_float2(A, A));
    };
    if (mine) out[j0] = from_f<T>(flat ? 0.f : grad(make_float2(x0, 0.f)).x);
    there = r + stride < a.r.S && id_next != -1;
    Part next = {nullptr, 0, 0};
    if (there) next = part_of(RowUnits<T>(a.r.logits, a.r.ld, r + stride, a.r.V));
    auto put_unit = [&](int i) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (!flat) {
        const uint4 v = seg[i];
        if constexpr (sizeof(T) == 2) {
          const float2 g0 = grad(pair<T>(v, 0)), g1 = grad(pair<T>(v, 1));
          const float2 g2 = grad(pair<T>(v, 2)), g3 = grad(pair<T>(v, 3));
          w = make_uint4(pack2<T>(g0.x, g0.y), pack2<T>(g1.x, g1.y), pack2<T>(g2.x, g2.y),
                         pack2<T>(g3.x, g3.y));
        } else {
          const float2 g0 = grad(pair<T>(v, 0)), g1 = grad(pair<T>(v, 1));
          w = make_uint4(__float_as_uint(g0.x), __float_as_uint(g0.y), __float_as_uint(g1.x),
                         __float_as_uint(g1.y));
        }
      }
      __stcs(dst + i, w);
    };
    for (int g = 0; g < groups; ++g) {
      const int i0 = t + U * g * threads;
      if (i0 + (U - 1) * threads < x.n) {
#pragma unroll
        for (int k = 0; k < U; ++k) put_unit(i0 + k * threads);
      } else {
        for (int i = i0; i < x.n; i += threads) put_unit(i);
      }
      if (there) send(next, i0);
    }
    if (live) {
      __syncthreads();   // the listed tokens' values go on top of what other threads wrote
      auto put = [&](int k) {
        float sum;
        const int j = added(sm.adds, n, k, &sum);
        if (j >= 0) out[j] = from_f<T>(grad(make_float2(sm.z[k], 0.f)).x + sum);
      };
      if (t < K && n > 0) put(t);
      if (t == 0 && n > 0) put(K);
    }
    if (rank == 0 && warp == 0) {
      float loss = 0.f;
      if (live) {
        if (a.t.w_ce != 0.f && id >= 0) loss = -a.t.w_ce * (l == -INFINITY ? l : c * (ex.target - m) - l);
        float kd = 0.f;
        bool any = false;
        for (int k = lane; k < K; k += 32) {
          const float q = sm.q[k];
          any |= q != 0.f;
          if (q != 0.f) kd += q * (sm.logq[k] - (l == -INFINITY ? l : c * (ex.z[k] - m) - l));
        }
        kd = warp_sum(kd);
        if (__any_sync(0xffffffffu, any)) loss += a.t.w_kd * kd;
      }
      if (lane == 0) {
        o.loss[p] = loss;
        o.stats[2 * (int64_t)p] = m;
        o.stats[2 * (int64_t)p + 1] = l;
      }
    }
    if (live) turn ^= 1;
    id = id_next;
  }
}

Rows rows_of(const tsp_logits& x, const void* ids, int id_bytes) {
  Rows r;
  r.logits = x.logits;
  r.ld = x.ld;
  r.ids = ids;
  r.id_bytes = id_bytes;
  r.S = (int)x.S;
  r.c = (int)(x.S / (2 * x.D));
  r.D = x.D;
  r.V = (int)x.V;
  r.scale = x.scale;
  r.status = status_word();
  return r;
}
Teacher teacher_of(const tsp_teacher* t, float w_ce) {
  Teacher k = {nullptr, nullptr, 0, 0, 1.f, w_ce, 0.f};
  if (t) {
    k.ids = t->ids;
    k.logits = t->logits;
    k.f32 = t->dtype == TSP_F32;
    k.K = t->K;
    k.scale = t->scale;
    k.w_kd = t->weight;
  }
  return k;
}

// Threads of a CTA for rows of V elements and lists of n: one for each unit up to 512.
int threads_for(int64_t V, int dtype, int n) {
  const int64_t units = V * (dtype == TSP_F32 ? 4 : 2) / 16;
  int t = 128;
  while (t < kThreads && (t < n || t * 4 <= units)) t *= 2;
  return t;
}

tsp_status launch_fwd(const FwdArgs& a, int dtype, const char* name, cudaStream_t st) {
  Prof prof(name, st);
  const int threads = threads_for(a.r.V, dtype, std::max(a.top, a.t.K));
  const bool ent = a.entropy != nullptr;
  if (dtype == TSP_BF16)
    ent ? fwd_kernel<__nv_bfloat16, true><<<a.r.S, threads, 0, st>>>(a)
        : fwd_kernel<__nv_bfloat16, false><<<a.r.S, threads, 0, st>>>(a);
  else
    ent ? fwd_kernel<float, true><<<a.r.S, threads, 0, st>>>(a)
        : fwd_kernel<float, false><<<a.r.S, threads, 0, st>>>(a);
  TSP_CUDA_TRY(cudaGetLastError());
  return TSP_OK;
}

template <typename T>
bool alike(const GradArgs& a) {   // rows that lie alike on 16-byte units
  return ((uintptr_t)a.r.logits - (uintptr_t)a.out) % 16 == 0 &&
         (a.r.S == 1 || (a.r.ld - a.ld_out) * (int64_t)sizeof(T) % 16 == 0);
}

template <typename T, bool ENT>
void grad_t(const GradArgs& a, dim3 grid, int threads, cudaStream_t st) {
  // rows that lie alike on 16-byte units are read and written in units, others by element
  if (alike<T>(a)) grad_kernel<T, ENT, 16 / (int)sizeof(T)><<<grid, threads, 0, st>>>(a);
  else grad_kernel<T, ENT, 1><<<grid, threads, 0, st>>>(a);
}
tsp_status launch_grad(const GradArgs& a, int dtype, const char* name, cudaStream_t st) {
  Prof prof(name, st);
  const int threads = threads_for(a.r.V, dtype, a.t.K);
  const int64_t units = (int64_t)a.r.V * (dtype == TSP_F32 ? 4 : 2) / 16;
  const dim3 grid(a.r.S, (unsigned)std::min<int64_t>(1024, std::max<int64_t>(1, units / (16 * threads))));
  const bool ent = a.up_entropy != nullptr;
  if (dtype == TSP_BF16)
    ent ? grad_t<__nv_bfloat16, true>(a, grid, threads, st)
        : grad_t<__nv_bfloat16, false>(a, grid, threads, st);
  else
    ent ? grad_t<float, true>(a, grid, threads, st) : grad_t<float, false>(a, grid, threads, st);
  TSP_CUDA_TRY(cudaGetLastError());
  return TSP_OK;
}

// The most dynamic shared memory a kernel may be launched with, set once.
template <auto KERNEL>
tsp_status allow_smem(int most) {
  static std::atomic<bool> set[kMaxDevices];
  const int dev = current_device();
  if (!set[dev]) {
    TSP_CUDA_TRY(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
    set[dev] = true;
  }
  return TSP_OK;
}

// How many clusters (CTAs, if those are alone) of a launch the GPU holds at once,
// looked up once for each kind of launch: a persistent grid takes as many.
int64_t resident(const void* kernel, const cudaLaunchConfig_t& cfg, int parts) {
  struct Known {
    const void* kernel;
    size_t smem;
    int dev, parts, threads, n;
  };
  static std::mutex mu;
  static Known known[32];   // (the oldest gives way)
  static unsigned at = 0;
  const int dev = current_device(), threads = (int)cfg.blockDim.x;
  std::lock_guard<std::mutex> lk(mu);
  for (const Known& k : known)
    if (k.kernel == kernel && k.smem == cfg.dynamicSmemBytes && k.dev == dev && k.parts == parts && k.threads == threads)
      return k.n;
  int n = 0;
  if (parts > 1) {
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) n = 0;
  } else if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, cfg.dynamicSmemBytes) == cudaSuccess) {
    n *= num_sms();
  } else {
    n = 0;
  }
  n = n > 0 ? n : std::max(1, num_sms() / parts);
  known[at++ % 32] = {kernel, cfg.dynamicSmemBytes, dev, parts, threads, n};
  return n;
}

template <typename T, bool CLUSTER>
tsp_status launch_one_pass_c(const OnePassArgs& o, int parts, cudaStream_t st) {
  const int64_t per = ((int64_t)o.g.r.V * sizeof(T) / 16 + parts - 1) / parts;
  int threads = 128;
  while (threads < kOneThreads && (threads < o.g.t.K || threads * 4 <= per)) threads *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (size_t)per * 16;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = parts;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CLUSTER ? 1 : 0;
  constexpr auto kernel = one_pass_kernel<T, CLUSTER>;
  const tsp_status r = allow_smem<kernel>(kOnePassMost);
  if (r != TSP_OK) return r;
  cfg.gridDim = dim3((unsigned)parts);
  cfg.gridDim = dim3((unsigned)(std::min<int64_t>(o.g.r.S, resident((const void*)kernel, cfg, parts)) * parts));
  Prof prof("token_loss_one_pass", st);
  TSP_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, o));
  return TSP_OK;
}
template <typename T>
tsp_status launch_one_pass_t(const OnePassArgs& o, int parts, cudaStream_t st) {
  return parts > 1 ? launch_one_pass_c<T, true>(o, parts, st) : launch_one_pass_c<T, false>(o, parts, st);
}

// CTAs a row for the loss with its gradient: parts of 66 KB at most, 200 KB in
// clusters of eight; for few rows more, down to 4 KB.  0: the row is too long.
int one_pass_parts(int64_t S, int64_t units) {
  int64_t parts = std::max<int64_t>(1, (units * 16 + kOnePassPart - 1) / kOnePassPart);
  if (parts > 8) parts = (units + 7) / 8 * 16 <= kOnePassMost ? 8 : 0;
  while (parts > 0 && parts <= 4 && S * parts < num_sms() && units / (2 * parts) >= 256) parts *= 2;
  return (int)parts;
}

}  // namespace

tsp_status launch_logprobs_fwd(const tsp_logits& x, const void* ids, int id_bytes, float* logp,
                               float* entropy, float* stats, int* top_ids, float* top_logp, int top,
                               cudaStream_t st) {
  FwdArgs a = {};
  a.r = rows_of(x, ids, id_bytes);
  a.t = teacher_of(nullptr, 0.f);
  a.logp = logp;
  a.entropy = entropy;
  a.stats = stats;
  a.top_ids = top_ids;
  a.top_logp = top_logp;
  a.top = top;
  return launch_fwd(a, x.dtype, "logprobs_fwd", st);
}

tsp_status launch_logprobs_bwd(const tsp_logits& x, const void* ids, int id_bytes, const float* stats,
                               const float* entropy, const float* dlogp, const float* dentropy,
                               void* dlogits, int64_t ld_d, cudaStream_t st) {
  GradArgs a = {};
  a.r = rows_of(x, ids, id_bytes);
  a.t = teacher_of(nullptr, 0.f);
  a.out = dlogits;
  a.ld_out = ld_d;
  a.stats = stats;
  a.entropy = entropy;
  a.up = dlogp;
  a.up_entropy = dentropy;
  return launch_grad(a, x.dtype, "logprobs_bwd", st);
}

tsp_status launch_token_loss_bwd(const tsp_logits& x, const void* ids, int id_bytes, float w_ce,
                                 const tsp_teacher* teacher, const float* stats, const float* dloss,
                                 void* dlogits, int64_t ld_d, cudaStream_t st) {
  GradArgs a = {};
  a.r = rows_of(x, ids, id_bytes);
  a.t = teacher_of(teacher, w_ce);
  a.out = dlogits;
  a.ld_out = ld_d;
  a.stats = stats;
  a.up = dloss;
  a.loss = true;
  return launch_grad(a, x.dtype, "token_loss_bwd", st);
}

tsp_status launch_token_loss_fwd(const tsp_logits& x, const void* ids, int id_bytes, float w_ce,
                                 const tsp_teacher* teacher, float* loss, float* stats,
                                 const float* dloss, void* dlogits, int64_t ld_d, cudaStream_t st) {
  if (dlogits) {
    OnePassArgs o = {};
    o.g.r = rows_of(x, ids, id_bytes);
    o.g.t = teacher_of(teacher, w_ce);
    o.g.out = dlogits;
    o.g.ld_out = ld_d;
    o.g.up = dloss;
    o.loss = loss;
    o.stats = stats;
    const bool bf = x.dtype == TSP_BF16;
    const int parts = one_pass_parts(x.S, x.V * (bf ? 2 : 4) / 16);
    if (parts > 0 && (bf ? alike<__nv_bfloat16>(o.g) : alike<float>(o.g)))
      return bf ? launch_one_pass_t<__nv_bfloat16>(o, parts, st) : launch_one_pass_t<float>(o, parts, st);
  }
  FwdArgs a = {};
  a.r = rows_of(x, ids, id_bytes);
  a.t = teacher_of(teacher, w_ce);
  a.loss = loss;
  a.stats = stats;
  const tsp_status r = launch_fwd(a, x.dtype, "token_loss_fwd", st);
  if (r != TSP_OK || !dlogits) return r;
  return launch_token_loss_bwd(x, ids, id_bytes, w_ce, teacher, stats, dloss, dlogits, ld_d, st);
}

}  // namespace tsp
