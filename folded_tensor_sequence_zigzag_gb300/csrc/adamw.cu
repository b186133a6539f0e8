// adamw.cu -- one AdamW update of many tensors in a few launches.
//
//   g = grad * gscale
//   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
//   w = w (1 - lr wd) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
//
// in fp32, each operation rounded by itself (no contraction), so the result is
// the same as the formula's evaluated one elementary operation at a time.  w is
// the fp32 master where there is one, else the weight itself; the weight is
// then the master rounded to its type, and `prep` the weight as the fp16
// operand copy of the prepared block calls, so no conversion pass follows the
// update.
//
// 8-bit states.  Blocks of 128 elements share an fp32 scale, the largest
// magnitude times 1/448; an element is held as e4m3 of value * (448 * (1 /
// largest)): one reciprocal a block instead of a division an element.
// m is held so, and of v its square root, which halves the range that the
// eight bits have to span and is what the update divides by.  A positive root
// never becomes code 0: the smallest code 2^-9 stands for it, so that an
// element next to a much larger one is not divided by eps alone.
//
// Bound by HBM: every element is read and written once.
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include <atomic>
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "kernels.h"

namespace tsp {

namespace {

constexpr int kTensors = 128;       // tensors of one launch (the descriptors are kernel arguments)
constexpr int kChunk = 4096;        // elements a CTA takes at a time: 8 warps x 4 x 128
constexpr float kScaleFloor = 7.888609052210118e-31f;   // 2^-100

struct Tensor {
  int64_t n;
  void* w;
  float* master;
  const float* g;
  void *m, *v;
  float *ms, *vs;
  __half* prep;
  float wd;
};
struct Args {
  Tensor t[kTensors];
  int64_t end[kTensors];   // chunks of tensors 0..i
  int count;
  int run;                 // consecutive chunks of a CTA (8-bit states)
  float b1, c1, b2, c2;    // beta, 1 - beta
  float eps, neg_zero;
  float lr, step_size, fix;   // lr, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  double dbeta1, dbeta2;
  const float* lr_dev;
  const int64_t* step_dev;
  const float* gscale;
  const int* held;   // the status word as the call found it (not in the cluster forms)
  int* status;
};

// While the status word holds an error the contraction kernels leave their outputs as
// they are, gradients among them, so an update made of those must not reach weights and
// states.  All CTAs of all of a call's launches have to decide alike, though an error
// may be recorded while they run (by this call too: a weight past fp16), or half of the
// tensors would be updated.  So the word is copied once, where the stream reaches the
// call, and the kernels look at the copy.  A call's place among the copies comes round
// again after kHeldPlaces calls, and captured calls, which keep theirs, have a set of
// their own.  (The first kernel follows this one as a dependent launch: 3 us of a
// call, 1 us in a graph; a copy of four bytes by the driver costs 4 us of a call.)
// Up to kClusterChunks chunks the grid is one cluster, whose first CTA looks at the word
// for all of them: nine tensors of the tiny block (12 chunks) take 13 us a call so, 16
// with the copy; in a graph 4.5 either way.
constexpr unsigned kHeldPlaces = 32768;
constexpr int kClusterChunks = 16;
__device__ int g_held[2][kHeldPlaces];

__global__ void adamw_held_kernel(int* held, const int* status) { *held = *status; }

tsp_status take_held(const int* status, cudaStream_t st, const int** held) {
  if (!status) return TSP_ERR_CUDA;
  static int* base[kMaxDevices] = {nullptr};
  static std::atomic<unsigned> calls[2];
  const int dev = current_device();
  if (!base[dev]) {
    void* p = nullptr;
    TSP_CUDA_TRY(cudaGetSymbolAddress(&p, g_held));
    base[dev] = (int*)p;
  }
  cudaStreamCaptureStatus capturing;
  TSP_CUDA_TRY(cudaStreamIsCapturing(st, &capturing));
  const int set = capturing != cudaStreamCaptureStatusNone;
  int* at = base[dev] + set * kHeldPlaces + calls[set].fetch_add(1) % kHeldPlaces;
  adamw_held_kernel<<<1, 1, 0, st>>>(at, status);
  TSP_CUDA_TRY(cudaGetLastError());
  *held = at;
  return TSP_OK;
}

// The status word as the first CTA of the cluster finds it, the same in all of its CTAs.
__device__ __forceinline__ int held_in_cluster(const Args& a) {
  __shared__ int word;
  const auto cluster = cooperative_groups::this_cluster();
  if (threadIdx.x == 0 && cluster.block_rank() == 0) word = *(const volatile int*)a.status;
  cluster.sync();
  const int held = *cluster.map_shared_rank(&word, 0);
  cluster.sync();   // (read by all before the first one may end)
  return held;
}

// x^n by squaring, n >= 1
__device__ double power(double x, int64_t n) {
  double r = 1.0;
  for (; n > 0; n >>= 1, x *= x)
    if (n & 1) r *= x;
  return r;
}

// The k (of four) elements at p; ALL: k is known to be four.
template <bool ALL, typename T>
__device__ __forceinline__ void load4(const T* p, int k, float (&v)[4]) {
  if (!ALL && k != 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = e < k ? to_f<T>(p[e]) : 0.f;
  } else if constexpr (sizeof(T) == 4) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = lo2<T>(u.x); v[1] = hi2<T>(u.x); v[2] = lo2<T>(u.y); v[3] = hi2<T>(u.y);
  }
}
template <bool ALL, typename T>
__device__ __forceinline__ void store4(T* p, int k, const float (&v)[4]) {
  if (!ALL && k != 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < k) p[e] = from_f<T>(v[e]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
  }
}
template <bool ALL>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int k) {
  if (ALL || k == 4) return *reinterpret_cast<const uint32_t*>(p);
  uint32_t u = 0;
  for (int e = 0; e < k; ++e) u |= (uint32_t)p[e] << (8 * e);
  return u;
}
template <bool ALL>
__device__ __forceinline__ void store_codes(uint8_t* p, int k, uint32_t u) {
  if (ALL || k == 4) {
    *reinterpret_cast<uint32_t*>(p) = u;
    return;
  }
  for (int e = 0; e < k; ++e) p[e] = (uint8_t)(u >> (8 * e));
}

// Four elements, two an instruction.  The compiler joins a packed product with the
// sum that follows it into one rounding; a product written as a * b + nz, nz a -0
// that it cannot see (an argument of the kernel), rounds as the product and stays
// apart.
__device__ __forceinline__ void mul4(float (&a)[4], const float (&b)[4], float nz) {
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const float2 r = ffma2(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]), make_float2(nz, nz));
    a[e] = r.x; a[e + 1] = r.y;
  }
}
__device__ __forceinline__ void mul4(float (&a)[4], float s, float nz) {
  const float b[4] = {s, s, s, s};
  mul4(a, b, nz);
}
__device__ __forceinline__ void add4(float (&a)[4], const float (&b)[4]) {
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const float2 r = fadd2(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
    a[e] = r.x; a[e + 1] = r.y;
  }
}
__device__ __forceinline__ void add4(float (&a)[4], float s) {
  const float b[4] = {s, s, s, s};
  add4(a, b);
}

// four e4m3 codes (lowest element in the low byte) and their values
__device__ __forceinline__ void codes_to_f(uint32_t u, float (&v)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw r =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> (16 * h)), __NV_E4M3);
    const float2 f = __half22float2(__half2(r));
    v[2 * h] = f.x;
    v[2 * h + 1] = f.y;
  }
}
__device__ __forceinline__ uint32_t f_to_codes(const float (&v)[4]) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
// The bits of the warp's largest magnitude: their order is that of non-negative
// floats with NaN above infinity, so a NaN is the largest.
__device__ __forceinline__ unsigned top_of(const float (&x)[4]) {
  float mine;
  asm("{\n\t.reg .f32 t;\n\t"
      "max.NaN.abs.f32 t, %1, %2, %3;\n\t"
      "max.NaN.f32 %0, t, %4;\n\t}"
      : "=f"(mine)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(fabsf(x[3])));
  return __reduce_max_sync(0xffffffffu, __float_as_uint(mine));
}
// Four values as codes of a block whose 448 / (largest magnitude) is inv.  ROOT: a
// positive one takes at least the smallest code, 2^-9.  (It is 2^-75 or more, so no
// block that is held as zeros has one.)
template <bool ROOT>
__device__ __forceinline__ uint32_t codes_of(const float (&x)[4], float inv) {
  float q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    q[e] = __fmul_rn(x[e], inv);
    if (ROOT && x[e] > 0.f) q[e] = fmaxf(q[e], 0.001953125f);
  }
  return f_to_codes(q);
}

struct Step {
  float lr, step_size, fix, gscale;
};

__device__ __forceinline__ float quick_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Where a lane's four elements of a group are (master, prep: or null), and the
// group's scales.
template <typename T>
struct Place {
  T* w;
  float *master, *m32, *v32;
  uint8_t *mq, *vq;
  float *ms, *vs;
  __half* prep;
  __device__ __forceinline__ Place(const Tensor& t, int64_t at)
      : w((T*)t.w + at), master(t.master ? t.master + at : nullptr), m32((float*)t.m + at),
        v32((float*)t.v + at), mq((uint8_t*)t.m + at), vq((uint8_t*)t.v + at), ms(t.ms + (at >> 7)),
        vs(t.vs + (at >> 7)), prep(t.prep ? t.prep + at : nullptr) {}
};

// One group of 128 elements, four a lane, that are in registers: the update, and
// what it writes at group o of the places.  k: how many of the lane's four there
// are (ALL: four).  mq, vq, sm, sv: the codes and scales of 8-bit states, whose
// values m and v then are to be.
template <typename T, int BITS, bool ALL>
__device__ __forceinline__ bool finish(const Args& a, const Place<T>& to, int o, const Step& s,
                                       float keep, int lane, int k, float (&g)[4], float (&p)[4],
                                       float (&m)[4], float (&v)[4], uint32_t mq, uint32_t vq,
                                       float sm, float sv) {
  const float nz = a.neg_zero;
  if constexpr (BITS == 8) {
    codes_to_f(mq, m);
    codes_to_f(vq, v);
    mul4(m, sm, nz);
    mul4(v, sv, nz);
    mul4(v, v, nz);
  }
  mul4(g, s.gscale, nz);
  float x[4], root[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = g[e];
  mul4(x, a.c1, nz);
  mul4(m, a.b1, nz);
  add4(m, x);
  mul4(g, g, nz);
  mul4(g, a.c2, nz);
  mul4(v, a.b2, nz);
  add4(v, g);
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = root[e] = __fsqrt_rn(v[e]);
  mul4(x, s.fix, nz);
  add4(x, a.eps);
  // With 8-bit states the quotient is the quick one, off by a few half spacings: it
  // enters w alone, and times lr is far below w's own spacing.  (Root and sums are
  // what the codes are made of and stay exact; quick ones gain nothing.)
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = BITS == 32 ? __fdiv_rn(m[e], x[e]) : m[e] * quick_rcp(x[e]);
  mul4(x, -s.step_size, nz);
  mul4(p, keep, nz);
  add4(p, x);
  if constexpr (BITS == 32) {
    store4<ALL>(to.m32 + o * 128, k, m);
    store4<ALL>(to.v32 + o * 128, k, v);
  } else {
    if constexpr (!ALL) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e >= k) m[e] = root[e] = 0.f;
    }
    // the two scales at once: even lanes for m, odd ones for the root
    const unsigned top_m = top_of(m), top_v = top_of(root);
    const float top = __uint_as_float(lane & 1 ? top_v : top_m);
    const bool live = !(top < kScaleFloor);
    const float inv = live ? __fmul_rn(448.f, __frcp_rn(top)) : 0.f;
    if (lane < 2) (lane ? to.vs : to.ms)[o] = live ? __fmul_rn(top, 1.f / 448.f) : 0.f;
    store_codes<ALL>(to.mq + o * 128, k, codes_of<false>(m, __shfl_sync(0xffffffffu, inv, 0)));
    store_codes<ALL>(to.vq + o * 128, k, codes_of<true>(root, __shfl_sync(0xffffffffu, inv, 1)));
  }
  bool bad = false;
  if (to.master) store4<ALL>(to.master + o * 128, k, p);
  if constexpr (sizeof(T) == 2) {
    if (to.prep) {
      // the operand copy is made of the rounded weight, like the one
      // tsp_block_weights_prepare makes
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[e] = to_f<T>(from_f<T>(p[e]));
        bad |= (ALL || e < k) && f16_bad(p[e]);
      }
      store4<ALL>(to.prep + o * 128, k, p);
    }
  }
  store4<ALL>(to.w + o * 128, k, p);
  return bad;
}

// One warp's 512 elements of a tensor from `first` on, in groups of 128, kBatch
// groups' loads ahead of their use.  ALL: none is past the end.  held: an error holds
// the update back; it is loaded next to the elements, not waited for before them.
constexpr int kGroups = 4, kBatch = 2;

template <typename T, int BITS, bool ALL>
__device__ __forceinline__ bool update(const Args& a, const Tensor& t, int64_t first, int lane,
                                       const Step& s, int held) {
  const float keep = __fsub_rn(1.f, __fmul_rn(s.lr, t.wd));
  const int64_t at = first + lane * 4;
  const float* gp = t.g + at;
  const Place<T> to(t, at);
  bool bad = false;
#pragma unroll
  for (int u0 = 0; u0 < kGroups; u0 += kBatch) {
    float g[kBatch][4], p[kBatch][4], m[kBatch][4], v[kBatch][4], sm[kBatch], sv[kBatch];
    uint32_t mq[kBatch], vq[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int o = u0 + u;
      const int k = ALL ? 4 : (int)max((int64_t)0, min((int64_t)4, t.n - at - o * 128));
      load4<ALL>(gp + o * 128, k, g[u]);
      if (to.master) load4<ALL>(to.master + o * 128, k, p[u]);
      else load4<ALL>(to.w + o * 128, k, p[u]);
      if constexpr (BITS == 32) {
        load4<ALL>(to.m32 + o * 128, k, m[u]);
        load4<ALL>(to.v32 + o * 128, k, v[u]);
      } else {
        mq[u] = load_codes<ALL>(to.mq + o * 128, k);
        vq[u] = load_codes<ALL>(to.vq + o * 128, k);
        const bool there = ALL || first + o * 128 < t.n;
        sm[u] = there ? to.ms[o] : 0.f;
        sv[u] = there ? to.vs[o] : 0.f;
      }
    }
    __syncwarp();   // every lane has read the old scales
    if (held) return false;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int o = u0 + u;
      if (!ALL && first + o * 128 >= t.n) break;
      const int k = ALL ? 4 : (int)max((int64_t)0, min((int64_t)4, t.n - at - o * 128));
      bad |= finish<T, BITS, ALL>(a, to, o, s, keep, lane, k, g[u], p[u], m[u], v[u], mq[u], vq[u],
                                  sm[u], sv[u]);
    }
  }
  return bad;
}

// The tensor of chunk ch, and where this warp's part of it starts.
__device__ __forceinline__ int find(const Args& a, int64_t ch, int warp, int64_t* first) {
  int lo = 0, hi = a.count - 1;   // the first tensor whose end is past ch
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.end[mid] > ch) hi = mid; else lo = mid + 1;
  }
  *first = (ch - (lo > 0 ? a.end[lo - 1] : 0)) * kChunk + warp * 512;
  return lo;
}

__device__ __forceinline__ Step step_of(const Args& a) {
  Step s = {a.lr, a.step_size, a.fix, a.gscale ? *a.gscale : 1.f};
  if (a.lr_dev || a.step_dev) {
    __shared__ Step shared;
    if (threadIdx.x == 0) {
      const double lr = a.lr_dev ? (double)*a.lr_dev : (double)a.lr;
      s.lr = (float)lr;
      if (a.step_dev) {
        const int64_t t = *a.step_dev;
        s.step_size = (float)(lr / (1.0 - power(a.dbeta1, t)));
        s.fix = (float)(1.0 / sqrt(1.0 - power(a.dbeta2, t)));
      } else {   // the host folded lr = 1 into step_size
        s.step_size = (float)(lr * (double)a.step_size);
      }
      shared = s;
    }
    __syncthreads();
    s = shared;
  }
  return s;
}

// 32-bit states: 28 to 32 bytes an element and little to compute; CTAs in order of
// the elements (a 7B-shaped block: 922 us, 962 with 8 CTAs a multiprocessor walking).
template <typename T, bool CLUSTER>   // the grid is one cluster
__global__ void __launch_bounds__(256, 3) adamw_kernel(const __grid_constant__ Args a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int held;
  if constexpr (CLUSTER) {
    held = held_in_cluster(a);
  } else {
    after_previous_kernel();
    held = *a.held;
  }
  const Step s = step_of(a);
  bool bad = false;
  const int64_t chunks = a.end[a.count - 1];
  for (int64_t ch = blockIdx.x; ch < chunks; ch += gridDim.x) {
    int64_t first;
    const Tensor& t = a.t[find(a, ch, warp, &first)];
    bad |= first + 512 <= t.n ? update<T, 32, true>(a, t, first, lane, s, held)
                              : update<T, 32, false>(a, t, first, lane, s, held);
  }
  if (bad) report_status(a.status, (int)TSP_ERR_RANGE);
}

// 8-bit states: a third fewer bytes and twice the instructions, so the loads have
// to go on while the warps compute.  Every lane copies what it will itself read to
// shared memory, the next chunk's group into the places of this one's as soon as
// that is in registers.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES)
                 : "memory");
}

struct Ahead {   // one warp's groups on their way
  float g[kGroups][128];
  float p[kGroups][128];
  uint32_t m[kGroups][32], v[kGroups][32];
};
constexpr int kAheadSmem = 8 * sizeof(Ahead);

template <typename T, int CTAS>   // CTAs a multiprocessor; 1: the grid is one cluster
__global__ void __launch_bounds__(256, CTAS) adamw_coded_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Ahead& in = reinterpret_cast<Ahead*>(smem)[warp];
  float *const in_g = in.g[0] + lane * 4, *const in_p = in.p[0] + lane * 4;
  uint32_t *const in_m = in.m[0] + lane, *const in_v = in.v[0] + lane;
  if (CTAS != 1) after_previous_kernel();
  // Loaded and tested in the way that costs least: for runs here, and as any value (593.9
  // us of a 7B-shaped block, 593.6 without; 598 in the other way); for single chunks
  // behind the first one's scales, with a vote (34.1 us of 3.1 M elements, 36 otherwise).
  int held = 0;
  if (CTAS == 1) held = held_in_cluster(a);
  if (CTAS == 2) held = *a.held;
  const Step s = step_of(a);
  bool bad = false;
  const int64_t begin = (int64_t)blockIdx.x * a.run, chunks = min(a.end[a.count - 1], begin + a.run);
  // the next chunk: its tensor, where this warp's part starts, whether all of its
  // 512 elements are there (they come ahead), its scales (lanes 0..3: of m, 4..7: of v)
  int next = 0;
  int64_t next_first = 0;
  bool whole = false;
  float scale = 0.f;
  const float *from_g = nullptr, *from_s = nullptr;
  const uint8_t *from_p = nullptr, *from_m = nullptr, *from_v = nullptr;
  bool wide = true;   // p is fp32
  // Long runs stay in a tensor for many chunks: the search is for its first alone (a
  // bf16 block without masters, 202 M elements: 448 us, 482 with a search a chunk).
  int64_t end_next = 0;
  auto look = [&](int64_t ch) {
    whole = false;
    if (ch >= chunks) return;
    if (CTAS == 2 && ch < end_next) {
      next_first += kChunk;
      whole = next_first + 512 <= a.t[next].n;
      if (!whole) return;
      from_s += kChunk / 128;
      if (lane < 8) scale = *from_s;
      from_g += kChunk;
      from_p += wide ? kChunk * 4 : kChunk * 2;
      from_m += kChunk;
      from_v += kChunk;
      return;
    }
    next = find(a, ch, warp, &next_first);
    const Tensor& t = a.t[next];
    if (CTAS == 2) end_next = a.end[next];
    whole = next_first + 512 <= t.n;
    if (!whole) return;
    const int64_t at = next_first + lane * 4;
    from_s = (lane < 4 ? t.ms : t.vs) + (next_first >> 7) + (lane & 3);
    if (lane < 8) scale = *from_s;
    wide = sizeof(T) == 4 || t.master;
    from_g = t.g + at;
    from_p = t.master ? (const uint8_t*)(t.master + at) : (const uint8_t*)((T*)t.w + at);
    from_m = (uint8_t*)t.m + at;
    from_v = (uint8_t*)t.v + at;
  };
  auto issue = [&](int u) {
    if (whole) {
      copy_async<16>(in_g + u * 128, from_g + u * 128);
      if (wide) copy_async<16>(in_p + u * 128, from_p + u * 512);
      else copy_async<8>(in_p + u * 128, from_p + u * 256);
      copy_async<4>(in_m + u * 32, from_m + u * 128);
      copy_async<4>(in_v + u * 32, from_v + u * 128);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  look(begin);
  if (CTAS == 3) held = *a.held;
#pragma unroll
  for (int u = 0; u < kGroups; ++u) issue(u);
  if (CTAS != 3 ? held != 0 : __any_sync(0xffffffffu, held)) {   // the copies have to arrive before their places go
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  for (int64_t ch = begin; ch < chunks; ++ch) {
    const Tensor& t = a.t[next];
    const int64_t first = next_first;
    const bool ahead = whole, fp32 = wide;
    const float old = scale;
    look(ch + 1);
    if (!ahead) {
      bad |= update<T, 8, false>(a, t, first, lane, s, 0);
#pragma unroll
      for (int u = 0; u < kGroups; ++u) issue(u);
      continue;
    }
    const float keep = __fsub_rn(1.f, __fmul_rn(s.lr, t.wd));
    const Place<T> to(t, first + lane * 4);
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kGroups - 1) : "memory");
      float g[4], p[4], m[4], v[4];
      load4<true>(in_g + u * 128, 4, g);
      if (fp32) load4<true>(in_p + u * 128, 4, p);
      else load4<true>((const T*)(in_p + u * 128), 4, p);
      const uint32_t mq = in_m[u * 32], vq = in_v[u * 32];
      const float sm = __shfl_sync(0xffffffffu, old, u), sv = __shfl_sync(0xffffffffu, old, 4 + u);
      __syncwarp();   // read, before the copies into the same places
      issue(u);
      bad |= finish<T, 8, true>(a, to, u, s, keep, lane, 4, g, p, m, v, mq, vq, sm, sv);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (bad) report_status(a.status, (int)TSP_ERR_RANGE);
}

// A launch of 256 threads a CTA: an ordinary one, behind adamw_held_kernel (see
// launch_after, which would copy the arguments' 11 KB), or of one cluster.
enum class How { ordinary, dependent, cluster };
tsp_status launch(void (*kernel)(Args), unsigned grid, size_t smem, How how, cudaStream_t st, Args& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  if (how == How::cluster) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = grid;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  } else {
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = how == How::ordinary ? 0 : 1;
  void* args[] = {&a};
  TSP_CUDA_TRY(cudaLaunchKernelExC(&cfg, (const void*)kernel, args));
  return TSP_OK;
}

// The whole grid as one cluster, of up to 16 CTAs (more than 8 have to be allowed).
template <auto KERNEL>
tsp_status launch_cluster(unsigned grid, size_t smem, cudaStream_t st, Args& a) {
  static std::atomic<bool> allowed[kMaxDevices];
  const int dev = current_device();
  if (!allowed[dev]) {
    TSP_CUDA_TRY(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    allowed[dev] = true;
  }
  return launch(KERNEL, grid, smem, How::cluster, st, a);
}

}  // namespace

tsp_status launch_adamw(const tsp_adamw_tensor* ts, int count, const tsp_adamw_hyper* h,
                        int state_bits, int dtype, cudaStream_t st) {
  Args a;
  a.b1 = (float)h->beta1;
  a.c1 = (float)(1.0 - h->beta1);
  a.b2 = (float)h->beta2;
  a.c2 = (float)(1.0 - h->beta2);
  a.eps = (float)h->eps;
  a.neg_zero = -0.f;
  a.lr = (float)h->lr;
  a.dbeta1 = h->beta1;
  a.dbeta2 = h->beta2;
  a.lr_dev = h->lr_dev;
  a.step_dev = h->step_dev;
  a.gscale = h->gscale_dev;
  a.status = status_word();
  a.held = nullptr;
  a.step_size = a.fix = 0.f;
  if (!h->step_dev) {
    a.step_size = (float)((h->lr_dev ? 1.0 : h->lr) / (1.0 - std::pow(h->beta1, (double)h->step)));
    a.fix = (float)(1.0 / std::sqrt(1.0 - std::pow(h->beta2, (double)h->step)));
  }
  int at = 0;
  while (at < count) {
    int64_t chunks = 0;
    a.count = 0;
    for (; at < count && a.count < kTensors; ++at) {
      const tsp_adamw_tensor& s = ts[at];
      if (s.n == 0) continue;
      a.t[a.count] = {s.n, s.w, s.master, s.g, s.m, s.v, s.m_scale, s.v_scale, (__half*)s.prep,
                      s.weight_decay};
      chunks += (s.n + kChunk - 1) / kChunk;
      a.end[a.count++] = chunks;
    }
    if (a.count == 0) break;
    const bool first = !a.held;
    const bool bf = dtype == TSP_BF16;
    if (first && chunks <= kClusterChunks) {   // (so few hold all of the call's tensors)
      if (!a.status) return TSP_ERR_CUDA;
      unsigned grid = 1;
      while (grid < chunks) grid *= 2;
      a.run = 1;
      Prof prof("adamw", st);
      if (state_bits == 8)
        return bf ? launch_cluster<adamw_coded_kernel<__nv_bfloat16, 1>>(grid, kAheadSmem, st, a)
                  : launch_cluster<adamw_coded_kernel<float, 1>>(grid, kAheadSmem, st, a);
      return bf ? launch_cluster<adamw_kernel<__nv_bfloat16, true>>(grid, 0, st, a)
                : launch_cluster<adamw_kernel<float, true>>(grid, 0, st, a);
    }
    tsp_status r = TSP_OK;
    if (first) r = take_held(a.status, st, &a.held);   // (all of the call's launches use it)
    if (r != TSP_OK) return r;
    const How how = first ? How::dependent : How::ordinary;
    Prof prof("adamw", st);
    if (state_bits == 8) {
      // Runs of several chunks to copy ahead in, in order, so that what is written at a
      // time lies together (a 7B-shaped block: 594 us, with resident CTAs walking all
      // chunks 738).  With masters (20 bytes an element) memory is the bound: runs of 4
      // (8: 600 us), shorter ones where that leaves less than three for every resident
      // CTA (12.8 M elements: 46 us in twos, 50 in single chunks).  Without (12 to 16
      // bytes) the warps' instructions are: runs of 8 (180 M bf16 elements: 404 us, 424
      // with 4), six for every resident CTA (10.4 M: 35 us, 40 with three).  Runs take two CTAs a multiprocessor and no spills (a
      // 7B-shaped block: 602 us against 631 with three), single chunks three (10.4 M
      // elements: 36 us against 43 with two).
      const bool masters = a.t[0].master != nullptr;
      a.run = (int)std::max<int64_t>(
          1, std::min<int64_t>(masters ? 4 : 8, chunks / ((int64_t)num_sms() * (masters ? 6 : 12))));
      const unsigned grid = (unsigned)((chunks + a.run - 1) / a.run);
      if (a.run >= 2)
        r = launch(bf ? adamw_coded_kernel<__nv_bfloat16, 2> : adamw_coded_kernel<float, 2>, grid,
                   kAheadSmem, how, st, a);
      else
        r = launch(bf ? adamw_coded_kernel<__nv_bfloat16, 3> : adamw_coded_kernel<float, 3>, grid,
                   kAheadSmem, how, st, a);
    } else {
      const unsigned grid = (unsigned)std::min<int64_t>(chunks, (int64_t)num_sms() * 256);
      r = launch(bf ? adamw_kernel<__nv_bfloat16, false> : adamw_kernel<float, false>, grid, 0, how, st, a);
    }
    if (r != TSP_OK) return r;
  }
  return TSP_OK;
}

}  // namespace tsp
