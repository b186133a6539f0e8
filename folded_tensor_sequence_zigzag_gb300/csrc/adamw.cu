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
#include <cuda_fp8.h>

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
  float b1, c1, b2, c2;    // beta, 1 - beta
  float eps, neg_zero;
  float lr, step_size, fix;   // lr, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  double dbeta1, dbeta2;
  const float* lr_dev;
  const int64_t* step_dev;
  const float* gscale;
  int* status;
};

// x^n by squaring, n >= 1
__device__ double power(double x, int64_t n) {
  double r = 1.0;
  for (; n > 0; n >>= 1, x *= x)
    if (n & 1) r *= x;
  return r;
}

// The k (of four) elements at p; ALL: all four, one access.
template <bool ALL, typename T>
__device__ __forceinline__ void load4(const T* p, int k, float (&v)[4]) {
  if constexpr (!ALL) {
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
  if constexpr (!ALL) {
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
  if constexpr (ALL) return *reinterpret_cast<const uint32_t*>(p);
  uint32_t u = 0;
  for (int e = 0; e < k; ++e) u |= (uint32_t)p[e] << (8 * e);
  return u;
}
template <bool ALL>
__device__ __forceinline__ void store_codes(uint8_t* p, int k, uint32_t u) {
  if constexpr (ALL) {
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
// The warp's 128 values as codes and a scale (written by lane 0).  The largest
// magnitude is found on the bits, whose order is that of non-negative floats with
// NaN above infinity: one instruction for the warp, and a NaN reaches the scale.
template <bool ROOT>
__device__ __forceinline__ uint32_t quantise(const float (&x)[4], float* scale, int lane) {
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) bits = max(bits, __float_as_uint(x[e]) & 0x7fffffffu);
  const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, bits));
  const bool live = !(top < kScaleFloor);
  const float inv = live ? __fmul_rn(448.f, __frcp_rn(top)) : 0.f;
  if (lane == 0) *scale = live ? __fmul_rn(top, 1.f / 448.f) : 0.f;
  float q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    q[e] = __fmul_rn(x[e], inv);
    // below half of the smallest code the rounding would give 0 (the tie too)
    if (ROOT && live && x[e] > 0.f && q[e] <= 0.0009765625f) q[e] = 0.001953125f;
  }
  return f_to_codes(q);
}

struct Step {
  float lr, step_size, fix, gscale;
};

// One warp's 512 elements of a tensor from `first` on, in groups of 128 (four a
// lane), kBatch groups' loads ahead of their use.  ALL: none is past the end.
constexpr int kGroups = 4, kBatch = 2;

template <typename T, int BITS, bool ALL>
__device__ __forceinline__ bool update(const Args& a, const Tensor& t, int64_t first, int lane,
                                       const Step& s) {
  const float nz = a.neg_zero;
  const float keep = __fsub_rn(1.f, __fmul_rn(s.lr, t.wd));
  const int64_t at = first + lane * 4;
  const float* gp = t.g + at;
  T* wp = (T*)t.w + at;
  float* pp = t.master ? t.master + at : nullptr;
  __half* hp = t.prep ? t.prep + at : nullptr;
  float *m32 = (float*)t.m + at, *v32 = (float*)t.v + at;
  uint8_t *mc = (uint8_t*)t.m + at, *vc = (uint8_t*)t.v + at;
  float *ms = t.ms + (first >> 7), *vs = t.vs + (first >> 7);
  bool bad = false;
#pragma unroll
  for (int u0 = 0; u0 < kGroups; u0 += kBatch) {
    float g[kBatch][4], p[kBatch][4], m[kBatch][4], v[kBatch][4], sm[kBatch], sv[kBatch];
    uint32_t mq[kBatch], vq[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int o = (u0 + u) * 128;
      const int k = ALL ? 4 : (int)max((int64_t)0, min((int64_t)4, t.n - at - o));
      load4<ALL>(gp + o, k, g[u]);
      if (pp) load4<ALL>(pp + o, k, p[u]);
      else load4<ALL>(wp + o, k, p[u]);
      if constexpr (BITS == 32) {
        load4<ALL>(m32 + o, k, m[u]);
        load4<ALL>(v32 + o, k, v[u]);
      } else {
        mq[u] = load_codes<ALL>(mc + o, k);
        vq[u] = load_codes<ALL>(vc + o, k);
        const bool there = ALL || first + o < t.n;
        sm[u] = there ? ms[u0 + u] : 0.f;
        sv[u] = there ? vs[u0 + u] : 0.f;
      }
    }
    __syncwarp();   // every lane has read the old scales
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int o = (u0 + u) * 128;
      if (!ALL && first + o >= t.n) break;
      const int k = ALL ? 4 : (int)max((int64_t)0, min((int64_t)4, t.n - at - o));
      if constexpr (BITS == 8) {
        codes_to_f(mq[u], m[u]);
        codes_to_f(vq[u], v[u]);
        mul4(m[u], sm[u], nz);
        mul4(v[u], sv[u], nz);
        mul4(v[u], v[u], nz);
      }
      mul4(g[u], s.gscale, nz);
      float x[4], root[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = g[u][e];
      mul4(x, a.c1, nz);
      mul4(m[u], a.b1, nz);
      add4(m[u], x);
      mul4(g[u], g[u], nz);
      mul4(g[u], a.c2, nz);
      mul4(v[u], a.b2, nz);
      add4(v[u], g[u]);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = root[e] = __fsqrt_rn(v[u][e]);
      mul4(x, s.fix, nz);
      add4(x, a.eps);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = __fdiv_rn(m[u][e], x[e]);
      mul4(x, -s.step_size, nz);
      mul4(p[u], keep, nz);
      add4(p[u], x);
      if constexpr (BITS == 32) {
        store4<ALL>(m32 + o, k, m[u]);
        store4<ALL>(v32 + o, k, v[u]);
      } else {
        if constexpr (!ALL) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e >= k) m[u][e] = root[e] = 0.f;
        }
        store_codes<ALL>(mc + o, k, quantise<false>(m[u], ms + u0 + u, lane));
        store_codes<ALL>(vc + o, k, quantise<true>(root, vs + u0 + u, lane));
      }
      if (pp) store4<ALL>(pp + o, k, p[u]);
      if constexpr (sizeof(T) == 2) {
        if (hp) {
          // the operand copy is made of the rounded weight, like the one
          // tsp_block_weights_prepare makes
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[u][e] = to_f<T>(from_f<T>(p[u][e]));
            bad |= (ALL || e < k) && f16_bad(p[u][e]);
          }
          store4<ALL>(hp + o, k, p[u]);
        }
      }
      store4<ALL>(wp + o, k, p[u]);
    }
  }
  return bad;
}

template <typename T, int BITS>
__global__ void __launch_bounds__(256, BITS == 8 ? 4 : 3) adamw_kernel(const __grid_constant__ Args a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
  bool bad = false;
  const int64_t chunks = a.end[a.count - 1];
  for (int64_t ch = blockIdx.x; ch < chunks; ch += gridDim.x) {
    int lo = 0, hi = a.count - 1;   // the first tensor whose end is past ch
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.end[mid] > ch) hi = mid; else lo = mid + 1;
    }
    const Tensor& t = a.t[lo];
    const int64_t first = (ch - (lo > 0 ? a.end[lo - 1] : 0)) * kChunk + warp * 512;
    bad |= first + 512 <= t.n ? update<T, BITS, true>(a, t, first, lane, s)
                              : update<T, BITS, false>(a, t, first, lane, s);
  }
  if (bad) report_status(a.status, (int)TSP_ERR_RANGE);
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
    const int grid = (int)std::min<int64_t>(chunks, (int64_t)num_sms() * 8);
    Prof prof("adamw", st);
    if (dtype == TSP_BF16) {
      if (state_bits == 8) adamw_kernel<__nv_bfloat16, 8><<<grid, 256, 0, st>>>(a);
      else adamw_kernel<__nv_bfloat16, 32><<<grid, 256, 0, st>>>(a);
    } else {
      if (state_bits == 8) adamw_kernel<float, 8><<<grid, 256, 0, st>>>(a);
      else adamw_kernel<float, 32><<<grid, 256, 0, st>>>(a);
    }
    TSP_CUDA_TRY(cudaGetLastError());
  }
  return TSP_OK;
}

}  // namespace tsp
