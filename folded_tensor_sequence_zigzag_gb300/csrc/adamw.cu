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
  float eps;
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

template <typename T>
__device__ __forceinline__ void load4(const T* p, int64_t i, int k, float (&v)[4]) {
  if (k == 4) {
    if constexpr (sizeof(T) == 4) {
      const float4 f = *reinterpret_cast<const float4*>(p + i);
      v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(p + i);
      v[0] = lo2<T>(u.x); v[1] = hi2<T>(u.x); v[2] = lo2<T>(u.y); v[3] = hi2<T>(u.y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = e < k ? to_f<T>(p[i + e]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, int64_t i, int k, const float (&v)[4]) {
  if (k == 4) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(p + i) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < k) p[i + e] = from_f<T>(v[e]);
  }
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
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t i, int k) {
  if (k == 4) return *reinterpret_cast<const uint32_t*>(p + i);
  uint32_t u = 0;
  for (int e = 0; e < k; ++e) u |= (uint32_t)p[i + e] << (8 * e);
  return u;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int k, uint32_t u) {
  if (k == 4) {
    *reinterpret_cast<uint32_t*>(p + i) = u;
    return;
  }
  for (int e = 0; e < k; ++e) p[i + e] = (uint8_t)(u >> (8 * e));
}
// the larger of a and b; a NaN wins, so that it reaches the block's scale
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The warp's 128 values as codes and a scale (written by lane 0).
template <bool ROOT>
__device__ __forceinline__ uint32_t quantise(const float (&x)[4], float* scale, int lane) {
  float top = max_nan(max_nan(fabsf(x[0]), fabsf(x[1])), max_nan(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
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

template <typename T, int BITS>
__global__ void __launch_bounds__(256) adamw_kernel(const __grid_constant__ Args a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float lr = a.lr, step_size = a.step_size, fix = a.fix;
  if (a.lr_dev || a.step_dev) {
    __shared__ float sh[3];
    if (threadIdx.x == 0) {
      const double l = a.lr_dev ? (double)*a.lr_dev : (double)a.lr;
      sh[0] = (float)l;
      if (a.step_dev) {
        const int64_t t = *a.step_dev;
        sh[1] = (float)(l / (1.0 - power(a.dbeta1, t)));
        sh[2] = (float)(1.0 / sqrt(1.0 - power(a.dbeta2, t)));
      } else {   // the host folded lr = 1 into step_size
        sh[1] = (float)(l * (double)a.step_size);
        sh[2] = a.fix;
      }
    }
    __syncthreads();
    lr = sh[0];
    step_size = sh[1];
    fix = sh[2];
  }
  const float gs = a.gscale ? *a.gscale : 1.f;
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
    const float keep = __fsub_rn(1.f, __fmul_rn(lr, t.wd));
    T* w = (T*)t.w;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t b0 = first + u * 128;
      if (b0 >= t.n) break;
      const int64_t i = b0 + lane * 4;
      const int k = (int)max((int64_t)0, min((int64_t)4, t.n - i));
      float g[4], m[4], v[4], p[4];
      load4<float>(t.g, i, k, g);
      if (t.master) load4<float>(t.master, i, k, p);
      else load4<T>(w, i, k, p);
      if constexpr (BITS == 32) {
        load4<float>((const float*)t.m, i, k, m);
        load4<float>((const float*)t.v, i, k, v);
      } else {
        codes_to_f(load_codes((const uint8_t*)t.m, i, k), m);
        codes_to_f(load_codes((const uint8_t*)t.v, i, k), v);
        const float sm = t.ms[b0 >> 7], sv = t.vs[b0 >> 7];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          m[e] = __fmul_rn(m[e], sm);
          v[e] = __fmul_rn(v[e], sv);
          v[e] = __fmul_rn(v[e], v[e]);
        }
      }
      float root[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[e] = __fmul_rn(g[e], gs);
        m[e] = __fadd_rn(__fmul_rn(m[e], a.b1), __fmul_rn(g[e], a.c1));
        v[e] = __fadd_rn(__fmul_rn(v[e], a.b2), __fmul_rn(__fmul_rn(g[e], g[e]), a.c2));
        root[e] = __fsqrt_rn(v[e]);
        const float q = __fdiv_rn(m[e], __fadd_rn(__fmul_rn(root[e], fix), a.eps));
        p[e] = __fsub_rn(__fmul_rn(p[e], keep), __fmul_rn(step_size, q));
      }
      if constexpr (BITS == 32) {
        store4<float>((float*)t.m, i, k, m);
        store4<float>((float*)t.v, i, k, v);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e >= k) m[e] = root[e] = 0.f;
        __syncwarp();   // every lane has read the old scales
        store_codes((uint8_t*)t.m, i, k, quantise<false>(m, t.ms + (b0 >> 7), lane));
        store_codes((uint8_t*)t.v, i, k, quantise<true>(root, t.vs + (b0 >> 7), lane));
      }
      if (t.master) store4<float>(t.master, i, k, p);
      if constexpr (sizeof(T) == 2) {
        // the operand copy is made of the rounded weight, like the one
        // tsp_block_weights_prepare makes
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = to_f<T>(from_f<T>(p[e]));
        if (t.prep) {
#pragma unroll
          for (int e = 0; e < 4; ++e) bad |= e < k && f16_bad(p[e]);
          store4<__half>(t.prep, i, k, p);
        }
      }
      store4<T>(w, i, k, p);
    }
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
