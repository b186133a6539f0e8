// norm_residual.cu -- the step between two sub-layers in one pass over the row:
//
//   u = f * rstd_f * g_post,  rstd_f = 1 / sqrt(mean(f^2) + eps)     (u = f without g_post)
//   h = x + s * sigmoid(z) * u                                        (sigmoid(z) = 1 without z)
//   b = h * rstd_h * g_pre,   rstd_h = 1 / sqrt(mean(h^2) + eps)     (none without g_pre)
//
// and its backward: with dh, db the gradients that reach h and b,
//
//   dx = dh + rstd_h (db g_pre - n_h mean(db g_pre n_h)),   n_h = h rstd_h
//   dz = s dx u sigmoid(z) (1 - sigmoid(z)),   du = s sigmoid(z) dx
//   df = rstd_f (du g_post - n_f mean(du g_post n_f)),      n_f = f rstd_f
//   dg_pre = sum over rows of db n_h,   dg_post = sum over rows of du n_f.
//
// Sums and statistics are fp32.  rstd_h is the norm of h as it is stored, so b
// is what tsp_rmsnorm_fwd gives for the h the caller sees, and the backward,
// which reads that h, differentiates the same function.
#include "common.cuh"
#include "kernels.h"

namespace tsp {

namespace {

// N consecutive elements (N = 8: 16-byte accesses; N = 1: any alignment).
template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float (&v)[N]) {
  if constexpr (N == 1) {
    v[0] = to_f<T>(*p);
  } else if constexpr (sizeof(T) == 2) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = lo2<T>(w[i]);
      v[2 * i + 1] = hi2<T>(w[i]);
    }
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0];
    const float4 b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float (&v)[N]) {
  if constexpr (N == 1) {
    *p = from_f<T>(v[0]);
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]),
                                              pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// sigmoid and its derivative from e = exp(-|z|), which neither overflows nor
// cancels: sigmoid(|z|) = 1 / (1 + e), sigmoid(-|z|) = e / (1 + e).
__device__ __forceinline__ float gate_of(float z) {
  const float e = expf(-fabsf(z)), r = 1.f / (1.f + e);
  return z >= 0.f ? r : (z < 0.f ? e * r : z);   // a NaN stays one
}
__device__ __forceinline__ float gate_slope(float z) {
  const float e = expf(-fabsf(z)), r = 1.f / (1.f + e);
  return e * r * r;
}

// Sum over the CTA, the same in every thread; `part` holds one value a warp
// and is reused by the next call only after another barrier.
__device__ __forceinline__ float cta_sum(float v, float* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  v = warp_sum(v);
  if (nw == 1) return v;
  if (lane == 0) part[warp] = v;
  __syncthreads();
  return warp_sum(lane < nw ? part[lane] : 0.f);
}

struct FwdArgs {
  const void *f, *x, *z, *g_post, *g_pre;
  void *h, *b;
  float *rstd_f, *rstd_h;
  int64_t rows;
  int n;
  float s, eps;
};

// A CTA a row (grid-stride), the row in registers: UPT units of N elements a
// thread, unit i of thread t at (i * blockDim + t) * N.
template <typename T, typename Ts, int N, int UPT>
__global__ void __launch_bounds__(1024) norm_residual_fwd_kernel(const __grid_constant__ FwdArgs a) {
  __shared__ float part[2][32];
  const int n = a.n, t = threadIdx.x;
  const float inv_n = 1.f / (float)n;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t base = row * n;
    float v[UPT][N];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int c = (i * blockDim.x + t) * N;
      if (c < n) {
        load_n<T, N>((const T*)a.f + base + c, v[i]);
#pragma unroll
        for (int e = 0; e < N; ++e) ss = fmaf(v[i][e], v[i][e], ss);
      }
    }
    float r = 1.f;
    if (a.g_post) {
      r = rsqrtf(cta_sum(ss, part[0]) * inv_n + a.eps);
      if (t == 0 && a.rstd_f) a.rstd_f[row] = r;
    }
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int c = (i * blockDim.x + t) * N;
      if (c < n) {
        float q[N];
        if (a.g_post) {
          load_n<T, N>((const T*)a.g_post + c, q);
#pragma unroll
          for (int e = 0; e < N; ++e) v[i][e] *= r * q[e];
        }
        if (a.z) {
          load_n<T, N>((const T*)a.z + base + c, q);
#pragma unroll
          for (int e = 0; e < N; ++e) v[i][e] *= gate_of(q[e]);
        }
        load_n<Ts, N>((const Ts*)a.x + base + c, q);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          v[i][e] = to_f<Ts>(from_f<Ts>(fmaf(a.s, v[i][e], q[e])));
          ss = fmaf(v[i][e], v[i][e], ss);
        }
        store_n<Ts, N>((Ts*)a.h + base + c, v[i]);
      }
    }
    if (a.g_pre) {
      r = rsqrtf(cta_sum(ss, part[1]) * inv_n + a.eps);
      if (t == 0 && a.rstd_h) a.rstd_h[row] = r;
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int c = (i * blockDim.x + t) * N;
        if (c < n) {
          float q[N];
          load_n<T, N>((const T*)a.g_pre + c, q);
#pragma unroll
          for (int e = 0; e < N; ++e) q[e] *= v[i][e] * r;
          store_n<T, N>((T*)a.b + base + c, q);
        }
      }
    }
    if (!(a.g_post && a.g_pre)) __syncthreads();   // one barrier a row would let `part` be reused early
  }
}

// Rows wider than the registers hold: the row is read again for each step
// (from L2), and h is read back by the thread that wrote it.
template <typename T, typename Ts>
__global__ void __launch_bounds__(1024) norm_residual_fwd_wide_kernel(const __grid_constant__ FwdArgs a) {
  __shared__ float part[2][32];
  const int n = a.n;
  const float inv_n = 1.f / (float)n;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* f = (const T*)a.f + row * n;
    const T* z = a.z ? (const T*)a.z + row * n : nullptr;
    const Ts* x = (const Ts*)a.x + row * n;
    Ts* h = (Ts*)a.h + row * n;
    float r = 1.f, ss = 0.f;
    if (a.g_post) {
      for (int c = threadIdx.x; c < n; c += blockDim.x) ss = fmaf(to_f<T>(f[c]), to_f<T>(f[c]), ss);
      r = rsqrtf(cta_sum(ss, part[0]) * inv_n + a.eps);
      if (threadIdx.x == 0 && a.rstd_f) a.rstd_f[row] = r;
    }
    ss = 0.f;
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
      float u = to_f<T>(f[c]);
      if (a.g_post) u *= r * to_f<T>(((const T*)a.g_post)[c]);
      if (z) u *= gate_of(to_f<T>(z[c]));
      const Ts o = from_f<Ts>(fmaf(a.s, u, to_f<Ts>(x[c])));
      h[c] = o;
      ss = fmaf(to_f<Ts>(o), to_f<Ts>(o), ss);
    }
    if (a.g_pre) {
      r = rsqrtf(cta_sum(ss, part[1]) * inv_n + a.eps);
      if (threadIdx.x == 0 && a.rstd_h) a.rstd_h[row] = r;
      for (int c = threadIdx.x; c < n; c += blockDim.x)
        ((T*)a.b)[row * n + c] = from_f<T>(to_f<Ts>(h[c]) * r * to_f<T>(((const T*)a.g_pre)[c]));
    }
    __syncthreads();
  }
}

struct BwdArgs {
  const float *dh, *db;
  const void *f, *z, *h, *g_post, *g_pre;
  const float *rstd_f, *rstd_h;
  float* dx;
  void *df, *dz;
  float *part_post, *part_pre;   // [gridDim][n]
  int64_t rows;
  int n;
  float s;
};

// The same layout; a thread's columns are the same in every row, so its share
// of the gain gradients stays in registers until the CTA's last row.
template <typename T, typename Ts, int N, int UPT>
__global__ void __launch_bounds__(UPT * N > 8 ? 512 : 1024) norm_residual_bwd_kernel(const __grid_constant__ BwdArgs a) {
  __shared__ float part[2][32];
  const int n = a.n, t = threadIdx.x;
  const float inv_n = 1.f / (float)n;
  float dpost[UPT][N], dpre[UPT][N];
#pragma unroll
  for (int i = 0; i < UPT; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) dpost[i][e] = dpre[i][e] = 0.f;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t base = row * n;
    float d[UPT][N], q[N];
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int c = (i * blockDim.x + t) * N;
#pragma unroll
      for (int e = 0; e < N; ++e) d[i][e] = 0.f;
      if (c < n && a.dh) load_n<float, N>(a.dh + base + c, d[i]);
    }
    if (a.g_pre) {
      const float r = a.rstd_h[row];
      float y[UPT][N], gd[UPT][N], dot = 0.f;
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int c = (i * blockDim.x + t) * N;
        if (c < n) {
          load_n<Ts, N>((const Ts*)a.h + base + c, y[i]);
          load_n<float, N>(a.db + base + c, gd[i]);
          load_n<T, N>((const T*)a.g_pre + c, q);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            y[i][e] *= r;
            dpre[i][e] = fmaf(gd[i][e], y[i][e], dpre[i][e]);
            gd[i][e] *= q[e];
            dot = fmaf(gd[i][e], y[i][e], dot);
          }
        }
      }
      dot = cta_sum(dot, part[0]) * inv_n;
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int c = (i * blockDim.x + t) * N;
        if (c < n) {
#pragma unroll
          for (int e = 0; e < N; ++e) d[i][e] = fmaf(r, gd[i][e] - y[i][e] * dot, d[i][e]);
        }
      }
    }
    const float rf = a.g_post ? a.rstd_f[row] : 1.f;
    float y[UPT][N], dot = 0.f;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int c = (i * blockDim.x + t) * N;
      if (c < n) {
        store_n<float, N>(a.dx + base + c, d[i]);
        load_n<T, N>((const T*)a.f + base + c, y[i]);
        float g[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          y[i][e] *= rf;
          d[i][e] *= a.s;
          g[e] = 1.f;
        }
        if (a.g_post) load_n<T, N>((const T*)a.g_post + c, g);
        if (a.z) {
          float dz[N];
          load_n<T, N>((const T*)a.z + base + c, q);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            dz[e] = d[i][e] * (y[i][e] * g[e]) * gate_slope(q[e]);
            d[i][e] *= gate_of(q[e]);
          }
          store_n<T, N>((T*)a.dz + base + c, dz);
        }
        if (a.g_post) {
#pragma unroll
          for (int e = 0; e < N; ++e) {
            dpost[i][e] = fmaf(d[i][e], y[i][e], dpost[i][e]);
            d[i][e] *= g[e];
            dot = fmaf(d[i][e], y[i][e], dot);
          }
        }
      }
    }
    if (a.g_post) dot = cta_sum(dot, part[1]) * inv_n;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int c = (i * blockDim.x + t) * N;
      if (c < n) {
        if (a.g_post) {
#pragma unroll
          for (int e = 0; e < N; ++e) d[i][e] = rf * (d[i][e] - y[i][e] * dot);
        }
        store_n<T, N>((T*)a.df + base + c, d[i]);
      }
    }
    if (!(a.g_post && a.g_pre)) __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    const int c = (i * blockDim.x + t) * N;
    if (c < n) {
      if (a.g_post) store_n<float, N>(a.part_post + (int64_t)blockIdx.x * n + c, dpost[i]);
      if (a.g_pre) store_n<float, N>(a.part_pre + (int64_t)blockIdx.x * n + c, dpre[i]);
    }
  }
}

// Wide rows: the row is read again for each step; the gain gradients of a CTA
// are summed in its own rows of the partials, by the thread that owns the column.
template <typename T, typename Ts>
__global__ void __launch_bounds__(1024) norm_residual_bwd_wide_kernel(const __grid_constant__ BwdArgs a) {
  __shared__ float part[2][32];
  const int n = a.n;
  const float inv_n = 1.f / (float)n;
  float* ppost = a.g_post ? a.part_post + (int64_t)blockIdx.x * n : nullptr;
  float* ppre = a.g_pre ? a.part_pre + (int64_t)blockIdx.x * n : nullptr;
  for (int c = threadIdx.x; c < n; c += blockDim.x) {
    if (ppost) ppost[c] = 0.f;
    if (ppre) ppre[c] = 0.f;
  }
  const T* gpost = (const T*)a.g_post;
  const T* gpre = (const T*)a.g_pre;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t base = row * n;
    float r = 0.f, dot = 0.f;
    if (gpre) {
      r = a.rstd_h[row];
      for (int c = threadIdx.x; c < n; c += blockDim.x) {
        const float y = to_f<Ts>(((const Ts*)a.h)[base + c]) * r, d = a.db[base + c];
        ppre[c] = fmaf(d, y, ppre[c]);
        dot = fmaf(d * to_f<T>(gpre[c]), y, dot);
      }
      dot = cta_sum(dot, part[0]) * inv_n;
    }
    const float rf = gpost ? a.rstd_f[row] : 1.f;
    float dot2 = 0.f;
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
      float d = a.dh ? a.dh[base + c] : 0.f;
      if (gpre) {
        const float y = to_f<Ts>(((const Ts*)a.h)[base + c]) * r;
        d = fmaf(r, a.db[base + c] * to_f<T>(gpre[c]) - y * dot, d);
      }
      a.dx[base + c] = d;
      d *= a.s;
      const float y = to_f<T>(((const T*)a.f)[base + c]) * rf;
      const float g = gpost ? to_f<T>(gpost[c]) : 1.f;
      if (a.z) {
        const float z = to_f<T>(((const T*)a.z)[base + c]);
        ((T*)a.dz)[base + c] = from_f<T>(d * (y * g) * gate_slope(z));
        d *= gate_of(z);
      }
      if (gpost) {
        ppost[c] = fmaf(d, y, ppost[c]);
        dot2 = fmaf(d * g, y, dot2);
      } else {
        ((T*)a.df)[base + c] = from_f<T>(d);
      }
    }
    if (gpost) {
      dot2 = cta_sum(dot2, part[1]) * inv_n;
      for (int c = threadIdx.x; c < n; c += blockDim.x) {
        float d = a.dx[base + c] * a.s;
        if (a.z) d *= gate_of(to_f<T>(((const T*)a.z)[base + c]));
        const float y = to_f<T>(((const T*)a.f)[base + c]) * rf;
        ((T*)a.df)[base + c] = from_f<T>(rf * (d * to_f<T>(gpost[c]) - y * dot2));
      }
    }
    __syncthreads();
  }
}

// dg[i] = the column sums of the CTAs' partials, in a fixed order; blockIdx.y
// picks the gain.
__global__ void __launch_bounds__(256) norm_residual_gain_kernel(const float* __restrict__ p0,
                                                                 float* __restrict__ o0,
                                                                 const float* __restrict__ p1,
                                                                 float* __restrict__ o1, int nb,
                                                                 int n) {
  __shared__ float acc[8][33];
  const float* part = blockIdx.y ? p1 : p0;
  float* out = blockIdx.y ? o1 : o0;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + tx;
  float s = 0.f;
  if (i < n)
    for (int b = ty; b < nb; b += 8) s += part[(int64_t)b * n + i];
  acc[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && i < n) {
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) o += acc[w][tx];
    out[i] = o;
  }
}

// Units a thread and threads a CTA for rows of n elements; upt == 0: wide.
struct Shape {
  int N, upt, threads;
};
Shape shape_of(int n, int max_threads) {
  Shape s;
  s.N = n % 8 == 0 ? 8 : 1;
  const int units = n / s.N;
  s.upt = s.N == 8 ? 2 : 8;
  if (units <= 32) s.upt = 1;
  s.threads = ((units + s.upt - 1) / s.upt + 31) / 32 * 32;
  if (s.threads > max_threads) {
    s.upt = 0;
    s.threads = max_threads;
  }
  return s;
}
int bwd_blocks(int64_t rows, const Shape& s) {
  const int per_sm = std::max(1, 512 / s.threads);
  return (int)std::min<int64_t>(rows, (int64_t)152 * per_sm);
}

template <typename T, typename Ts>
tsp_status fwd_t(const FwdArgs& a, cudaStream_t st) {
  const Shape s = shape_of(a.n, 1024);
  const int grid = (int)std::min<int64_t>(a.rows, (int64_t)num_sms() * std::max(1, 2048 / s.threads));
  Prof prof("norm_residual_fwd", st);
  if (s.upt == 0)
    norm_residual_fwd_wide_kernel<T, Ts><<<grid, s.threads, 0, st>>>(a);
  else if (s.N == 8 && s.upt == 1)
    norm_residual_fwd_kernel<T, Ts, 8, 1><<<grid, s.threads, 0, st>>>(a);
  else if (s.N == 8)
    norm_residual_fwd_kernel<T, Ts, 8, 2><<<grid, s.threads, 0, st>>>(a);
  else if (s.upt == 1)
    norm_residual_fwd_kernel<T, Ts, 1, 1><<<grid, s.threads, 0, st>>>(a);
  else
    norm_residual_fwd_kernel<T, Ts, 1, 8><<<grid, s.threads, 0, st>>>(a);
  TSP_CUDA_TRY(cudaGetLastError());
  return TSP_OK;
}

template <typename T, typename Ts>
tsp_status bwd_t(const BwdArgs& a, float* dg_post, float* dg_pre, cudaStream_t st) {
  const Shape s = shape_of(a.n, 512);
  const int grid = bwd_blocks(a.rows, s);
  const bool gains = a.g_post || a.g_pre;
  Prof prof("norm_residual_bwd", st, gains ? 2 : 1);
  if (s.upt == 0)
    norm_residual_bwd_wide_kernel<T, Ts><<<grid, s.threads, 0, st>>>(a);
  else if (s.N == 8 && s.upt == 1)
    norm_residual_bwd_kernel<T, Ts, 8, 1><<<grid, s.threads, 0, st>>>(a);
  else if (s.N == 8)
    norm_residual_bwd_kernel<T, Ts, 8, 2><<<grid, s.threads, 0, st>>>(a);
  else if (s.upt == 1)
    norm_residual_bwd_kernel<T, Ts, 1, 1><<<grid, s.threads, 0, st>>>(a);
  else
    norm_residual_bwd_kernel<T, Ts, 1, 8><<<grid, s.threads, 0, st>>>(a);
  TSP_CUDA_TRY(cudaGetLastError());
  if (gains) {
    const bool both = a.g_post && a.g_pre;
    const float* p0 = a.g_post ? a.part_post : a.part_pre;
    float* o0 = a.g_post ? dg_post : dg_pre;
    norm_residual_gain_kernel<<<dim3((a.n + 31) / 32, both ? 2 : 1), 256, 0, st>>>(
        p0, o0, a.part_pre, dg_pre, grid, a.n);
    TSP_CUDA_TRY(cudaGetLastError());
  }
  return TSP_OK;
}

}  // namespace

tsp_status launch_norm_residual_fwd(const void* f, const void* x, const void* gate,
                                    const void* g_post, const void* g_pre, void* h, void* b,
                                    float* rstd_f, float* rstd_h, int64_t rows, int n, float scale,
                                    float eps, int dtype, int stream_dtype, cudaStream_t st) {
  const FwdArgs a = {f, x, gate, g_post, g_pre, h, b, rstd_f, rstd_h, rows, n, scale, eps};
  if (dtype != TSP_BF16) return fwd_t<float, float>(a, st);
  return stream_dtype == TSP_BF16 ? fwd_t<__nv_bfloat16, __nv_bfloat16>(a, st)
                                  : fwd_t<__nv_bfloat16, float>(a, st);
}

size_t norm_residual_bwd_ws_bytes(int64_t rows, int n) {
  return (size_t)bwd_blocks(rows, shape_of(n, 512)) * n * 4 * 2;
}

tsp_status launch_norm_residual_bwd(const float* dh, const float* db, const void* f,
                                    const void* gate, const void* h, const void* g_post,
                                    const void* g_pre, const float* rstd_f, const float* rstd_h,
                                    float* dx, void* df, void* dgate, float* dg_post, float* dg_pre,
                                    int64_t rows, int n, float scale, int dtype, int stream_dtype,
                                    void* ws, cudaStream_t st) {
  float* part = (float*)ws;
  const int64_t one = (int64_t)bwd_blocks(rows, shape_of(n, 512)) * n;
  const BwdArgs a = {dh, db, f,  gate,  h,        g_post, g_pre, rstd_f, rstd_h,
                     dx, df, dgate, part, part + one, rows, n,  scale};
  if (dtype != TSP_BF16) return bwd_t<float, float>(a, dg_post, dg_pre, st);
  return stream_dtype == TSP_BF16 ? bwd_t<__nv_bfloat16, __nv_bfloat16>(a, dg_post, dg_pre, st)
                                  : bwd_t<__nv_bfloat16, float>(a, dg_post, dg_pre, st);
}

}  // namespace tsp
