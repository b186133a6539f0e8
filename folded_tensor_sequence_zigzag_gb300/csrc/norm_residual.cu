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
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace tsp {

namespace {

// N consecutive elements as they are stored (N = 4: one 8- or 16-byte access, n
// a multiple of 4; N = 1: any n).
template <typename T, int N>
struct Unit {
  T e[N];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (N == 1) e[0] = *p;
    else if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(p);
    else *reinterpret_cast<float4*>(e) = *reinterpret_cast<const float4*>(p);
  }
  __device__ __forceinline__ void get(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_f<T>(e[i]);
  }
} __attribute__((aligned(sizeof(T) * N)));

template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float (&v)[N]) {
  Unit<T, N> u;
  u.load(p);
  u.get(v);
}
template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float (&v)[N]) {
  if constexpr (N == 1)
    *p = from_f<T>(v[0]);
  else if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
  else
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Elementwise on N values, two at a time where there are four: the .f32x2 forms
// round as the scalar ones and take half the issue slots, of which the backward
// needs most.
template <int N, typename F2, typename F1>
__device__ __forceinline__ void pairs(F2 two, F1 one) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int e = 0; e < N; e += 2) two(e);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) one(e);
  }
}
template <int N>   // a = a * b
__device__ __forceinline__ void mul_n(float (&a)[N], const float (&b)[N]) {
  pairs<N>([&](int e) {
    const float2 r = fmul2(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
    a[e] = r.x; a[e + 1] = r.y;
  }, [&](int e) { a[e] *= b[e]; });
}
template <int N>   // a = a * s
__device__ __forceinline__ void mul_n(float (&a)[N], float s) {
  pairs<N>([&](int e) {
    const float2 r = fmul2(make_float2(a[e], a[e + 1]), make_float2(s, s));
    a[e] = r.x; a[e + 1] = r.y;
  }, [&](int e) { a[e] *= s; });
}
template <int N>   // c = a * b + c
__device__ __forceinline__ void fma_n(float (&c)[N], const float (&a)[N], const float (&b)[N]) {
  pairs<N>([&](int e) {
    const float2 r = ffma2(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]),
                           make_float2(c[e], c[e + 1]));
    c[e] = r.x; c[e + 1] = r.y;
  }, [&](int e) { c[e] = fmaf(a[e], b[e], c[e]); });
}
template <int N>   // c = a * s + c
__device__ __forceinline__ void fma_n(float (&c)[N], const float (&a)[N], float s) {
  pairs<N>([&](int e) {
    const float2 r = ffma2(make_float2(a[e], a[e + 1]), make_float2(s, s), make_float2(c[e], c[e + 1]));
    c[e] = r.x; c[e + 1] = r.y;
  }, [&](int e) { c[e] = fmaf(a[e], s, c[e]); });
}
template <int N>
__device__ __forceinline__ float total(const float (&v)[N]) {
  float t = v[0];
#pragma unroll
  for (int e = 1; e < N; ++e) t += v[e];
  return t;
}

// sigmoid(z) and its derivative from e = exp(-|z|), which neither overflows nor
// cancels: sigmoid(|z|) = 1 / (1 + e), sigmoid(-|z|) = e / (1 + e).  e is 2^x of
// the rounded x = -|z| log2(e): off by |z| + 2 half spacings, which the sigmoid
// has only where it is e itself, near a closed gate.
__device__ __forceinline__ float gate_of(float z, float* slope) {
  const float e = ex2_approx(-1.4426950408889634f * fabsf(z));
  float r;   // 1 / (1 + e): 1 <= 1 + e <= 2, one half spacing off at most
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  *slope = e * r * r;
  return z >= 0.f ? r : e * r;   // (a NaN gives NaN: e is one)
}
__device__ __forceinline__ float gate_of(float z) {
  float slope;
  return gate_of(z, &slope);
}

// Sum over the TPR threads of a row (TPR <= 32: a part of a warp; 0: the CTA),
// the same in every one of them.  `part` holds one value a warp and may be
// reused only after another barrier of the CTA.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
  if constexpr (TPR > 0) {
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  } else {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    v = warp_sum(v);
    if (lane == 0) part[warp] = v;
    __syncthreads();
    return warp_sum(lane < nw ? part[lane] : 0.f);
  }
}

// A copy on its way to shared memory.  Every thread copies what it will read
// itself, so waiting for its own copies is all the synchronisation there is.
template <typename T, int N>
__device__ __forceinline__ void copy_ahead(T* dst, const T* src) {
  constexpr int B = sizeof(T) * N;
  static_assert(B == 4 || B == 8 || B == 16, "a copy is 4, 8 or 16 bytes");
  // 16 bytes go past L1, which then keeps the gains (there is no such form for 4 and 8)
  if constexpr (B == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(B)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until at most `LEFT` of the groups committed last are on their way
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// The columns of a thread: UPT units of N, unit i at first + i * 32 * N, those of
// a warp next to each other.
template <int N, int UPT, int TPR>
__device__ __forceinline__ int first_col() {
  if constexpr (TPR > 0) return (int)(threadIdx.x % TPR) * N;
  return (int)((threadIdx.x >> 5) * UPT * 32 + (threadIdx.x & 31)) * N;
}

struct FwdArgs {
  const void *f, *x, *z, *g_post, *g_pre;
  void *h, *b;
  float *rstd_f, *rstd_h;
  int64_t rows;
  int n;
  float s, eps;
};

// The row in registers (first_col).
//   TPR > 0: TPR threads a row, 256 / TPR rows a CTA (short rows);
//   TPR = 0: a CTA a row.
// AHEAD (TPR = 0): past the barrier of a row sum, the next row's inputs are sent
// for, each thread's into the places it has read before that barrier, and arrive
// while this row is worked on.  Without that the loads of a row wait for the
// barriers of the one before.
template <typename T, typename Ts, int N, int UPT, int TPR, bool AHEAD>
__global__ void __launch_bounds__(UPT * N < 8 || UPT == 2 ? 512 : 1024, UPT * N < 8 || UPT == 2 ? 3 : 1)
    norm_residual_fwd_kernel(const __grid_constant__ FwdArgs a) {
  __shared__ float part[2][32];
  extern __shared__ __align__(16) uint8_t ahead[];
  constexpr int kStep = 32 * N;
  const int n = a.n, c0 = first_col<N, UPT, TPR>();
  const int group = TPR > 0 ? threadIdx.x / (TPR > 0 ? TPR : 1) : 0;
  const int64_t per = TPR > 0 ? blockDim.x / TPR : 1;
  const float inv_n = 1.f / (float)n;
  // a warp's f, z, x next to each other, at constant distances
  constexpr int kWarp = UPT * kStep;
  uint8_t* const mine = ahead + (threadIdx.x >> 5) * kWarp * (2 * sizeof(T) + sizeof(Ts));
  T* const f_in = (T*)mine + (threadIdx.x & 31) * N;
  T* const z_in = f_in + kWarp;
  Ts* const x_in = (Ts*)(mine + 2 * sizeof(T) * kWarp) + (threadIdx.x & 31) * N;
  // The copies of a row go in two groups: f, whose place is free after the first
  // sum's barrier, and x and z, free after the second's.
  auto issue_f = [&](int64_t row) {
    if constexpr (AHEAD) {
      if (row < a.rows) {
        const int64_t at = row * n + c0;
#pragma unroll
        for (int i = 0; i < UPT; ++i)
          if (c0 + i * kStep < n) copy_ahead<T, N>(f_in + i * kStep, (const T*)a.f + at + i * kStep);
      }
      copies_commit();
    }
  };
  auto issue_x = [&](int64_t row) {
    if constexpr (AHEAD) {
      if (row < a.rows) {
        const int64_t at = row * n + c0;
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
          if (c0 + i * kStep < n) {
            copy_ahead<Ts, N>(x_in + i * kStep, (const Ts*)a.x + at + i * kStep);
            if (a.z) copy_ahead<T, N>(z_in + i * kStep, (const T*)a.z + at + i * kStep);
          }
        }
      }
      copies_commit();
    }
  };
  issue_f(blockIdx.x);
  issue_x(blockIdx.x);
  for (int64_t row0 = (int64_t)blockIdx.x * per; row0 < a.rows; row0 += (int64_t)gridDim.x * per) {
    const int64_t row = row0 + group;
    const int nrow = TPR == 0 || row < a.rows ? n : 0;   // (a group past the last row does nothing)
    const int64_t at = row * n + c0;
    if constexpr (AHEAD) copies_wait<1>();   // f is there
    const T* fp = AHEAD ? f_in : (const T*)a.f + at;
    const T* zp = AHEAD ? z_in : (const T*)a.z + at;
    const Ts* xp = AHEAD ? x_in : (const Ts*)a.x + at;
    float v[UPT][N], ss[N];
    float early[AHEAD ? 1 : UPT][N];   // without copies ahead: x, on its way during the first sum
#pragma unroll
    for (int e = 0; e < N; ++e) ss[e] = 0.f;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
#pragma unroll
      for (int e = 0; e < N; ++e) v[i][e] = 0.f;
      if (c0 + i * kStep < nrow) {
        load_n<T, N>(fp + i * kStep, v[i]);
        if constexpr (!AHEAD) load_n<Ts, N>(xp + i * kStep, early[i]);
      }
    }
    float r = 1.f;
    if (a.g_post) {
#pragma unroll
      for (int i = 0; i < UPT; ++i) fma_n<N>(ss, v[i], v[i]);
      r = rsqrtf(row_sum<TPR>(total<N>(ss), part[0]) * inv_n + a.eps);
      if (c0 == 0 && nrow && a.rstd_f) a.rstd_f[row] = r;
    } else if (AHEAD) {
      __syncthreads();
    }
    if constexpr (AHEAD) copies_wait<0>();   // x and z too
    issue_f(row + gridDim.x);
#pragma unroll
    for (int e = 0; e < N; ++e) ss[e] = 0.f;
    Ts* h = (Ts*)a.h + at;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      if (c0 + i * kStep < nrow) {
        float w[N];
        if (a.g_post) {
          load_n<T, N>((const T*)a.g_post + c0 + i * kStep, w);
          mul_n<N>(w, r);
          mul_n<N>(v[i], w);
        }
        if (a.z) {
          load_n<T, N>(zp + i * kStep, w);
#pragma unroll
          for (int e = 0; e < N; ++e) w[e] = gate_of(w[e]);
          mul_n<N>(v[i], w);
        }
        if constexpr (AHEAD) {
          load_n<Ts, N>(xp + i * kStep, w);
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e) w[e] = early[i][e];
        }
        fma_n<N>(w, v[i], a.s);
#pragma unroll
        for (int e = 0; e < N; ++e) v[i][e] = to_f<Ts>(from_f<Ts>(w[e]));
        fma_n<N>(ss, v[i], v[i]);
        store_n<Ts, N>(h + i * kStep, v[i]);
      }
    }
    if (a.g_pre) {
      r = rsqrtf(row_sum<TPR>(total<N>(ss), part[1]) * inv_n + a.eps);
      if (c0 == 0 && nrow && a.rstd_h) a.rstd_h[row] = r;
      issue_x(row + gridDim.x);
      T* b = (T*)a.b + at;
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        if (c0 + i * kStep < nrow) {
          float g[N];
          load_n<T, N>((const T*)a.g_pre + c0 + i * kStep, g);
          mul_n<N>(v[i], r);
          mul_n<N>(g, v[i]);
          store_n<T, N>(b + i * kStep, g);
        }
      }
    }
    // with one barrier a row, `part` would be written again before all have read it
    if (TPR == 0 && !(a.g_post && a.g_pre)) __syncthreads();
    if (!a.g_pre) issue_x(row + gridDim.x);
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
      r = rsqrtf(row_sum<0>(ss, part[0]) * inv_n + a.eps);
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
      r = rsqrtf(row_sum<0>(ss, part[1]) * inv_n + a.eps);
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

// The same layout and the same copies ahead (dh, db, h, f, z).  A thread's
// columns are the same in every row, so its share of the gain gradients stays
// with it until the CTA's last row: in registers, or with AHEAD, where 64
// registers a thread let two CTAs of 512 run on a multiprocessor, in its own
// places in shared memory.  With several rows a CTA the groups' shares are added
// in the order of the groups.
template <typename T, typename Ts, int N, int UPT, int TPR, bool AHEAD>
__global__ void __launch_bounds__(512, UPT * N <= 8 ? 2 : 1) norm_residual_bwd_kernel(const __grid_constant__ BwdArgs a) {
  __shared__ float part[2][32];
  extern __shared__ __align__(16) uint8_t ahead[];
  constexpr int kStep = 32 * N;
  const int n = a.n, c0 = first_col<N, UPT, TPR>();
  const int group = TPR > 0 ? threadIdx.x / (TPR > 0 ? TPR : 1) : 0;
  const int64_t per = TPR > 0 ? blockDim.x / TPR : 1;
  const float inv_n = 1.f / (float)n;
  // a warp's dh, db (fp32), h, f, z and its gain sums next to each other, at
  // constant distances
  constexpr int kWarp = UPT * kStep;
  uint8_t* const mine = ahead + (threadIdx.x >> 5) * kWarp * (16 + sizeof(Ts) + 2 * sizeof(T));
  float* const sum_in = (float*)(mine + (8 + sizeof(Ts) + 2 * sizeof(T)) * kWarp) + (threadIdx.x & 31) * N;
  float dpost[AHEAD ? 1 : UPT][N], dpre[AHEAD ? 1 : UPT][N];
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
#pragma unroll
    for (int e = 0; e < N; ++e) dpost[AHEAD ? 0 : i][e] = dpre[AHEAD ? 0 : i][e] = 0.f;
    if constexpr (AHEAD) {
      store_n<float, N>(sum_in + i * kStep, dpost[0]);
      store_n<float, N>(sum_in + kWarp + i * kStep, dpost[0]);
    }
  }
  // c += a * b, in registers or in the thread's place in shared memory
  auto add_to = [&](int i, bool post, const float (&x)[N], const float (&y)[N]) {
    if constexpr (AHEAD) {
      float* at = sum_in + (post ? kWarp : 0) + i * kStep;
      float c[N];
      load_n<float, N>(at, c);
      fma_n<N>(c, x, y);
      store_n<float, N>(at, c);
    } else {
      fma_n<N>(post ? dpost[i] : dpre[i], x, y);
    }
  };
  float* const dh_in = (float*)mine + (threadIdx.x & 31) * N;
  float* const db_in = dh_in + kWarp;
  Ts* const h_in = (Ts*)(mine + 8 * kWarp) + (threadIdx.x & 31) * N;
  T* const f_in = (T*)(mine + (8 + sizeof(Ts)) * kWarp) + (threadIdx.x & 31) * N;
  T* const z_in = f_in + kWarp;
  // The copies of a row go in two groups: db and h, whose places are free after
  // the first sum's barrier, and dh, f, z, free after the second's.
  auto issue_pre = [&](int64_t row) {
    if constexpr (AHEAD) {
      if (row < a.rows && a.g_pre) {
        const int64_t at = row * n + c0;
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
          if (c0 + i * kStep < n) {
            copy_ahead<float, N>(db_in + i * kStep, a.db + at + i * kStep);
            copy_ahead<Ts, N>(h_in + i * kStep, (const Ts*)a.h + at + i * kStep);
          }
        }
      }
      copies_commit();
    }
  };
  auto issue_post = [&](int64_t row) {
    if constexpr (AHEAD) {
      if (row < a.rows) {
        const int64_t at = row * n + c0;
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
          if (c0 + i * kStep < n) {
            if (a.dh) copy_ahead<float, N>(dh_in + i * kStep, a.dh + at + i * kStep);
            copy_ahead<T, N>(f_in + i * kStep, (const T*)a.f + at + i * kStep);
            if (a.z) copy_ahead<T, N>(z_in + i * kStep, (const T*)a.z + at + i * kStep);
          }
        }
      }
      copies_commit();
    }
  };
  issue_pre(blockIdx.x);
  issue_post(blockIdx.x);
  // a row's inverse norms are loaded with the copies for it, a row ahead
  float rf_next = 1.f, rh_next = 0.f;
  auto load_rstd = [&](int64_t row) {
    if (row < a.rows) {
      if (a.g_post) rf_next = a.rstd_f[row];
      if (a.g_pre) rh_next = a.rstd_h[row];
    }
  };
  load_rstd((int64_t)blockIdx.x * per + group);
  for (int64_t row0 = (int64_t)blockIdx.x * per; row0 < a.rows; row0 += (int64_t)gridDim.x * per) {
    const int64_t row = row0 + group;
    const int nrow = TPR == 0 || row < a.rows ? n : 0;   // (a group past the last row does nothing)
    const int64_t at = row * n + c0;
    const float rf = rf_next, rh = rh_next;
    load_rstd(row + (int64_t)gridDim.x * per);
    if constexpr (AHEAD) copies_wait<1>();   // db and h are there
    const float* dhp = AHEAD ? dh_in : a.dh + at;
    const float* dbp = AHEAD ? db_in : a.db + at;
    const Ts* hp = AHEAD ? h_in : (const Ts*)a.h + at;
    const T* fp = AHEAD ? f_in : (const T*)a.f + at;
    const T* zp = AHEAD ? z_in : (const T*)a.z + at;
    float d[UPT][N];
    float dot[N];
#pragma unroll
    for (int e = 0; e < N; ++e) dot[e] = 0.f;
    if (a.g_pre) {
      float y[UPT][N], gd[UPT][N];
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        if (c0 + i * kStep < nrow) {
          float g[N];
          load_n<Ts, N>(hp + i * kStep, y[i]);
          load_n<float, N>(dbp + i * kStep, gd[i]);
          load_n<T, N>((const T*)a.g_pre + c0 + i * kStep, g);
          mul_n<N>(y[i], rh);
          add_to(i, false, gd[i], y[i]);
          mul_n<N>(gd[i], g);
          fma_n<N>(dot, gd[i], y[i]);
        }
      }
      const float mean = row_sum<TPR>(total<N>(dot), part[0]) * inv_n;
      if constexpr (AHEAD) copies_wait<0>();   // dh, f and z too
      issue_pre(row + gridDim.x);
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
#pragma unroll
        for (int e = 0; e < N; ++e) d[i][e] = 0.f;
        if (c0 + i * kStep < nrow) {
          if (a.dh) load_n<float, N>(dhp + i * kStep, d[i]);
          fma_n<N>(gd[i], y[i], -mean);
          fma_n<N>(d[i], gd[i], rh);
        }
      }
    } else {
      if constexpr (AHEAD) copies_wait<0>();
      issue_pre(row + gridDim.x);   // (an empty group)
#pragma unroll
      for (int i = 0; i < UPT; ++i)
        if (c0 + i * kStep < nrow) load_n<float, N>(dhp + i * kStep, d[i]);
    }
    float y[UPT][N];
#pragma unroll
    for (int e = 0; e < N; ++e) dot[e] = 0.f;
    float* dx = a.dx + at;
    T* dz = (T*)a.dz + at;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      if (c0 + i * kStep < nrow) {
        store_n<float, N>(dx + i * kStep, d[i]);
        load_n<T, N>(fp + i * kStep, y[i]);
        mul_n<N>(y[i], rf);
        mul_n<N>(d[i], a.s);
        float g[N];
        if (a.g_post) load_n<T, N>((const T*)a.g_post + c0 + i * kStep, g);
        if (a.z) {
          float open[N], slope[N];
          load_n<T, N>(zp + i * kStep, open);
#pragma unroll
          for (int e = 0; e < N; ++e) open[e] = gate_of(open[e], &slope[e]);
          mul_n<N>(slope, d[i]);
          mul_n<N>(slope, y[i]);
          if (a.g_post) mul_n<N>(slope, g);
          store_n<T, N>(dz + i * kStep, slope);
          mul_n<N>(d[i], open);
        }
        if (a.g_post) {
          add_to(i, true, d[i], y[i]);
          mul_n<N>(d[i], g);
          fma_n<N>(dot, d[i], y[i]);
        }
      }
    }
    T* df = (T*)a.df + at;
    if (a.g_post) {
      const float mean = row_sum<TPR>(total<N>(dot), part[1]) * inv_n;
      issue_post(row + gridDim.x);
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        if (c0 + i * kStep < nrow) {
          fma_n<N>(d[i], y[i], -mean);
          mul_n<N>(d[i], rf);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < UPT; ++i)
      if (c0 + i * kStep < nrow) store_n<T, N>(df + i * kStep, d[i]);
    if (TPR == 0 && !(a.g_post && a.g_pre)) __syncthreads();
    if (!a.g_post) issue_post(row + gridDim.x);
  }
  if constexpr (TPR > 0) {
    constexpr int kPlane = TPR * UPT * N;
    float* sum = reinterpret_cast<float*>(ahead);   // [2][groups][kPlane]
    const int groups = (int)per;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      store_n<float, N>(sum + group * kPlane + c0 + i * kStep, dpost[i]);
      store_n<float, N>(sum + (groups + group) * kPlane + c0 + i * kStep, dpre[i]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
      float p = 0.f, q = 0.f;
      for (int g = 0; g < groups; ++g) {
        p += sum[g * kPlane + c];
        q += sum[(groups + g) * kPlane + c];
      }
      if (a.g_post) a.part_post[(int64_t)blockIdx.x * n + c] = p;
      if (a.g_pre) a.part_pre[(int64_t)blockIdx.x * n + c] = q;
    }
  } else {
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      if (c0 + i * kStep < n) {
        const int64_t o = (int64_t)blockIdx.x * n + c0 + i * kStep;
        if constexpr (AHEAD) {
          load_n<float, N>(sum_in + kWarp + i * kStep, dpost[0]);
          load_n<float, N>(sum_in + i * kStep, dpre[0]);
        }
        if (a.g_post) store_n<float, N>(a.part_post + o, dpost[AHEAD ? 0 : i]);
        if (a.g_pre) store_n<float, N>(a.part_pre + o, dpre[AHEAD ? 0 : i]);
      }
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
      dot = row_sum<0>(dot, part[0]) * inv_n;
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
        float slope;
        const float open = gate_of(z, &slope);
        ((T*)a.dz)[base + c] = from_f<T>(d * (y * g) * slope);
        d *= open;
      }
      if (gpost) {
        ppost[c] = fmaf(d, y, ppost[c]);
        dot2 = fmaf(d * g, y, dot2);
      } else {
        ((T*)a.df)[base + c] = from_f<T>(d);
      }
    }
    if (gpost) {
      dot2 = row_sum<0>(dot2, part[1]) * inv_n;
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

// dg[i] = the column sums of the CTAs' partials, in a fixed order: 32 columns a
// CTA, 32 warps over the partials; blockIdx.y picks the gain.
__global__ void __launch_bounds__(1024) norm_residual_gain_kernel(const float* __restrict__ p0,
                                                                  float* __restrict__ o0,
                                                                  const float* __restrict__ p1,
                                                                  float* __restrict__ o1, int nb,
                                                                  int n) {
  __shared__ float acc[32][33];
  const float* part = blockIdx.y ? p1 : p0;
  float* out = blockIdx.y ? o1 : o0;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + tx;
  float s = 0.f;
  if (i < n) {
#pragma unroll 4
    for (int b = ty; b < nb; b += 32) s += part[(int64_t)b * n + i];
  }
  acc[ty][tx] = s;
  __syncthreads();
  s = warp_sum(acc[tx][ty]);   // column ty of this CTA
  if (tx == 0 && blockIdx.x * 32 + ty < n) out[blockIdx.x * 32 + ty] = s;
}

// How rows of n elements are laid on threads.
struct Shape {
  int N, upt;      // units of N elements, units a thread; upt == 0: the wide kernel
  int tpr;         // threads a row below 32 or of one warp; 0: the CTA
  int threads;     // of the CTA
};
Shape shape_of(int n, int max_threads) {
  Shape s;
  s.N = n % 4 == 0 ? 4 : 1;
  const int units = n / s.N;
  if (units <= 64) {              // up to two units a lane of one warp
    s.upt = units <= 32 ? 1 : 2;
    s.tpr = units <= 8 ? 8 : units <= 16 ? 16 : 32;
    s.threads = 256;
    return s;
  }
  s.tpr = 0;
  s.upt = units <= 512 ? 1 : units <= 1024 ? 2 : 4;
  if (s.N == 1 && units > 512) s.upt = units <= 2048 ? 4 : 8;
  s.threads = ((units + s.upt - 1) / s.upt + 31) / 32 * 32;
  if (s.threads > max_threads) s.upt = 0, s.threads = 1024;
  return s;
}
// CTAs a multiprocessor: what 2048 threads and the copies' shared memory allow.
// The GB300's 152 multiprocessors are a constant here because the backward's
// workspace, sized without a device, holds a partial row a CTA.
constexpr int kSms = 152, kSmemPerSm = 220 * 1024;

struct Plan {
  Shape s;
  bool ahead;
  int smem, grid;
};
Plan plan_of(int64_t rows, const Shape& s, int row_bytes_per_el, bool ahead, int threads_per_sm) {
  Plan p;
  p.s = s;
  p.ahead = false;
  p.smem = 0;
  const int per = p.s.tpr > 0 ? p.s.threads / p.s.tpr : 1;
  int per_sm = std::max(1, threads_per_sm / p.s.threads);
  const int64_t items = (rows + per - 1) / per;
  const int stage = p.s.threads * p.s.upt * p.s.N * row_bytes_per_el;
  if (ahead && p.s.tpr == 0 && p.s.upt > 0 && stage <= kSmemPerSm) {
    p.ahead = true;
    p.smem = stage;
    per_sm = std::max(1, std::min(per_sm, kSmemPerSm / (stage + 1024)));
  }
  p.grid = (int)std::min<int64_t>(items, (int64_t)kSms * per_sm);
  return p;
}

template <typename T, typename Ts>
Plan fwd_plan(int64_t rows, int n) {
  const Shape s = shape_of(n, 1024);
  // 40 registers a thread up to 8 elements, 64 above
  return plan_of(rows, s, 2 * sizeof(T) + sizeof(Ts), sizeof(T) * s.N >= 4,
                 s.upt * s.N < 8 || s.upt == 2 ? 1536 : 1024);
}
template <typename T, typename Ts>
Plan bwd_plan(int64_t rows, int n) {
  const Shape s = shape_of(n, 512);   // 128 registers a thread: gain sums and a row
  // (the inputs of a row, and two gain sums)
  return plan_of(rows, s, 16 + sizeof(Ts) + 2 * sizeof(T), sizeof(T) * s.N >= 4, 1024);
}

template <typename K, typename A>
tsp_status launch(K kernel, const Plan& p, const A& a, cudaStream_t st) {
  if (p.smem > 47 * 1024)   // (the kernels' static shared memory counts too)
    TSP_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, p.smem));
  kernel<<<p.grid, p.s.threads, p.smem, st>>>(a);
  TSP_CUDA_TRY(cudaGetLastError());
  return TSP_OK;
}

template <typename T, typename Ts, int N, int UPT>
tsp_status fwd_cta(const Plan& p, const FwdArgs& a, cudaStream_t st) {
  if constexpr (sizeof(T) * N >= 4)
    if (p.ahead) return launch(norm_residual_fwd_kernel<T, Ts, N, UPT, 0, true>, p, a, st);
  return launch(norm_residual_fwd_kernel<T, Ts, N, UPT, 0, false>, p, a, st);
}
template <typename T, typename Ts, int N>
tsp_status fwd_n(const Plan& p, const FwdArgs& a, cudaStream_t st) {
  if (p.s.tpr == 8) return launch(norm_residual_fwd_kernel<T, Ts, N, 1, 8, false>, p, a, st);
  if (p.s.tpr == 16) return launch(norm_residual_fwd_kernel<T, Ts, N, 1, 16, false>, p, a, st);
  if (p.s.tpr == 32)
    return p.s.upt == 1 ? launch(norm_residual_fwd_kernel<T, Ts, N, 1, 32, false>, p, a, st)
                        : launch(norm_residual_fwd_kernel<T, Ts, N, 2, 32, false>, p, a, st);
  if (p.s.upt == 1) return fwd_cta<T, Ts, N, 1>(p, a, st);
  if constexpr (N == 4)
    if (p.s.upt == 2) return fwd_cta<T, Ts, N, 2>(p, a, st);
  if (p.s.upt == 4) return fwd_cta<T, Ts, N, 4>(p, a, st);
  if constexpr (N == 1)
    if (p.s.upt == 8) return fwd_cta<T, Ts, N, 8>(p, a, st);
  return launch(norm_residual_fwd_wide_kernel<T, Ts>, p, a, st);
}
template <typename T, typename Ts>
tsp_status fwd_t(const FwdArgs& a, cudaStream_t st) {
  const Plan p = fwd_plan<T, Ts>(a.rows, a.n);
  Prof prof("norm_residual_fwd", st);
  return p.s.N == 4 ? fwd_n<T, Ts, 4>(p, a, st) : fwd_n<T, Ts, 1>(p, a, st);
}

template <typename T, typename Ts, int N, int UPT>
tsp_status bwd_cta(const Plan& p, const BwdArgs& a, cudaStream_t st) {
  if constexpr (sizeof(T) * N >= 4)
    if (p.ahead) return launch(norm_residual_bwd_kernel<T, Ts, N, UPT, 0, true>, p, a, st);
  return launch(norm_residual_bwd_kernel<T, Ts, N, UPT, 0, false>, p, a, st);
}
template <typename T, typename Ts, int N>
tsp_status bwd_n(Plan p, const BwdArgs& a, cudaStream_t st) {
  if (p.s.tpr > 0) {
    p.smem = 2 * p.s.threads * p.s.upt * p.s.N * 4;   // the groups' gain gradients
    if (p.s.tpr == 8) return launch(norm_residual_bwd_kernel<T, Ts, N, 1, 8, false>, p, a, st);
    if (p.s.tpr == 16) return launch(norm_residual_bwd_kernel<T, Ts, N, 1, 16, false>, p, a, st);
    return p.s.upt == 1 ? launch(norm_residual_bwd_kernel<T, Ts, N, 1, 32, false>, p, a, st)
                        : launch(norm_residual_bwd_kernel<T, Ts, N, 2, 32, false>, p, a, st);
  }
  if (p.s.upt == 1) return bwd_cta<T, Ts, N, 1>(p, a, st);
  if constexpr (N == 4)
    if (p.s.upt == 2) return bwd_cta<T, Ts, N, 2>(p, a, st);
  if (p.s.upt == 4) return bwd_cta<T, Ts, N, 4>(p, a, st);
  if constexpr (N == 1)
    if (p.s.upt == 8) return bwd_cta<T, Ts, N, 8>(p, a, st);
  return launch(norm_residual_bwd_wide_kernel<T, Ts>, p, a, st);
}

template <typename T, typename Ts>
tsp_status bwd_t(BwdArgs a, float* dg_post, float* dg_pre, void* ws, cudaStream_t st) {
  const Plan p = bwd_plan<T, Ts>(a.rows, a.n);
  const bool gains = a.g_post || a.g_pre;
  a.part_post = (float*)ws;
  a.part_pre = (float*)ws + (int64_t)p.grid * a.n;
  Prof prof("norm_residual_bwd", st, gains ? 2 : 1);
  const tsp_status r = p.s.N == 4 ? bwd_n<T, Ts, 4>(p, a, st) : bwd_n<T, Ts, 1>(p, a, st);
  if (r != TSP_OK || !gains) return r;
  const bool both = a.g_post && a.g_pre;
  const float* p0 = a.g_post ? a.part_post : a.part_pre;
  float* o0 = a.g_post ? dg_post : dg_pre;
  norm_residual_gain_kernel<<<dim3((a.n + 31) / 32, both ? 2 : 1), 1024, 0, st>>>(
      p0, o0, a.part_pre, dg_pre, p.grid, a.n);
  TSP_CUDA_TRY(cudaGetLastError());
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
  // the types differ in how many CTAs fit a multiprocessor
  typedef __nv_bfloat16 bf;
  const int grid = std::max({bwd_plan<float, float>(rows, n).grid, bwd_plan<bf, float>(rows, n).grid,
                             bwd_plan<bf, bf>(rows, n).grid});
  return (size_t)grid * n * 4 * 2;
}

tsp_status launch_norm_residual_bwd(const float* dh, const float* db, const void* f,
                                    const void* gate, const void* h, const void* g_post,
                                    const void* g_pre, const float* rstd_f, const float* rstd_h,
                                    float* dx, void* df, void* dgate, float* dg_post, float* dg_pre,
                                    int64_t rows, int n, float scale, int dtype, int stream_dtype,
                                    void* ws, cudaStream_t st) {
  const BwdArgs a = {dh, db, f,     gate,    h,       g_post, g_pre, rstd_f, rstd_h,
                     dx, df, dgate, nullptr, nullptr, rows,   n,     scale};
  if (dtype != TSP_BF16) return bwd_t<float, float>(a, dg_post, dg_pre, ws, st);
  return stream_dtype == TSP_BF16
             ? bwd_t<__nv_bfloat16, __nv_bfloat16>(a, dg_post, dg_pre, ws, st)
             : bwd_t<__nv_bfloat16, float>(a, dg_post, dg_pre, ws, st);
}

}  // namespace tsp
