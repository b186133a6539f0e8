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
#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace tsp {

namespace {

// Rows are worked on in units of four elements, one 8- or 16-byte access.  Where
// n % 4 != 0 (RAGGED) the units are those of the whole tensor, so that they are
// aligned all the same: a row starts s = row * n % 4 elements into its first unit,
// and the units at its two ends hold elements of other rows too, which are left
// alone.  A thread's rows are a multiple of four apart, so its s is one number and
// its columns (c .. c + 3, c = 4 * unit - s) are the same in all of them.
template <bool RAGGED>
__device__ __forceinline__ bool is_here(int c, int n) {
  return c < n && (!RAGGED || c + 4 > 0);
}
template <bool RAGGED>
__device__ __forceinline__ bool is_whole(int c, int n) {
  return !RAGGED || (c >= 0 && c + 4 <= n);
}
template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&v)[4]) {
  if constexpr (sizeof(T) == 2) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = lo2<T>(q.x); v[1] = hi2<T>(q.x); v[2] = lo2<T>(q.y); v[3] = hi2<T>(q.y);
  } else {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  }
}
// the unit at column c of the row at `row`; elements of other rows are 0
template <bool RAGGED, typename T>
__device__ __forceinline__ void load_unit(const T* row, int c, int n, float (&v)[4]) {
  if (is_whole<RAGGED>(c, n)) {
    load4<T>(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = c + e >= 0 && c + e < n ? to_f<T>(row[c + e]) : 0.f;
  }
}
// a gain, whose own start is column 0: not aligned to the units of a ragged row
template <bool RAGGED, typename T>
__device__ __forceinline__ void load_gain(const T* g, int c, int n, float (&v)[4]) {
  if constexpr (RAGGED) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = c + e >= 0 && c + e < n ? to_f<T>(g[c + e]) : 0.f;
  } else {
    load4<T>(g + c, v);
  }
}
// a unit copied ahead, whole: what is not this row's is masked
template <bool RAGGED, typename T>
__device__ __forceinline__ void load_copied(const T* unit, int c, int n, float (&v)[4]) {
  load4<T>(unit, v);
  if (!is_whole<RAGGED>(c, n)) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < 0 || c + e >= n) v[e] = 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&v)[4]) {
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
  else
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <bool RAGGED, typename T>
__device__ __forceinline__ void store_unit(T* row, int c, int n, const float (&v)[4]) {
  if (is_whole<RAGGED>(c, n)) {
    store4<T>(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e >= 0 && c + e < n) row[c + e] = from_f<T>(v[e]);
  }
}

// Elementwise on four values, two an instruction: the .f32x2 forms take half the
// issue slots, of which the backward needs most.
__device__ __forceinline__ void mul4(float (&a)[4], const float (&b)[4]) {   // a = a * b
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const float2 r = fmul2(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
    a[e] = r.x; a[e + 1] = r.y;
  }
}
__device__ __forceinline__ void mul4(float (&a)[4], float s) {
  const float b[4] = {s, s, s, s};
  mul4(a, b);
}
// c = a * b + c
__device__ __forceinline__ void fma4(float (&c)[4], const float (&a)[4], const float (&b)[4]) {
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const float2 r = ffma2(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]),
                           make_float2(c[e], c[e + 1]));
    c[e] = r.x; c[e + 1] = r.y;
  }
}
__device__ __forceinline__ void fma4(float (&c)[4], const float (&a)[4], float s) {
  const float b[4] = {s, s, s, s};
  fma4(c, a, b);
}
__device__ __forceinline__ void zero4(float (&v)[4]) { v[0] = v[1] = v[2] = v[3] = 0.f; }
__device__ __forceinline__ float total(const float (&v)[4]) { return (v[0] + v[1]) + (v[2] + v[3]); }

// sigmoid(z) and its derivative from e = exp(-|z|), which neither overflows nor
// cancels: sigmoid(|z|) = 1 / (1 + e), sigmoid(-|z|) = e / (1 + e).  e is 2^x of the
// rounded x = -|z| log2(e), off by |z| half spacings of fp32 and what ex2 adds (2 or
// 3), which the sigmoid has only where it is e itself, near a closed gate: far below
// what a gate held in bf16 is uncertain by.  For gates in fp32 the rounding y of x is
// made up for, 2^(x + y) = 2^x (1 + y ln 2): against 64 bits, every z of 1e-30 <= |z|
// <= 87, an open gate is then off by 3 half spacings at most, a closed one by 5.3, the
// slope by 7.4 (16384 x 4096 fp32: 201 us with and without; bf16 would go from 115 to
// 120).  Beyond 87.3 e is 0.
template <typename T>
__device__ __forceinline__ float gate_of(float z, float* slope) {
  constexpr float hi = 1.4426950408889634f, lo = (float)(1.4426950408889634074 - (double)hi);
  float e;
  if constexpr (sizeof(T) == 4) {
    const float a = fabsf(z) > 128.f ? 128.f : fabsf(z);   // (infinity has no y; a NaN stays)
    const float x = -hi * a, y = fmaf(-lo, a, fmaf(-hi, a, -x));
    e = ex2_approx(x);
    e = fmaf(e, 0.6931471805599453f * y, e);
  } else {
    e = ex2_approx(-hi * fabsf(z));
  }
  float r;   // 1 / (1 + e): 1 <= 1 + e <= 2, a spacing off at most
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  *slope = e * r * r;
  return z >= 0.f ? r : e * r;   // (a NaN gives NaN: e is one)
}
template <typename T>
__device__ __forceinline__ float gate_of(float z) {
  float slope;
  return gate_of<T>(z, &slope);
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

// A unit on its way to shared memory, whole (what it holds of other rows is read
// past); only the tensor's last one may end beyond it, and is loaded by element.
// Every thread copies what it will read itself, so waiting for its own copies is
// all the synchronisation there is.  left: elements from the unit's first to the
// tensor's end.  copy_own: the same of the row's own elements alone, where the
// tensor is also the output and other CTAs may be writing its other rows.
template <bool RAGGED, typename T>
__device__ __forceinline__ void copy_ahead(T* dst, const T* src, int64_t left) {
  constexpr int B = sizeof(T) * 4;
  if (RAGGED && left < 4) {
    for (int e = 0; e < 4; ++e)
      if (e < left) dst[e] = src[e];
    return;
  }
  // 16 bytes go past L1, which then keeps the gains (there is no such form for 8)
  if constexpr (B == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
template <bool RAGGED, typename T>
__device__ __forceinline__ void copy_own(T* dst, const T* src, int c, int n) {
  if (is_whole<RAGGED>(c, n)) {
    copy_ahead<false>(dst, src, 4);
    return;
  }
  for (int e = 0; e < 4; ++e)
    if (c + e >= 0 && c + e < n) dst[e] = src[e];
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until at most `LEFT` of the groups committed last are on their way
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// A thread's UPT units are kStep elements apart, those of a warp next to each other.
constexpr int kStep = 128;
template <int UPT, int TPR>
__device__ __forceinline__ int first_unit() {
  if constexpr (TPR > 0) return (int)(threadIdx.x % TPR) * 4;
  return (int)((threadIdx.x >> 5) * UPT * 32 + (threadIdx.x & 31)) * 4;
}
// s of the rows of a thread (see RAGGED)
template <bool RAGGED>
__device__ __forceinline__ int start_of(int64_t row, int n) {
  return RAGGED ? (int)((row * n) & 3) : 0;
}

struct FwdArgs {
  const void *f, *x, *z, *g_post, *g_pre;
  void *h, *b;
  float *rstd_f, *rstd_h;
  int64_t rows;
  int n;
  float s, eps;
};

// The row in registers:
//   TPR > 0: TPR threads a row, 256 / TPR rows a CTA (short rows, no barriers);
//   TPR = 0: a CTA a row.
// AHEAD (TPR = 0): past the barrier of a row sum, the next row's inputs are sent
// for, each thread's into the places it has read before that barrier, and arrive
// while this row is worked on.  Without that the loads of a row wait for the
// barriers of the one before.
// HBM-bound: 16384 x 4096 bf16 beside an fp32 stream (0.94 GB) in 147 us, 6.4 TB/s,
// with 41% of the issue slots used; one row of 4096 takes 2.8 us.
template <typename T, typename Ts, int UPT, int TPR, bool AHEAD, bool RAGGED>
__global__ void __launch_bounds__(TPR > 0 ? 256 : 1024, TPR > 0 ? 6 : 1) norm_residual_fwd_kernel(const __grid_constant__ FwdArgs a) {
  __shared__ float part[2][32];
  extern __shared__ __align__(16) uint8_t ahead[];
  const int n = a.n;
  const int group = TPR > 0 ? threadIdx.x / (TPR > 0 ? TPR : 1) : 0;
  const int64_t per = TPR > 0 ? blockDim.x / TPR : 1;
  const int64_t total_n = a.rows * n;
  const int unit0 = first_unit<UPT, TPR>();
  const int c0 = unit0 - start_of<RAGGED>((int64_t)blockIdx.x * per + group, n);
  const float inv_n = 1.f / (float)n;
  // a warp's f, z, x next to each other, at constant distances
  constexpr int kWarp = UPT * kStep;
  uint8_t* const mine = ahead + (threadIdx.x >> 5) * kWarp * (2 * sizeof(T) + sizeof(Ts));
  T* const f_in = (T*)mine + (threadIdx.x & 31) * 4;
  T* const z_in = f_in + kWarp;
  Ts* const x_in = (Ts*)(mine + 2 * sizeof(T) * kWarp) + (threadIdx.x & 31) * 4;
  // The copies of a row go in two groups: f, whose place is free after the first
  // sum's barrier, and x and z, free after the second's.
  auto issue_f = [&](int64_t row) {
    if constexpr (AHEAD) {
      if (row < a.rows) {
        const int64_t at = row * n + c0;
#pragma unroll
        for (int i = 0; i < UPT; ++i)
          if (is_here<RAGGED>(c0 + i * kStep, n))
            copy_ahead<RAGGED>(f_in + i * kStep, (const T*)a.f + at + i * kStep, total_n - at - i * kStep);
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
          if (is_here<RAGGED>(c0 + i * kStep, n)) {
            const int64_t left = total_n - at - i * kStep;
            const Ts* x = (const Ts*)a.x + at + i * kStep;
            if (RAGGED && a.x == a.h) copy_own<RAGGED>(x_in + i * kStep, x, c0 + i * kStep, n);
            else copy_ahead<RAGGED>(x_in + i * kStep, x, left);
            if (a.z) copy_ahead<RAGGED>(z_in + i * kStep, (const T*)a.z + at + i * kStep, left);
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
    const int nrow = TPR == 0 || row < a.rows ? n : -4;   // (a group past the last row does nothing)
    const int64_t base = row * n;
    if constexpr (AHEAD) copies_wait<1>();   // f is there
    float v[UPT][4], ss[4];
    // without copies ahead: x and z, on their way during the first sum
    float early[AHEAD ? 1 : UPT][4], early_z[AHEAD ? 1 : UPT][4];
    zero4(ss);
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int c = c0 + i * kStep;
      zero4(v[i]);
      if (is_here<RAGGED>(c, nrow)) {
        if constexpr (AHEAD) {
          load_copied<RAGGED>(f_in + i * kStep, c, n, v[i]);
        } else {
          load_unit<RAGGED>((const T*)a.f + base, c, n, v[i]);
          load_unit<RAGGED>((const Ts*)a.x + base, c, n, early[i]);
          if (a.z) load_unit<RAGGED>((const T*)a.z + base, c, n, early_z[i]);
        }
      }
    }
    float r = 1.f;
    if (a.g_post) {
#pragma unroll
      for (int i = 0; i < UPT; ++i) fma4(ss, v[i], v[i]);
      r = rsqrtf(row_sum<TPR>(total(ss), part[0]) * inv_n + a.eps);
      if (unit0 == 0 && nrow > 0 && a.rstd_f) a.rstd_f[row] = r;
    } else if (AHEAD) {
      __syncthreads();
    }
    if constexpr (AHEAD) copies_wait<0>();   // x and z too
    issue_f(row + gridDim.x);
    zero4(ss);
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int c = c0 + i * kStep;
      if (is_here<RAGGED>(c, nrow)) {
        float w[4];
        if (a.g_post) {
          load_gain<RAGGED>((const T*)a.g_post, c, n, w);
          mul4(v[i], r);
          mul4(v[i], w);
        }
        if (a.z) {
          if constexpr (AHEAD) load_copied<RAGGED>(z_in + i * kStep, c, n, w);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = gate_of<T>(AHEAD ? w[e] : early_z[AHEAD ? 0 : i][e]);
          mul4(v[i], w);
        }
        if constexpr (AHEAD) {
          load_copied<RAGGED>(x_in + i * kStep, c, n, w);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = early[i][e];
        }
        fma4(w, v[i], a.s);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = to_f<Ts>(from_f<Ts>(w[e]));
        fma4(ss, v[i], v[i]);
        store_unit<RAGGED>((Ts*)a.h + base, c, n, v[i]);
      }
    }
    if (a.g_pre) {
      r = rsqrtf(row_sum<TPR>(total(ss), part[1]) * inv_n + a.eps);
      if (unit0 == 0 && nrow > 0 && a.rstd_h) a.rstd_h[row] = r;
      issue_x(row + gridDim.x);
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int c = c0 + i * kStep;
        if (is_here<RAGGED>(c, nrow)) {
          float g[4];
          load_gain<RAGGED>((const T*)a.g_pre, c, n, g);
          mul4(v[i], r);
          mul4(g, v[i]);
          store_unit<RAGGED>((T*)a.b + base, c, n, g);
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
    // columns whose loads are ahead of the first one's store (2000 x 20000 fp32: 330 us, 500
    // with one; bf16: 412 with four, 398 with one)
    constexpr int K = sizeof(T) == 4 ? 4 : 1;
    for (int c0 = threadIdx.x; c0 < n; c0 += K * blockDim.x) {
      float u[K], gate[K], old[K], gain[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = c0 + k * blockDim.x;
        u[k] = c < n ? to_f<T>(f[c]) : 0.f;
        gate[k] = z && c < n ? to_f<T>(z[c]) : 0.f;
        old[k] = c < n ? to_f<Ts>(x[c]) : 0.f;
        gain[k] = a.g_post && c < n ? to_f<T>(((const T*)a.g_post)[c]) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = c0 + k * blockDim.x;
        if (c >= n) continue;
        if (a.g_post) u[k] = u[k] * r * gain[k];
        if (z) u[k] *= gate_of<T>(gate[k]);
        const Ts o = from_f<Ts>(fmaf(a.s, u[k], old[k]));
        h[c] = o;
        ss = fmaf(to_f<Ts>(o), to_f<Ts>(o), ss);
      }
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

// The gain sums of a CTA-wide row are in shared memory where 64 registers a thread
// let two CTAs of 512 run on a multiprocessor (two units a thread).  (Of fp32 rows of
// more than 3840 elements the copies and sums leave room for one: 16384 x 4096 with a
// gate takes 388 us, 82% of the copy rate; bf16 with an fp32 stream 249 us, 95%.)
// (Four units a thread need 128 registers: 512 threads, rows of up to 8192.)
constexpr int kMaxBwdThreads = 512;
constexpr bool gain_sums_in_smem(int upt, bool ahead) { return ahead && upt <= 2; }

// The same layout and the same copies ahead (dh, db, h, f, z).  A thread's
// columns are the same in every row, so its share of the gain gradients stays
// with it until the CTA's last row, in registers or in its own places in shared
// memory.  With several rows a CTA the groups' shares are added in the order of
// the groups.
// HBM-bound where rows are a multiple of four: 32768 x 4096, both norms and the
// gate, (3.2 GB) in 486 us, 6.6 TB/s; the gain kernel's 7 us are in that.  Ragged
// rows (4099 x 1001 fp32: 28 us, half the copy rate) wait for the barriers of short rows
// and the element accesses at their ends.
template <typename T, typename Ts, int UPT, int TPR, bool AHEAD, bool RAGGED>
__global__ void __launch_bounds__(TPR > 0 ? 256 : kMaxBwdThreads,
                                  TPR > 0 ? 3 : UPT <= 2 ? 2 : 1)
    norm_residual_bwd_kernel(const __grid_constant__ BwdArgs a) {
  __shared__ float part[2][32];
  extern __shared__ __align__(16) uint8_t ahead[];
  constexpr bool kSums = gain_sums_in_smem(UPT, AHEAD);
  const int n = a.n;
  const int group = TPR > 0 ? threadIdx.x / (TPR > 0 ? TPR : 1) : 0;
  const int64_t per = TPR > 0 ? blockDim.x / TPR : 1;
  const int64_t total_n = a.rows * n;
  const int c0 = first_unit<UPT, TPR>() - start_of<RAGGED>((int64_t)blockIdx.x * per + group, n);
  const float inv_n = 1.f / (float)n;
  // a warp's dh, db (fp32), h, f, z and its gain sums next to each other, at
  // constant distances
  constexpr int kWarp = UPT * kStep;
  uint8_t* const mine = ahead + (threadIdx.x >> 5) * kWarp * ((kSums ? 16 : 8) + sizeof(Ts) + 2 * sizeof(T));
  float* const dh_in = (float*)mine + (threadIdx.x & 31) * 4;
  float* const db_in = dh_in + kWarp;
  Ts* const h_in = (Ts*)(mine + 8 * kWarp) + (threadIdx.x & 31) * 4;
  T* const f_in = (T*)(mine + (8 + sizeof(Ts)) * kWarp) + (threadIdx.x & 31) * 4;
  T* const z_in = f_in + kWarp;
  float* const sum_in = (float*)(mine + (8 + sizeof(Ts) + 2 * sizeof(T)) * kWarp) + (threadIdx.x & 31) * 4;
  float dpost[kSums ? 1 : UPT][4], dpre[kSums ? 1 : UPT][4];
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    zero4(dpost[kSums ? 0 : i]);
    zero4(dpre[kSums ? 0 : i]);
    if constexpr (kSums) {
      store4(sum_in + i * kStep, dpost[0]);
      store4(sum_in + kWarp + i * kStep, dpost[0]);
    }
  }
  // the gain sum += x * y
  auto add_to = [&](int i, bool post, const float (&x)[4], const float (&y)[4]) {
    if constexpr (kSums) {
      float* at = sum_in + (post ? kWarp : 0) + i * kStep;
      float c[4];
      load4(at, c);
      fma4(c, x, y);
      store4(at, c);
    } else {
      fma4(post ? dpost[i] : dpre[i], x, y);
    }
  };
  // The copies of a row go in two groups: db and h, whose places are free after
  // the first sum's barrier, and dh, f, z, free after the second's.
  auto issue_pre = [&](int64_t row) {
    if constexpr (AHEAD) {
      if (row < a.rows && a.g_pre) {
        const int64_t at = row * n + c0;
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
          if (is_here<RAGGED>(c0 + i * kStep, n)) {
            const int64_t left = total_n - at - i * kStep;
            copy_ahead<RAGGED>(db_in + i * kStep, a.db + at + i * kStep, left);
            copy_ahead<RAGGED>(h_in + i * kStep, (const Ts*)a.h + at + i * kStep, left);
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
          if (is_here<RAGGED>(c0 + i * kStep, n)) {
            const int64_t left = total_n - at - i * kStep;
            if (RAGGED && a.dh == a.dx) copy_own<RAGGED>(dh_in + i * kStep, a.dh + at + i * kStep, c0 + i * kStep, n);
            else if (a.dh) copy_ahead<RAGGED>(dh_in + i * kStep, a.dh + at + i * kStep, left);
            copy_ahead<RAGGED>(f_in + i * kStep, (const T*)a.f + at + i * kStep, left);
            if (a.z) copy_ahead<RAGGED>(z_in + i * kStep, (const T*)a.z + at + i * kStep, left);
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
    const int nrow = TPR == 0 || row < a.rows ? n : -4;   // (a group past the last row does nothing)
    const int64_t base = row * n;
    const float rf = rf_next, rh = rh_next;
    load_rstd(row + (int64_t)gridDim.x * per);
    if constexpr (AHEAD) copies_wait<1>();   // db and h are there
    float d[UPT][4], y[UPT][4], dot[4];
    // without copies ahead: f and z too are on their way before the first sum
    float early_f[AHEAD ? 1 : UPT][4], early_z[AHEAD ? 1 : UPT][4];
    zero4(dot);
    if constexpr (!AHEAD) {
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int c = c0 + i * kStep;
        zero4(d[i]);
        if (is_here<RAGGED>(c, nrow)) {
          if (a.dh) load_unit<RAGGED>(a.dh + base, c, n, d[i]);
          load_unit<RAGGED>((const T*)a.f + base, c, n, early_f[i]);
          if (a.z) load_unit<RAGGED>((const T*)a.z + base, c, n, early_z[i]);
        }
      }
    }
    if (a.g_pre) {
      float gd[UPT][4];
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int c = c0 + i * kStep;
        if (is_here<RAGGED>(c, nrow)) {
          float g[4];
          if constexpr (AHEAD) {
            load_copied<RAGGED>(h_in + i * kStep, c, n, y[i]);
            load_copied<RAGGED>(db_in + i * kStep, c, n, gd[i]);
          } else {
            load_unit<RAGGED>((const Ts*)a.h + base, c, n, y[i]);
            load_unit<RAGGED>(a.db + base, c, n, gd[i]);
          }
          load_gain<RAGGED>((const T*)a.g_pre, c, n, g);
          mul4(y[i], rh);
          add_to(i, false, gd[i], y[i]);
          mul4(gd[i], g);
          fma4(dot, gd[i], y[i]);
        }
      }
      const float mean = row_sum<TPR>(total(dot), part[0]) * inv_n;
      if constexpr (AHEAD) copies_wait<0>();   // dh, f and z too
      issue_pre(row + gridDim.x);
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int c = c0 + i * kStep;
        if constexpr (AHEAD) zero4(d[i]);
        if (is_here<RAGGED>(c, nrow)) {
          if constexpr (AHEAD)
            if (a.dh) load_copied<RAGGED>(dh_in + i * kStep, c, n, d[i]);
          fma4(gd[i], y[i], -mean);
          fma4(d[i], gd[i], rh);
        }
      }
    } else if constexpr (AHEAD) {
      copies_wait<0>();
      issue_pre(row + gridDim.x);   // (an empty group)
#pragma unroll
      for (int i = 0; i < UPT; ++i)
        if (is_here<RAGGED>(c0 + i * kStep, nrow))
          load_copied<RAGGED>(dh_in + i * kStep, c0 + i * kStep, n, d[i]);
    }
    zero4(dot);
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int c = c0 + i * kStep;
      if (is_here<RAGGED>(c, nrow)) {
        store_unit<RAGGED>(a.dx + base, c, n, d[i]);
        if constexpr (AHEAD) {
          load_copied<RAGGED>(f_in + i * kStep, c, n, y[i]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[i][e] = early_f[i][e];
        }
        mul4(y[i], rf);
        mul4(d[i], a.s);
        float g[4];
        if (a.g_post) load_gain<RAGGED>((const T*)a.g_post, c, n, g);
        if (a.z) {
          float open[4], slope[4];
          if constexpr (AHEAD) {
            load_copied<RAGGED>(z_in + i * kStep, c, n, open);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) open[e] = early_z[i][e];
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) open[e] = gate_of<T>(open[e], &slope[e]);
          mul4(slope, d[i]);
          mul4(slope, y[i]);
          if (a.g_post) mul4(slope, g);
          store_unit<RAGGED>((T*)a.dz + base, c, n, slope);
          mul4(d[i], open);
        }
        if (a.g_post) {
          add_to(i, true, d[i], y[i]);
          mul4(d[i], g);
          fma4(dot, d[i], y[i]);
        }
      }
    }
    if (a.g_post) {
      const float mean = row_sum<TPR>(total(dot), part[1]) * inv_n;
      issue_post(row + gridDim.x);
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        if (is_here<RAGGED>(c0 + i * kStep, nrow)) {
          fma4(d[i], y[i], -mean);
          mul4(d[i], rf);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < UPT; ++i)
      if (is_here<RAGGED>(c0 + i * kStep, nrow)) store_unit<RAGGED>((T*)a.df + base, c0 + i * kStep, n, d[i]);
    if (TPR == 0 && !(a.g_post && a.g_pre)) __syncthreads();
    if (!a.g_post) issue_post(row + gridDim.x);
  }
  if constexpr (TPR > 0) {
    float* sum = reinterpret_cast<float*>(ahead);   // [2][groups][n]
    const int groups = (int)per;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = c0 + i * kStep + e;
        if (c < 0 || c >= n) continue;
        sum[group * n + c] = dpost[i][e];
        sum[(groups + group) * n + c] = dpre[i][e];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
      float p = 0.f, q = 0.f;
      for (int g = 0; g < groups; ++g) {
        p += sum[g * n + c];
        q += sum[(groups + g) * n + c];
      }
      if (a.g_post) a.part_post[(int64_t)blockIdx.x * n + c] = p;
      if (a.g_pre) a.part_pre[(int64_t)blockIdx.x * n + c] = q;
    }
  } else {
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int c = c0 + i * kStep;
      if (is_here<RAGGED>(c, n)) {
        if constexpr (kSums) {
          load4(sum_in + kWarp + i * kStep, dpost[0]);
          load4(sum_in + i * kStep, dpre[0]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (c + e < 0 || c + e >= n) continue;
          if (a.g_post) a.part_post[(int64_t)blockIdx.x * n + c + e] = dpost[kSums ? 0 : i][e];
          if (a.g_pre) a.part_pre[(int64_t)blockIdx.x * n + c + e] = dpre[kSums ? 0 : i][e];
        }
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
        const float open = gate_of<T>(z, &slope);
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
        if (a.z) d *= gate_of<T>(to_f<T>(((const T*)a.z)[base + c]));
        const float y = to_f<T>(((const T*)a.f)[base + c]) * rf;
        ((T*)a.df)[base + c] = from_f<T>(rf * (d * to_f<T>(gpost[c]) - y * dot2));
      }
    }
    __syncthreads();
  }
}

// dg[i] = the column sums of the CTAs' partials, in a fixed order: COLS columns a
// CTA, 1024 / COLS partial rows at a time; blockIdx.y picks the gain.
template <int COLS>
__global__ void __launch_bounds__(1024) norm_residual_gain_kernel(const float* p0, float* __restrict__ o0,
                                                                  const float* p1, float* __restrict__ o1,
                                                                  int nb, int n) {
  constexpr int R = 1024 / COLS;
  __shared__ float acc[COLS][R + 1];
  after_previous_kernel();
  const float* part = blockIdx.y ? p1 : p0;
  float* out = blockIdx.y ? o1 : o0;
  const int tx = threadIdx.x % COLS, ty = threadIdx.x / COLS;
  const int i = blockIdx.x * COLS + tx;
  float s = 0.f;
  if (i < n) {
#pragma unroll 4
    for (int b = ty; b < nb; b += R) s += part[(int64_t)b * n + i];
  }
  acc[tx][ty] = s;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp >= COLS) return;
  s = 0.f;
#pragma unroll
  for (int r = 0; r < R; r += 32) s += acc[warp][r + lane];
  s = warp_sum(s);
  if (lane == 0 && blockIdx.x * COLS + warp < n) out[blockIdx.x * COLS + warp] = s;
}

// How rows of n elements are laid on threads, and the grid.
struct Plan {
  int upt;         // units a thread; 0: the wide kernel
  int tpr;         // threads a row, of one warp at most; 0: the CTA
  int threads;     // of the CTA
  bool ahead, ragged;
  int smem, grid;
};
// The GB300's 152 multiprocessors are a constant here because the backward's
// workspace, sized without a device, holds a partial row a CTA.  (A multiple of
// four, as ragged rows need: a grid below it gives every CTA one row.)
constexpr int kSms = 152, kSmemPerSm = 224 * 1024;

void set_grid(Plan* p, int64_t rows, int per_sm) {
  const int per = p->tpr > 0 ? p->threads / p->tpr : 1;
  p->grid = (int)std::min<int64_t>((rows + per - 1) / per, (int64_t)kSms * std::max(1, per_sm));
}
// upt units a thread of a CTA, with the next row's `bytes` an element copied ahead
// (0: nothing is).  What the widest rows take fits: launch() asserts it.
void set_cta(Plan* p, int64_t rows, int units, int upt, int bytes, int threads_per_sm) {
  p->upt = upt;
  p->tpr = 0;
  p->threads = ((units + upt - 1) / upt + 31) / 32 * 32;
  p->ahead = bytes > 0;
  p->smem = p->threads * upt * 4 * bytes;
  set_grid(p, rows, std::min({32, threads_per_sm / p->threads, kSmemPerSm / (p->smem + 1024)}));
}
// Rows of up to 256 elements lie in a part of a warp.  With two units a lane (132 to 256)
// the backward spills 36 to 136 bytes a thread at three CTAs a multiprocessor, the
// forward 8 to 48 at six: 131072 x 256 with a gate and both norms takes 112 us forward
// and 181 backward in fp32 (88% of the copy rate), 64 and 158 in bf16 (78 and 69%).
Plan start_plan(int n, int* units) {
  Plan p = {};
  p.ragged = n % 4 != 0;
  *units = p.ragged ? (n + 6) / 4 : n / 4;   // (up to three elements before the row)
  p.threads = 256;
  p.tpr = *units <= 8 ? 8 : *units <= 16 ? 16 : 32;
  p.upt = *units <= 32 ? 1 : 2;
  return p;
}

// Shared memory for an element of a row that is copied ahead.
template <typename T, typename Ts>
constexpr int fwd_bytes() {
  return 2 * sizeof(T) + sizeof(Ts);
}
template <typename T, typename Ts>
constexpr int bwd_bytes(int upt) {
  return (gain_sums_in_smem(upt, true) ? 16 : 8) + sizeof(Ts) + 2 * sizeof(T);
}

template <typename T, typename Ts>
Plan fwd_plan(int64_t rows, int n) {
  int units;
  Plan p = start_plan(n, &units);
  if (units <= 64) {
    set_grid(&p, rows, 6);
  } else if (rows <= kSms && units <= 2 * 1024) {
    // a row a CTA and nothing to copy ahead (decoded tokens): as many threads as
    // there are units, all loads at once (1 x 4096: 2.8 us, 4.6 with four units each)
    set_cta(&p, rows, units, units <= 1024 ? 1 : 2, 0, 1024);
  } else if (units <= 4 * 1024) {
    // four units a thread: more rows at a time than with two or one (2048 bf16,
    // fp32 stream: 91% of the copy rate against 69% with one)
    set_cta(&p, rows, units, 4, fwd_bytes<T, Ts>(), 1024);
  } else {
    p.upt = p.tpr = 0;
    p.threads = 1024;
    set_grid(&p, rows, 1);
  }
  return p;
}
template <typename T, typename Ts>
Plan bwd_plan(int64_t rows, int n) {
  int units;
  Plan p = start_plan(n, &units);
  if (units <= 64) {
    p.smem = 2 * (p.threads / p.tpr) * n * 4;   // the groups' gain gradients
    set_grid(&p, rows, 3);
  } else if (units <= 4 * kMaxBwdThreads) {
    const int upt = units <= 1024 ? 2 : 4;
    set_cta(&p, rows, units, upt, bwd_bytes<T, Ts>(upt), upt == 2 ? 1024 : kMaxBwdThreads);
    // two rows a CTA at least: a CTA's partial gains cost about the traffic of one
    if (p.grid > kSms) p.grid = (int)std::max<int64_t>(kSms, std::min<int64_t>(p.grid, rows / 8 * 4));
  } else {
    p.upt = p.tpr = 0;
    p.threads = 1024;
    set_grid(&p, rows, 1);
  }
  return p;
}

// MOST: the dynamic shared memory of the kernel's widest row.  The limit is a property of
// the kernel on a device, which calls of all widths and host threads share: it is set
// once, to that.
template <auto KERNEL, int MOST, typename A>
tsp_status launch(const Plan& p, const A& a, cudaStream_t st) {
  static_assert(MOST <= kSmemPerSm, "a row's copies have to fit");
  if constexpr (MOST > 47 * 1024) {   // (the kernels' static shared memory counts too)
    static std::atomic<bool> set[kMaxDevices];
    const int dev = current_device();
    if (!set[dev]) {
      TSP_CUDA_TRY(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST));
      set[dev] = true;
    }
  }
  KERNEL<<<p.grid, p.threads, p.smem, st>>>(a);
  TSP_CUDA_TRY(cudaGetLastError());
  return TSP_OK;
}

template <typename T, typename Ts, bool RAGGED>
tsp_status fwd_r(const Plan& p, const FwdArgs& a, cudaStream_t st) {
#define TSP_NRF(upt, tpr, most) \
  launch<norm_residual_fwd_kernel<T, Ts, upt, tpr, (most > 0), RAGGED>, most>(p, a, st)
  if (p.tpr == 8) return TSP_NRF(1, 8, 0);
  if (p.tpr == 16) return TSP_NRF(1, 16, 0);
  if (p.tpr == 32) return p.upt == 1 ? TSP_NRF(1, 32, 0) : TSP_NRF(2, 32, 0);
  if (!p.ahead) return p.upt == 1 ? TSP_NRF(1, 0, 0) : TSP_NRF(2, 0, 0);
  return TSP_NRF(4, 0, (1024 * 16 * fwd_bytes<T, Ts>()));
#undef TSP_NRF
}
template <typename T, typename Ts>
tsp_status fwd_t(const FwdArgs& a, cudaStream_t st) {
  const Plan p = fwd_plan<T, Ts>(a.rows, a.n);
  Prof prof("norm_residual_fwd", st);
  if (p.upt == 0) return launch<norm_residual_fwd_wide_kernel<T, Ts>, 0>(p, a, st);
  return p.ragged ? fwd_r<T, Ts, true>(p, a, st) : fwd_r<T, Ts, false>(p, a, st);
}

template <typename T, typename Ts, bool RAGGED>
tsp_status bwd_r(const Plan& p, const BwdArgs& a, cudaStream_t st) {
#define TSP_NRB(upt, tpr, most) \
  launch<norm_residual_bwd_kernel<T, Ts, upt, tpr, (tpr == 0), RAGGED>, most>(p, a, st)
  if (p.tpr == 8) return TSP_NRB(1, 8, 0);
  if (p.tpr == 16) return TSP_NRB(1, 16, 0);
  if (p.tpr == 32) return p.upt == 1 ? TSP_NRB(1, 32, 0) : TSP_NRB(2, 32, 0);
  if (p.upt == 2) return TSP_NRB(2, 0, (kMaxBwdThreads * 8 * bwd_bytes<T, Ts>(2)));
  return TSP_NRB(4, 0, (kMaxBwdThreads * 16 * bwd_bytes<T, Ts>(4)));
#undef TSP_NRB
}

template <typename T, typename Ts>
tsp_status bwd_t(BwdArgs a, float* dg_post, float* dg_pre, void* ws, cudaStream_t st) {
  const Plan p = bwd_plan<T, Ts>(a.rows, a.n);
  const bool gains = a.g_post || a.g_pre;
  a.part_post = (float*)ws;
  a.part_pre = (float*)ws + (int64_t)p.grid * a.n;
  Prof prof("norm_residual_bwd", st, gains ? 2 : 1);
  const tsp_status r = p.upt == 0 ? launch<norm_residual_bwd_wide_kernel<T, Ts>, 0>(p, a, st)
                       : p.ragged ? bwd_r<T, Ts, true>(p, a, st)
                                  : bwd_r<T, Ts, false>(p, a, st);
  if (r != TSP_OK || !gains) return r;
  const bool both = a.g_post && a.g_pre;
  const float* p0 = a.g_post ? a.part_post : a.part_pre;
  float* o0 = a.g_post ? dg_post : dg_pre;
  // short rows: few columns a CTA (a 32-byte sector of each partial row), so that
  // there are CTAs enough (1001 columns, 1064 partial rows: 4 us of 31, 7 with 32
  // columns; the other way round 4096 x 304 in 4 us less)
  const int cols = a.n <= 2048 ? 8 : 32;
  return launch_after(cols == 8 ? norm_residual_gain_kernel<8> : norm_residual_gain_kernel<32>,
                      dim3((a.n + cols - 1) / cols, both ? 2 : 1), 1024, 0, st, p0, o0,
                      (const float*)a.part_pre, dg_pre, p.grid, a.n);
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
