// Layer norm over the last axis, forward and backward, with the reduction of the parameters'
// gradients (the norm in front of a transformer's linears).
//
//   forward   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps), y = (x - mu) rstd gamma + beta
//   backward  h = (x - mu) rstd, u = dy gamma:  dx = rstd (u - mean(u) - h mean(u h)),
//             dgamma = sum over rows of dy h,  dbeta = sum over rows of dy
//
// Everything is summed in fp32; y and dx are rounded once to the activation type.  x - mu is taken before
// anything is multiplied, and mu is the sum divided by D, so that a row of equal values with an exact sum
// has deviations of 0 (x rstd - mu rstd leaves the rounding of mu rstd, which is 8e-3 for 416 / sqrt(1e-5)).
// Both passes are bound by HBM: 2 (forward) and 3 (backward) activations move, at a few flops per
// byte.  A row is held in the registers of a group of threads, so that it is read once, and the
// variance is the mean of the squared deviations from the mean already known (no cancellation).
#include <mutex>

#include "common.cuh"
#include "kernels.h"

namespace poetx {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRing = 8;  // stages of a backward ring at most
constexpr int kRingBytes = 192 * 1024;  // both rings: three stages at least (16 KB rows)

// VEC elements of a row as they are stored, and their fp32 values.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC > 16 ? 16 : sizeof(T) * VEC) Vec {
  T v[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ void unpack(const Vec<T, VEC>& a, float (&f)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) f[j] = to_f32(a.v[j]);
}
__device__ __forceinline__ void unpack(const Vec<__nv_bfloat16, 8>& a, float (&f)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(&a);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float(u[j] << 16);
    f[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
  }
}
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> pack(const float (&f)[VEC]) {
  Vec<T, VEC> o;
  if constexpr (sizeof(T) == 2 && VEC == 8) {
    *reinterpret_cast<uint4*>(&o) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                               pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) o.v[j] = from_f32<T>(f[j]);
  }
  return o;
}

template <typename T, int VEC>
__device__ __forceinline__ void unpack2(const Vec<T, VEC>& a, float2 (&f)[VEC / 2]) {
  float w[VEC];
  unpack(a, w);
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) f[j] = make_float2(w[2 * j], w[2 * j + 1]);
}
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> pack2(const float2 (&f)[VEC / 2]) {
  float w[VEC];
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    w[2 * j] = f[j].x;
    w[2 * j + 1] = f[j].y;
  }
  return pack<T, VEC>(w);
}

// Sum of s[0..NS) over the TPR threads of a row group; every thread gets it.  red: one slot set
// per warp; two sets, used in turn, so that one barrier per call is enough.
template <int TPR, int NS>
__device__ __forceinline__ void group_sum(float (&s)[NS], float (*red)[kThreads / 32][2], int turn) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < NS; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  if (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5, base = warp / W * W;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < NS; ++i) red[turn & 1][warp][i] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) t += red[turn & 1][base + w][i];
      s[i] = t;
    }
  }
}

// s / D correctly rounded from inv, the rounded 1 / D: the quotient and its remainder's (Markstein,
// Computation of elementary functions on the IBM RISC System/6000, 1990).  A division in the chain of every
// row cost the many-row kernels 2-3 %, s * inv is not exact where s / D is.
__device__ __forceinline__ float row_mean(float s, float D, float inv) {
  const float q = s * inv, r = fmaf(-q, D, s);
  return r == r ? fmaf(r, inv, q) : q;  // (an infinite sum has no remainder)
}

// Few rows, or wide or odd ones (1 x 4096: 4 us, latency): a row per group of TPR threads, NV vectors of VEC
// elements per thread (NV * TPR * VEC >= D; D a multiple of VEC).
template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(kThreads)
    layernorm_fwd_kernel(const T* __restrict__ x, int N, int D, const float* __restrict__ gamma,
                         const float* __restrict__ beta, float eps, T* __restrict__ y,
                         float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int RPC = kThreads / TPR;
  __shared__ float red[2][kThreads / 32][2];
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x % TPR, nvec = D / VEC;
  const long long row = (long long)blockIdx.x * RPC + threadIdx.x / TPR;
  const bool live = row < N;  // dead groups still take part in the barriers
  const Vec<T, VEC>* xr = reinterpret_cast<const Vec<T, VEC>*>(x + row * D);
  Vec<T, VEC> a[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (live && t + i * TPR < nvec) a[i] = xr[t + i * TPR];
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (live && t + i * TPR < nvec)
#pragma unroll
      for (int j = 0; j < VEC; ++j) s[0] += to_f32(a[i].v[j]);
  group_sum<TPR>(s, red, 0);
  const float mu = s[0] / (float)D;
  s[0] = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (live && t + i * TPR < nvec)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float d = to_f32(a[i].v[j]) - mu;
        s[0] += d * d;
      }
  group_sum<TPR>(s, red, 1);
  const float rs = rsqrtf(s[0] / (float)D + eps);
  if (!live) return;
  if (t == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = rs;
  }
  Vec<T, VEC>* yr = reinterpret_cast<Vec<T, VEC>*>(y + row * D);
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (t + i * TPR < nvec) {
      const int c = (t + i * TPR) * VEC;
      Vec<T, VEC> o;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float g = gamma ? __ldg(gamma + c + j) : 1.f, b = beta ? __ldg(beta + c + j) : 0.f;
        o.v[j] = from_f32<T>((to_f32(a[i].v[j]) - mu) * rs * g + b);
      }
      yr[t + i * TPR] = o;
    }
}

// Many rows of up to 512 vectors: persistent CTAs, a warp per row (lane l holds vectors l, l + 32,
// ...), gamma and beta staged in shared memory once per CTA.  No barrier between rows, so the warps of
// an SM are at different phases of load, sums and store.  gamma and beta lie in planes of 16 bytes per
// vector (plane k: elements 4 k .. 4 k + 3 of every vector), which a warp reads without conflicts.
// 8192 x 4096 bf16: 26.8 us, 5.0 TB/s (0.75 of a plain copy's rate); bound by latency at 14 warps per
// SM, whose rows fill the registers.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kThreads, 2)
    layernorm_fwd_rows_kernel(const T* __restrict__ x, int N, int D, const float* __restrict__ gamma,
                              const float* __restrict__ beta, float eps, T* __restrict__ y,
                              float* __restrict__ mean, float* __restrict__ rstd) {
  extern __shared__ float4 gb[];  // gamma's VEC / 4 planes of nvec, beta's
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, nvec = D / VEC, warps = (int)blockDim.x / 32;
  const float inv = 1.f / (float)D;
  const long long step = (long long)gridDim.x * warps;
  long long row = (long long)blockIdx.x * warps + (threadIdx.x >> 5);
  Vec<T, VEC> a[NV];
  auto load = [&](long long r) {
    const Vec<T, VEC>* xr = reinterpret_cast<const Vec<T, VEC>*>(x + r * D);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 32 * i < nvec) a[i] = xr[lane + 32 * i];
  };
  if (row < N) load(row);  // in flight while gamma and beta are staged
  for (int q = threadIdx.x; q < D / 4; q += blockDim.x) {  // quad q: vector q / (VEC / 4)
    const int at = q % (VEC / 4) * nvec + q / (VEC / 4);
    gb[at] = gamma ? reinterpret_cast<const float4*>(gamma)[q] : make_float4(1.f, 1.f, 1.f, 1.f);
    gb[D / 4 + at] = beta ? reinterpret_cast<const float4*>(beta)[q] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  for (; row < N; row += step) {
    float p[2] = {0.f, 0.f};  // two chains
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 32 * i < nvec) {
        float f[VEC];
        unpack(a[i], f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) p[j & 1] += f[j];
      }
    float s[1] = {p[0] + p[1]};
    group_sum<32>(s, nullptr, 0);
    const float mu = row_mean(s[0], (float)D, inv);
    p[0] = p[1] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 32 * i < nvec) {
        float f[VEC];
        unpack(a[i], f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float d = f[j] - mu;
          p[j & 1] = fmaf(d, d, p[j & 1]);
        }
      }
    s[0] = p[0] + p[1];
    group_sum<32>(s, nullptr, 0);
    const float rs = rsqrtf(s[0] * inv + eps);
    if (lane == 0) {
      if (mean) mean[row] = mu;
      if (rstd) rstd[row] = rs;
    }
    Vec<T, VEC>* yr = reinterpret_cast<Vec<T, VEC>*>(y + row * D);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 32 * i < nvec) {
        float2 f[VEC / 2];
        unpack2(a[i], f);
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k) {
          const float4 g = gb[k * nvec + lane + 32 * i], b = gb[D / 4 + k * nvec + lane + 32 * i];
          float2 *lo = &f[2 * k], *hi = &f[2 * k + 1];
          *lo = fma2(mul2(add2(*lo, both(-mu)), both(rs)), make_float2(g.x, g.y), make_float2(b.x, b.y));
          *hi = fma2(mul2(add2(*hi, both(-mu)), both(rs)), make_float2(g.z, g.w), make_float2(b.z, b.w));
        }
        yr[lane + 32 * i] = pack2<T, VEC>(f);
      }
    if (row + step < N) load(row + step);
  }
}

// Rows wider than the register form takes: one CTA per row, the row read three times (from L2
// after the first).
template <typename T>
__global__ void __launch_bounds__(kThreads)
    layernorm_fwd_wide_kernel(const T* __restrict__ x, int D, const float* __restrict__ gamma,
                              const float* __restrict__ beta, float eps, T* __restrict__ y,
                              float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float red[2][kThreads / 32][2];
  pdl_trigger();
  pdl_wait();
  const long long row = blockIdx.x;
  const T* xr = x + row * D;
  float s[1] = {0.f};
  for (int c = threadIdx.x; c < D; c += kThreads) s[0] += to_f32(xr[c]);
  group_sum<kThreads>(s, red, 0);
  const float mu = s[0] / (float)D;
  s[0] = 0.f;
  for (int c = threadIdx.x; c < D; c += kThreads) {
    const float d = to_f32(xr[c]) - mu;
    s[0] += d * d;
  }
  group_sum<kThreads>(s, red, 1);
  const float rs = rsqrtf(s[0] / (float)D + eps);
  if (threadIdx.x == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = rs;
  }
  T* yr = y + row * D;
  for (int c = threadIdx.x; c < D; c += kThreads)
    yr[c] = from_f32<T>((to_f32(xr[c]) - mu) * rs * (gamma ? gamma[c] : 1.f) +
                        (beta ? beta[c] : 0.f));
}

// Backward over rows blockIdx.x * RPC + group, stepping by the grid: each thread keeps the sums of
// dy h and dy of its own columns in registers over all of its rows; the groups of a CTA are added
// in shared memory in a fixed order and the CTA writes one row of partials (pg, pb: [grid, D]).
template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(kThreads)
    layernorm_bwd_kernel(const T* __restrict__ x, const T* __restrict__ dy, int N, int D,
                         const float* __restrict__ gamma, const float* __restrict__ mean,
                         const float* __restrict__ rstd, T* __restrict__ dx,
                         float* __restrict__ pg, float* __restrict__ pb) {
  constexpr int RPC = kThreads / TPR;
  constexpr int WIDTH = RPC > 1 ? TPR * NV * VEC : 1;
  __shared__ float red[2][kThreads / 32][2];
  __shared__ float acc[RPC > 1 ? RPC : 1][WIDTH];
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR, nvec = D / VEC;
  float ag[NV][VEC], ab[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) ag[i][j] = ab[i][j] = 0.f;
  const float inv = 1.f / (float)D;
  int turn = 0;
  for (long long r0 = (long long)blockIdx.x * RPC; r0 < N; r0 += (long long)gridDim.x * RPC, ++turn) {
    const long long row = r0 + grp;
    const bool live = row < N;
    const Vec<T, VEC>* xr = reinterpret_cast<const Vec<T, VEC>*>(x + row * D);
    const Vec<T, VEC>* dr = reinterpret_cast<const Vec<T, VEC>*>(dy + row * D);
    Vec<T, VEC> a[NV], d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (live && t + i * TPR < nvec) {
        a[i] = xr[t + i * TPR];
        d[i] = dr[t + i * TPR];
      }
    const float mu = live ? mean[row] : 0.f, rs = live ? rstd[row] : 0.f;
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (live && t + i * TPR < nvec)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float h = (to_f32(a[i].v[j]) - mu) * rs, g = to_f32(d[i].v[j]);
          const float u = gamma ? g * __ldg(gamma + (t + i * TPR) * VEC + j) : g;
          s[0] += u;
          s[1] += u * h;
          ag[i][j] += g * h;
          ab[i][j] += g;
        }
    group_sum<TPR>(s, red, turn);
    const float mu_u = s[0] * inv, mu_uh = s[1] * inv;
    Vec<T, VEC>* oxr = reinterpret_cast<Vec<T, VEC>*>(dx + row * D);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (live && t + i * TPR < nvec) {
        Vec<T, VEC> o;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float h = (to_f32(a[i].v[j]) - mu) * rs, g = to_f32(d[i].v[j]);
          const float u = gamma ? g * __ldg(gamma + (t + i * TPR) * VEC + j) : g;
          o.v[j] = from_f32<T>((u - mu_u - h * mu_uh) * rs);
        }
        oxr[t + i * TPR] = o;
      }
  }
  for (int pass = 0; pass < 2; ++pass) {
    float* out = pass ? pb : pg;
    if (!out) continue;
    if (RPC == 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (t + i * TPR < nvec)
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            out[(long long)blockIdx.x * D + (t + i * TPR) * VEC + j] = pass ? ab[i][j] : ag[i][j];
    } else {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[grp][(t + i * TPR) * VEC + j] = pass ? ab[i][j] : ag[i][j];
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int g = 0; g < RPC; ++g) v += acc[g][c];
        out[(long long)blockIdx.x * D + c] = v;
      }
    }
  }
}

// The ring forms, for rows of 129 to 1024 16-byte vectors: one persistent CTA per SM of GROUPS thread
// groups (the forward: one), each on rows of its own (while one waits at its barrier another computes).  A
// group's first thread streams its rows into the group's shared-memory ring by 1-D TMA bulk copies, so that
// the next rows are in flight whatever the group does; the barrier that joins a row's sums also says that
// the row has been read, and its stage is refilled after it.  A thread owns NV vectors of every row and
// keeps what belongs to their columns in registers over all rows.
constexpr int kSite = 7 * 10000;
constexpr int kRingThreads = 512;

// Rows row0 + k stride (k < rows) of ARRAYS arrays, in the group's ring.
template <typename T, int ARRAYS>
struct RowRing {
  const T* src[ARRAYS];
  uint8_t* buf;      // [stages][ARRAYS][row]
  uint64_t* full;    // [stages]
  int stages, rows, D;
  long long row0, stride;
  int st = 0;        // stage and phase of the row being read
  uint32_t ph = 0;

  __device__ __forceinline__ uint32_t row_bytes() const { return (uint32_t)D * sizeof(T); }
  __device__ __forceinline__ const uint8_t* stage() const {
    return buf + (size_t)st * ARRAYS * row_bytes();
  }
  __device__ __forceinline__ void issue(int k, int s) {
    const long long row = row0 + k * stride;
    uint8_t* dst = buf + (size_t)s * ARRAYS * row_bytes();
    mbar_arrive_expect_tx(&full[s], ARRAYS * row_bytes());
#pragma unroll
    for (int a = 0; a < ARRAYS; ++a)
      bulk_load(dst + a * row_bytes(), src[a] + row * D, row_bytes(), &full[s]);
  }
  __device__ __forceinline__ void start() {
    for (int k = 0; k < rows && k < stages; ++k) issue(k, k);
  }
  __device__ __forceinline__ int before() const { return st ? st - 1 : stages - 1; }
  __device__ __forceinline__ void refill(int k, int s) {  // row k, in stage s, has been read by all
    if (k + stages < rows) issue(k + stages, s);
  }
  __device__ __forceinline__ void next() {
    if (++st == stages) {
      st = 0;
      ph ^= 1;
    }
  }
  // no copy may be in flight when the CTA exits (passes at once but after a timeout)
  __device__ __forceinline__ void drain(int* err, unsigned long long limit_ns) {
    for (int k = rows > stages ? rows - stages : 0; k < rows; ++k)
      mbar_wait_bounded(&full[k % stages], (uint32_t)((k / stages) & 1), err, limit_ns,
                        kSite + __LINE__);
  }
};

// Sum of v over the warps of a group (at most 16), through red; one barrier.
__device__ __forceinline__ float2 ring_join(float2 v, float2* red, int warp, int lane, int warps,
                                            int barrier, int threads) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o),
                            __shfl_xor_sync(0xffffffffu, v.y, o)));
  if (lane == 0) red[warp] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(threads) : "memory");
  v = (lane & 15) < warps ? red[lane & 15] : make_float2(0.f, 0.f);
#pragma unroll
  for (int o = 8; o; o >>= 1)
    v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o),
                            __shfl_xor_sync(0xffffffffu, v.y, o)));
  return v;
}

__device__ __forceinline__ float4 ring_join4(float4 v, float4* red, int warp, int lane, int warps,
                                             int barrier, int threads) {
  auto step = [&](int o) {
    const float2 a = add2(make_float2(v.x, v.y), make_float2(__shfl_xor_sync(0xffffffffu, v.x, o),
                                                             __shfl_xor_sync(0xffffffffu, v.y, o)));
    const float2 b = add2(make_float2(v.z, v.w), make_float2(__shfl_xor_sync(0xffffffffu, v.z, o),
                                                             __shfl_xor_sync(0xffffffffu, v.w, o)));
    v = make_float4(a.x, a.y, b.x, b.y);
  };
#pragma unroll
  for (int o = 16; o; o >>= 1) step(o);
  if (lane == 0) red[warp] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(threads) : "memory");
  v = (lane & 15) < warps ? red[lane & 15] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int o = 8; o; o >>= 1) step(o);
  return v;
}

// Forward, for many rows of more vectors than a warp's registers hold (513 to 1024): one group, two vectors
// per thread, gamma and beta of the thread's columns in registers; two joins for two rows (the means, then
// the squared deviations from them).
// 4096 x 8192 bf16: 28.0 us, 4.8 TB/s (32.0 us without the bound of one CTA per SM, which the ring's memory
// sets: the compiler then keeps to fewer registers).
template <typename T>
__global__ void __launch_bounds__(kRingThreads, 1)
    layernorm_fwd_ring_kernel(const T* __restrict__ x, int N, int D, const float* __restrict__ gamma,
                              const float* __restrict__ beta, float eps, T* __restrict__ y,
                              float* __restrict__ mean, float* __restrict__ rstd, int stages,
                              int* err, unsigned long long limit_ns) {
  constexpr int VEC = 16 / sizeof(T), H = VEC / 2, NV = 2;
  extern __shared__ __align__(128) uint8_t ring_mem[];
  __shared__ uint64_t full[kMaxRing];
  __shared__ float2 red[2][kRingThreads / 32];
  const int threads = (int)blockDim.x, warps = threads / 32;
  const int t = (int)threadIdx.x, warp = t >> 5, lane = t & 31;
  pdl_trigger();
  if (t == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  const long long row0 = blockIdx.x, stride = gridDim.x;
  const int rows = row0 < N ? (int)((N - 1 - row0) / stride) + 1 : 0;
  RowRing<T, 1> ring{{x}, ring_mem, full, stages, rows, D, row0, stride};
  if (t == 0) ring.start();
  const int nvec = D / VEC;
  float2 gm[NV][H], bt[NV][H];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < H; ++j) {
      const int c = (t + i * threads) * VEC + 2 * j;
      const bool in = t + i * threads < nvec;
      gm[i][j] = in && gamma ? make_float2(gamma[c], gamma[c + 1]) : both(1.f);
      bt[i][j] = in && beta ? make_float2(beta[c], beta[c + 1]) : both(0.f);
    }
  const float inv = 1.f / (float)D;
  bool ok = true;  // after an expired wait: no more waits, but every barrier
  for (int k = 0; k < rows; k += 2) {
    // rows k and k + 1, one in each half of the joins (the last may be alone: its partner repeats it)
    const bool two = k + 1 < rows;
    const long long row[2] = {row0 + k * stride, row0 + (k + two) * stride};
    float2 h[2][NV][H], s[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      ok = ok && mbar_wait_bounded(&full[ring.st], ring.ph, err, limit_ns, kSite + __LINE__);
      const Vec<T, VEC>* xr = reinterpret_cast<const Vec<T, VEC>*>(ring.stage());
      s[r] = both(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (t + i * threads < nvec) {
          unpack2(xr[t + i * threads], h[r][i]);
#pragma unroll
          for (int j = 0; j < H; ++j) s[r] = add2(s[r], h[r][i][j]);
        }
      if (r == 0 && two) ring.next();
    }
    float2 w = ring_join(make_float2(s[0].x + s[0].y, s[1].x + s[1].y), red[0], warp, lane, warps, 1,
                         threads);
    if (t == 0) {
      if (two) ring.refill(k, ring.before());
      ring.refill(k + two, ring.st);
    }
    ring.next();
    const float mu[2] = {row_mean(w.x, (float)D, inv), row_mean(w.y, (float)D, inv)};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      s[r] = both(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (t + i * threads < nvec)
#pragma unroll
          for (int j = 0; j < H; ++j) {
            h[r][i][j] = add2(h[r][i][j], both(-mu[r]));
            s[r] = fma2(h[r][i][j], h[r][i][j], s[r]);
          }
    }
    w = ring_join(make_float2(s[0].x + s[0].y, s[1].x + s[1].y), red[1], warp, lane, warps, 1, threads);
    const float rs[2] = {rsqrtf(w.x * inv + eps), rsqrtf(w.y * inv + eps)};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (r == 1 && !two) break;
      if (t == 0) {
        if (mean) mean[row[r]] = mu[r];
        if (rstd) rstd[row[r]] = rs[r];
      }
      Vec<T, VEC>* o = reinterpret_cast<Vec<T, VEC>*>(y + row[r] * D);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (t + i * threads < nvec) {
#pragma unroll
          for (int j = 0; j < H; ++j)
            h[r][i][j] = fma2(mul2(h[r][i][j], both(rs[r])), gm[i][j], bt[i][j]);
          o[t + i * threads] = pack2<T, VEC>(h[r][i]);
        }
    }
  }
  if (t == 0) ring.drain(err, limit_ns);
}

// Backward: a thread keeps gamma and the sums of dy h and dy of its columns; one join for two rows.  At
// the end the groups' sums are added through shared memory, so that there is one row of partials per SM.
// 8192 x 4096 bf16: 40.5 us with the reduction, 5.0 TB/s; without its loads and stores it takes three
// quarters of that (some 340 instructions per warp and row, and the join's chain).
template <typename T, int NV, int GROUPS>
__global__ void __launch_bounds__(kRingThreads)
    layernorm_bwd_ring_kernel(const T* __restrict__ x, const T* __restrict__ dy, int N, int D,
                              const float* __restrict__ gamma, const float* __restrict__ mean,
                              const float* __restrict__ rstd, T* __restrict__ dx,
                              float* __restrict__ pg, float* __restrict__ pb, int stages, int* err,
                              unsigned long long limit_ns) {
  constexpr int VEC = 16 / sizeof(T), H = VEC / 2;
  extern __shared__ __align__(128) uint8_t ring_mem[];
  __shared__ uint64_t full[GROUPS][kMaxRing];
  __shared__ float4 red[GROUPS][2][kRingThreads / 32 / GROUPS];
  const int threads = (int)blockDim.x / GROUPS, warps = threads / 32;
  const int grp = (int)threadIdx.x / threads, t = (int)threadIdx.x - grp * threads;
  const int warp = t >> 5, lane = t & 31;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int g = 0; g < GROUPS; ++g)
      for (int i = 0; i < stages; ++i) mbar_init(&full[g][i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  const long long row0 = blockIdx.x + (long long)grp * gridDim.x;
  const long long stride = (long long)gridDim.x * GROUPS;
  const int rows = row0 < N ? (int)((N - 1 - row0) / stride) + 1 : 0;
  RowRing<T, 2> ring{{x, dy}, ring_mem + (size_t)grp * stages * 2 * D * sizeof(T), full[grp], stages,
                     rows, D, row0, stride};
  if (t == 0) ring.start();
  const int nvec = D / VEC;
  float2 ag[NV][H], ab[NV][H], gm[NV][H];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < H; ++j) {
      ag[i][j] = ab[i][j] = both(0.f);
      const int c = (t + i * threads) * VEC + 2 * j;
      gm[i][j] = t + i * threads < nvec && gamma ? make_float2(gamma[c], gamma[c + 1]) : both(1.f);
    }
  const float inv = 1.f / (float)D;
  // mean and rstd are read two rows ahead
  float2 mu_next = both(0.f), rs_next = both(0.f);
  auto stats = [&](int k) {
    if (k < rows) {
      const long long r0 = row0 + k * stride, r1 = k + 1 < rows ? r0 + stride : r0;
      mu_next = make_float2(mean[r0], mean[r1]);
      rs_next = make_float2(rstd[r0], rstd[r1]);
    }
  };
  stats(0);
  bool ok = true;  // after an expired wait: no more waits, but every barrier
  for (int k = 0; k < rows; k += 2) {
    // rows k and k + 1, their sums in one join (the last may be alone)
    const bool two = k + 1 < rows;
    const long long row[2] = {row0 + k * stride, row0 + (k + two) * stride};
    const float mu[2] = {mu_next.x, mu_next.y}, rs[2] = {rs_next.x, rs_next.y};
    stats(k + 2);
    // the rows stay packed between the two passes over them (unpacking twice is cheaper than the
    // registers of both rows' h and u)
    Vec<T, VEC> xv[2][NV], dv[2][NV];
    float2 s0[2] = {both(0.f), both(0.f)}, s1[2] = {both(0.f), both(0.f)};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (r == 1 && !two) break;
      if (r == 1) ring.next();
      ok = ok && mbar_wait_bounded(&full[grp][ring.st], ring.ph, err, limit_ns, kSite + __LINE__);
      const Vec<T, VEC>* xr = reinterpret_cast<const Vec<T, VEC>*>(ring.stage());
      const Vec<T, VEC>* dr = reinterpret_cast<const Vec<T, VEC>*>(ring.stage() + ring.row_bytes());
      const float2 rs2 = both(rs[r]), nmu = both(-mu[r]);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (t + i * threads < nvec) {
          xv[r][i] = xr[t + i * threads];
          dv[r][i] = dr[t + i * threads];
          float2 h[H], u[H];
          unpack2(xv[r][i], h);
          unpack2(dv[r][i], u);
#pragma unroll
          for (int j = 0; j < H; ++j) {
            h[j] = mul2(add2(h[j], nmu), rs2);
            ag[i][j] = fma2(u[j], h[j], ag[i][j]);
            ab[i][j] = add2(ab[i][j], u[j]);
            u[j] = mul2(u[j], gm[i][j]);
            s0[r] = add2(s0[r], u[j]);
            s1[r] = fma2(u[j], h[j], s1[r]);
          }
        }
    }
    const float4 w = ring_join4(make_float4(s0[0].x + s0[0].y, s1[0].x + s1[0].y, s0[1].x + s0[1].y,
                                            s1[1].x + s1[1].y),
                                red[grp][k >> 1 & 1], warp, lane, warps, 1 + grp, threads);
    if (t == 0) {
      if (two) ring.refill(k, ring.before());
      ring.refill(k + two, ring.st);
    }
    ring.next();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (r == 1 && !two) break;
      // dx = dy (gamma rs) + ((x - mu) rs c1 + c0),  c0 = -rs mean(u), c1 = -rs mean(u h)
      const float c0 = -(r ? w.z : w.x) * inv * rs[r], c1 = -(r ? w.w : w.y) * inv * rs[r];
      const float2 rs2 = both(rs[r]), nmu = both(-mu[r]), kx = both(rs[r] * c1), k0 = both(c0);
      Vec<T, VEC>* o = reinterpret_cast<Vec<T, VEC>*>(dx + row[r] * D);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (t + i * threads < nvec) {
          float2 a[H], d[H];
          unpack2(xv[r][i], a);
          unpack2(dv[r][i], d);
#pragma unroll
          for (int j = 0; j < H; ++j)
            d[j] = fma2(d[j], mul2(gm[i][j], rs2), fma2(add2(a[j], nmu), kx, k0));
          o[t + i * threads] = pack2<T, VEC>(d);
        }
    }
  }
  if (t == 0) ring.drain(err, limit_ns);
  if (GROUPS > 1) {  // the second group's sums through the ring's memory: dgamma [D], dbeta [D]
    static_assert(GROUPS <= 2, "two groups are added");
    float2* sums = reinterpret_cast<float2*>(ring_mem);
    __syncthreads();
    if (grp == 1)
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (t + i * threads < nvec)
#pragma unroll
          for (int j = 0; j < H; ++j) {
            sums[(t + i * threads) * H + j] = ag[i][j];
            sums[D / 2 + (t + i * threads) * H + j] = ab[i][j];
          }
    __syncthreads();
    if (grp == 1) return;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (t + i * threads < nvec)
#pragma unroll
        for (int j = 0; j < H; ++j) {
          ag[i][j] = add2(ag[i][j], sums[(t + i * threads) * H + j]);
          ab[i][j] = add2(ab[i][j], sums[D / 2 + (t + i * threads) * H + j]);
        }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (t + i * threads < nvec) {
      const long long at = (long long)blockIdx.x * D + (t + i * threads) * VEC;
      if (pg) *reinterpret_cast<Vec<float, VEC>*>(pg + at) = pack2<float, VEC>(ag[i]);
      if (pb) *reinterpret_cast<Vec<float, VEC>*>(pb + at) = pack2<float, VEC>(ab[i]);
    }
}

// dx of rows wider than the register form takes: one CTA per row, x and dy read twice.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    layernorm_bwd_wide_kernel(const T* __restrict__ x, const T* __restrict__ dy, int D,
                              const float* __restrict__ gamma, const float* __restrict__ mean,
                              const float* __restrict__ rstd, T* __restrict__ dx) {
  __shared__ float red[2][kThreads / 32][2];
  pdl_trigger();
  pdl_wait();
  const long long row = blockIdx.x;
  const T *xr = x + row * D, *dr = dy + row * D;
  const float mu = mean[row], rs = rstd[row];
  float s[2] = {0.f, 0.f};
  for (int c = threadIdx.x; c < D; c += kThreads) {
    const float u = to_f32(dr[c]) * (gamma ? gamma[c] : 1.f);
    s[0] += u;
    s[1] += u * (to_f32(xr[c]) - mu) * rs;
  }
  group_sum<kThreads>(s, red, 0);
  const float inv = 1.f / (float)D;
  for (int c = threadIdx.x; c < D; c += kThreads) {
    const float u = to_f32(dr[c]) * (gamma ? gamma[c] : 1.f);
    dx[row * D + c] = from_f32<T>((u - s[0] * inv - (to_f32(xr[c]) - mu) * rs * s[1] * inv) * rs);
  }
}

// Partials of the parameters' gradients for wide rows: a thread per column, CTA row blockIdx.y
// takes rows blockIdx.y, + gridDim.y, ...
template <typename T>
__global__ void __launch_bounds__(kThreads)
    layernorm_param_kernel(const T* __restrict__ x, const T* __restrict__ dy, int N, int D,
                           const float* __restrict__ mean, const float* __restrict__ rstd,
                           float* __restrict__ pg, float* __restrict__ pb) {
  pdl_trigger();
  pdl_wait();
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= D) return;
  float g = 0.f, b = 0.f;
  for (long long row = blockIdx.y; row < N; row += gridDim.y) {
    const float d = to_f32(dy[row * D + c]);
    g += d * (to_f32(x[row * D + c]) - mean[row]) * rstd[row];
    b += d;
  }
  if (pg) pg[(long long)blockIdx.y * D + c] = g;
  if (pb) pb[(long long)blockIdx.y * D + c] = b;
}

// out[c] (+)= sum over P partial rows, in a fixed order: 32 columns x 32 row lanes per CTA (P is at
// most two per SM: some ten loads per thread, all in flight).
constexpr int kReduceLanes = 32;
__global__ void __launch_bounds__(32 * kReduceLanes)
    layernorm_reduce_kernel(const float* __restrict__ pg, const float* __restrict__ pb, int P, int D,
                            float* __restrict__ dgamma, float* __restrict__ dbeta, int accumulate) {
  __shared__ float part[kReduceLanes][33];
  pdl_trigger();
  pdl_wait();
  const float* src = blockIdx.y ? pb : pg;
  float* dst = blockIdx.y ? dbeta : dgamma;
  if (!dst) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < D) {
#pragma unroll 5
    for (int r = w; r < P; r += kReduceLanes) v += src[(long long)r * D + c];
  }
  part[w][lane] = v;
  __syncthreads();
  v = part[lane][w];  // column w of the CTA
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int k = blockIdx.x * 32 + w;
  if (lane == 0 && k < D) dst[k] = accumulate ? dst[k] + v : v;
}

// The register forms: threads per row and vectors per thread by the row's vectors.  The vectors
// are 16 bytes where the row is a multiple of that, else single elements.
struct NormShape {
  int vec, tpr, nv;  // nv 0: the wide form
};
NormShape norm_shape(size_t esize, int D) {
  const int vec = (int)((size_t)D * esize % 16 == 0 ? 16 / esize : 1);
  const int nvec = D / vec;
  if (nvec <= 32 * 4) return {vec, 32, 4};
  if (nvec <= 256 * 2) return {vec, 256, 2};
  if (nvec <= 256 * 4) return {vec, 256, 4};
  if (nvec <= 256 * 8 && vec < 8) return {vec, 256, 8};
  return {vec, 0, 0};
}

// The ring forms: rows of 129 to 1024 16-byte vectors.
bool ring_rows(const NormShape& f, int D) { return f.vec > 1 && D / f.vec > 128 && D / f.vec <= 1024; }
// Its groups and the vectors per thread: two groups of up to 256 threads with one or two vectors, or
// one of up to 512 with two (more would not fit the 128 registers of a thread).
struct RingShape {
  int groups, nv, threads;  // threads of a group
};
RingShape ring_shape(int nvec) {
  const int groups = nvec <= 512 ? 2 : 1, nv = nvec <= 256 ? 1 : 2;
  return {groups, nv, ((nvec + nv - 1) / nv + 31) / 32 * 32};
}

// Backward CTAs (= rows of partials): one (ring form) or two per SM, no more than there are rows
// or row groups.
int norm_bwd_parts(long long N, const NormShape& f, int D) {
  const bool ring = ring_rows(f, D);
  const long long rpc = f.nv && !ring ? kThreads / f.tpr : 1;
  const long long want = (N + rpc - 1) / rpc;
  const long long cap = (ring ? 1LL : 2LL) * sm_count();
  return (int)(want < cap ? (want > 0 ? want : 1) : cap);
}

template <typename T, int VEC, int TPR, int NV>
cudaError_t fwd_launch(const void* x, int N, int D, const float* gamma, const float* beta, float eps,
                       void* y, float* mean, float* rstd, cudaStream_t s) {
  const int rpc = kThreads / TPR;
  return launch_pdl(layernorm_fwd_kernel<T, VEC, TPR, NV>, dim3((unsigned)(((long long)N + rpc - 1) / rpc)),
                    dim3(kThreads),
                    0, s, static_cast<const T*>(x), N, D, gamma, beta, eps, static_cast<T*>(y), mean,
                    rstd);
}

// Two CTAs per SM of 5 to 8 warps: of these the count whose last round over the rows is fullest
// (8192 rows: 7 warps, four rounds at 96 %; 8 warps would leave the fourth at 37 %).
template <typename T, int VEC, int NV>
cudaError_t fwd_rows(const void* x, int N, int D, const float* gamma, const float* beta, float eps,
                     void* y, float* mean, float* rstd, cudaStream_t s) {
  const long long ctas = 2LL * sm_count();
  int warps = 8;
  double fill = 0;
  for (int w = 8; w >= 5; --w) {
    const long long at_once = ctas * w;
    const double f = (double)N / (double)((N + at_once - 1) / at_once * at_once);
    if (f > fill + 1e-9) {
      fill = f;
      warps = w;
    }
  }
  const long long want = ((long long)N + warps - 1) / warps;
  return launch_pdl(layernorm_fwd_rows_kernel<T, VEC, NV>, dim3((unsigned)(want < ctas ? want : ctas)),
                    dim3(32 * warps), (size_t)D * 8, s, static_cast<const T*>(x), N, D, gamma, beta,
                    eps, static_cast<T*>(y), mean, rstd);
}

// Stages of a group's ring for `bytes` per stage, and the shared memory of all rings.
int ring_stages(size_t bytes, int groups) {
  const int n = (int)((size_t)kRingBytes / (groups * bytes));
  return n < kMaxRing ? n : kMaxRing;
}
template <typename K>
cudaError_t ring_attr(K k) {
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
}

template <typename T>
cudaError_t fwd_ring(const void* x, int N, int D, const float* gamma, const float* beta, float eps,
                     void* y, float* mean, float* rstd, cudaStream_t s) {
  const size_t stage = (size_t)D * sizeof(T);
  const int threads = ring_shape(D / (16 / (int)sizeof(T))).threads;
  const int stages = ring_stages(stage, 1);
  auto k = layernorm_fwd_ring_kernel<T>;
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [&] { attr = ring_attr(k); });
  if (attr != cudaSuccess) return attr;
  return launch_pdl(k, dim3(N < sm_count() ? N : sm_count()), dim3(threads), stages * stage, s,
                    static_cast<const T*>(x), N, D, gamma, beta, eps, static_cast<T*>(y), mean, rstd,
                    stages, device_error_word(), kWaitLimitNs);
}

template <typename T, int NV, int GROUPS>
cudaError_t bwd_ring_launch(const void* x, const void* dy, int N, int D, const float* gamma,
                            const float* mean, const float* rstd, void* dx, float* pg, float* pb,
                            int parts, cudaStream_t s) {
  const size_t stage = 2 * (size_t)D * sizeof(T);
  const int threads = ring_shape(D / (16 / (int)sizeof(T))).threads;
  const int stages = ring_stages(stage, GROUPS);
  auto k = layernorm_bwd_ring_kernel<T, NV, GROUPS>;
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [&] { attr = ring_attr(k); });
  if (attr != cudaSuccess) return attr;
  return launch_pdl(k, dim3(parts), dim3(GROUPS * threads), GROUPS * stages * stage, s,
                    static_cast<const T*>(x), static_cast<const T*>(dy), N, D, gamma, mean, rstd,
                    static_cast<T*>(dx), pg, pb, stages, device_error_word(), kWaitLimitNs);
}

template <typename T, int VEC>
cudaError_t fwd_pick(const NormShape& f, const void* x, int N, int D, const float* gamma,
                     const float* beta, float eps, void* y, float* mean, float* rstd,
                     cudaStream_t s) {
  // from a few rows per SM on: a warp per row, or the ring for the rows that a warp's registers do
  // not hold (at 8192 x 4096 the ring takes 35 us, a warp per row 27)
  if constexpr (VEC > 1) {
    const int nvec = D / VEC;
    if (N >= 8 * sm_count()) {
      if (nvec <= 128) return fwd_rows<T, VEC, 4>(x, N, D, gamma, beta, eps, y, mean, rstd, s);
      if (nvec <= 256) return fwd_rows<T, VEC, 8>(x, N, D, gamma, beta, eps, y, mean, rstd, s);
      if (nvec <= 512) return fwd_rows<T, VEC, 16>(x, N, D, gamma, beta, eps, y, mean, rstd, s);
      if (ring_rows(f, D)) return fwd_ring<T>(x, N, D, gamma, beta, eps, y, mean, rstd, s);
    }
  }
  if (f.tpr == 32) return fwd_launch<T, VEC, 32, 4>(x, N, D, gamma, beta, eps, y, mean, rstd, s);
  if (f.nv == 2) return fwd_launch<T, VEC, 256, 2>(x, N, D, gamma, beta, eps, y, mean, rstd, s);
  if (f.nv == 4) return fwd_launch<T, VEC, 256, 4>(x, N, D, gamma, beta, eps, y, mean, rstd, s);
  if (VEC < 8 && f.nv == 8)
    return fwd_launch<T, VEC < 8 ? VEC : 1, 256, 8>(x, N, D, gamma, beta, eps, y, mean, rstd, s);
  return launch_pdl(layernorm_fwd_wide_kernel<T>, dim3(N), dim3(kThreads), 0, s,
                    static_cast<const T*>(x), D, gamma, beta, eps, static_cast<T*>(y), mean, rstd);
}

template <typename T, int VEC, int TPR, int NV>
cudaError_t bwd_launch(const void* x, const void* dy, int N, int D, const float* gamma,
                       const float* mean, const float* rstd, void* dx, float* pg, float* pb,
                       int parts, cudaStream_t s) {
  return launch_pdl(layernorm_bwd_kernel<T, VEC, TPR, NV>, dim3(parts), dim3(kThreads), 0, s,
                    static_cast<const T*>(x), static_cast<const T*>(dy), N, D, gamma, mean, rstd,
                    static_cast<T*>(dx), pg, pb);
}

template <typename T, int VEC>
cudaError_t bwd_pick(const NormShape& f, const void* x, const void* dy, int N, int D,
                     const float* gamma, const float* mean, const float* rstd, void* dx, float* pg,
                     float* pb, int parts, cudaStream_t s) {
  if constexpr (VEC > 1) {
    if (ring_rows(f, D)) {
      const RingShape r = ring_shape(D / VEC);
      if (r.groups == 1)
        return bwd_ring_launch<T, 2, 1>(x, dy, N, D, gamma, mean, rstd, dx, pg, pb, parts, s);
      if (r.nv == 2)
        return bwd_ring_launch<T, 2, 2>(x, dy, N, D, gamma, mean, rstd, dx, pg, pb, parts, s);
      return bwd_ring_launch<T, 1, 2>(x, dy, N, D, gamma, mean, rstd, dx, pg, pb, parts, s);
    }
  }
  if (f.tpr == 32)
    return bwd_launch<T, VEC, 32, 4>(x, dy, N, D, gamma, mean, rstd, dx, pg, pb, parts, s);
  // the wider register forms are reached by element vectors only
  if (VEC == 1 && f.nv == 2)
    return bwd_launch<T, 1, 256, 2>(x, dy, N, D, gamma, mean, rstd, dx, pg, pb, parts, s);
  if (VEC == 1 && f.nv == 4)
    return bwd_launch<T, 1, 256, 4>(x, dy, N, D, gamma, mean, rstd, dx, pg, pb, parts, s);
  if (VEC == 1 && f.nv == 8)
    return bwd_launch<T, 1, 256, 8>(x, dy, N, D, gamma, mean, rstd, dx, pg, pb, parts, s);
  cudaError_t e = launch_pdl(layernorm_bwd_wide_kernel<T>, dim3(N), dim3(kThreads), 0, s,
                             static_cast<const T*>(x), static_cast<const T*>(dy), D, gamma, mean,
                             rstd, static_cast<T*>(dx));
  if (e != cudaSuccess || (!pg && !pb)) return e;
  after_launch(s, ST_NORM);
  return launch_pdl(layernorm_param_kernel<T>, dim3((D + kThreads - 1) / kThreads, parts),
                    dim3(kThreads), 0, s, static_cast<const T*>(x), static_cast<const T*>(dy), N, D,
                    mean, rstd, pg, pb);
}

bool norm_dtype(poetx_dtype dt) { return dt == POETX_F32 || dt == POETX_BF16; }

}  // namespace
}  // namespace poetx

using namespace poetx;

extern "C" poetx_status poetx_layernorm_fwd(poetx_dtype dt, const void* x, int N, int D,
                                            const float* gamma, const float* beta, float eps,
                                            void* y, float* mean, float* rstd, cudaStream_t stream) {
  if (N < 0 || D < 1 || !(eps >= 0.f)) return POETX_ERR_ARG;
  if (!norm_dtype(dt)) return POETX_ERR_DTYPE;
  if (N == 0) return POETX_OK;
  if (!x || !y) return POETX_ERR_ARG;
  if (!aligned16(x) || !aligned16(y) || !aligned16(gamma) || !aligned16(beta) || !aligned16(mean) ||
      !aligned16(rstd))
    return POETX_ERR_ALIGN;
  const NormShape f = norm_shape(dtype_size(dt), D);
  cudaError_t e;
  if (dt == POETX_BF16)
    e = f.vec == 8 ? fwd_pick<__nv_bfloat16, 8>(f, x, N, D, gamma, beta, eps, y, mean, rstd, stream)
                   : fwd_pick<__nv_bfloat16, 1>(f, x, N, D, gamma, beta, eps, y, mean, rstd, stream);
  else
    e = f.vec == 4 ? fwd_pick<float, 4>(f, x, N, D, gamma, beta, eps, y, mean, rstd, stream)
                   : fwd_pick<float, 1>(f, x, N, D, gamma, beta, eps, y, mean, rstd, stream);
  POETX_CUDA_TRY(e);
  POETX_CUDA_TRY(cudaGetLastError());
  after_launch(stream, ST_NORM);
  return POETX_OK;
}

extern "C" size_t poetx_layernorm_bwd_workspace_bytes(poetx_dtype dt, int N, int D) {
  if (N < 0 || D < 1 || !norm_dtype(dt)) return 0;
  const int parts = norm_bwd_parts(N, norm_shape(dtype_size(dt), D), D);
  return 2 * align_up((size_t)parts * D * sizeof(float), 256);
}

extern "C" poetx_status poetx_layernorm_bwd(poetx_dtype dt, const void* x, const void* dy, int N,
                                            int D, const float* gamma, const float* mean,
                                            const float* rstd, void* dx, float* dgamma, float* dbeta,
                                            int accumulate, void* ws, size_t ws_bytes,
                                            cudaStream_t stream) {
  if (N < 0 || D < 1) return POETX_ERR_ARG;
  if (!norm_dtype(dt)) return POETX_ERR_DTYPE;
  if (!aligned16(x) || !aligned16(dy) || !aligned16(gamma) || !aligned16(mean) || !aligned16(rstd) ||
      !aligned16(dx) || !aligned16(dgamma) || !aligned16(dbeta) || !aligned16(ws))
    return POETX_ERR_ALIGN;
  if (N == 0) {
    if (!accumulate) {
      if (dgamma) POETX_CUDA_TRY(cudaMemsetAsync(dgamma, 0, (size_t)D * 4, stream));
      if (dbeta) POETX_CUDA_TRY(cudaMemsetAsync(dbeta, 0, (size_t)D * 4, stream));
    }
    return POETX_OK;
  }
  if (!x || !dy || !mean || !rstd || !dx) return POETX_ERR_ARG;
  const bool params = dgamma || dbeta;
  const size_t need = poetx_layernorm_bwd_workspace_bytes(dt, N, D);
  if (params && !ws) return POETX_ERR_ARG;
  if (params && ws_bytes < need) return POETX_ERR_WORKSPACE;
  const NormShape f = norm_shape(dtype_size(dt), D);
  const int parts = norm_bwd_parts(N, f, D);
  float* pg = dgamma ? static_cast<float*>(ws) : nullptr;
  float* pb = dbeta ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + need / 2) : nullptr;
  cudaError_t e;
  if (dt == POETX_BF16)
    e = f.vec == 8
            ? bwd_pick<__nv_bfloat16, 8>(f, x, dy, N, D, gamma, mean, rstd, dx, pg, pb, parts, stream)
            : bwd_pick<__nv_bfloat16, 1>(f, x, dy, N, D, gamma, mean, rstd, dx, pg, pb, parts, stream);
  else
    e = f.vec == 4 ? bwd_pick<float, 4>(f, x, dy, N, D, gamma, mean, rstd, dx, pg, pb, parts, stream)
                   : bwd_pick<float, 1>(f, x, dy, N, D, gamma, mean, rstd, dx, pg, pb, parts, stream);
  POETX_CUDA_TRY(e);
  POETX_CUDA_TRY(cudaGetLastError());
  after_launch(stream, ST_NORM);
  if (params) {
    POETX_CUDA_TRY(launch_pdl(layernorm_reduce_kernel, dim3((D + 31) / 32, 2),
                              dim3(32 * kReduceLanes), 0,
                              stream, (const float*)pg, (const float*)pb, parts, D, dgamma, dbeta,
                              accumulate));
    POETX_CUDA_TRY(cudaGetLastError());
    after_launch(stream, ST_NORM);
  }
  return POETX_OK;
}
