// Layer norm over the last axis, forward and backward, with the reduction of the parameters'
// gradients (the norm in front of a transformer's linears).
//
//   forward   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps), y = (x - mu) rstd gamma + beta
//   backward  h = (x - mu) rstd, u = dy gamma:  dx = rstd (u - mean(u) - h mean(u h)),
//             dgamma = sum over rows of dy h,  dbeta = sum over rows of dy
//
// Everything is summed in fp32; y and dx are rounded once to the activation type.
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

// Few rows, or wide ones: a row per group of TPR threads, NV vectors of VEC elements per thread
// (NV * TPR * VEC >= D; D a multiple of VEC).
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
  const float rs = 1.f / sqrtf(s[0] / (float)D + eps);
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

// Many rows: persistent CTAs, a warp per row (lane l holds vectors l, l + 32, ...), gamma and beta
// staged in shared memory once per CTA.  No barrier between rows, so the warps of an SM are at
// different phases of load, sums and store.  Two CTAs per SM: 16 rows in flight (more registers
// per thread, one CTA: 2.2 times as long at 8192 x 4096).
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kThreads, 2)
    layernorm_fwd_rows_kernel(const T* __restrict__ x, int N, int D, const float* __restrict__ gamma,
                              const float* __restrict__ beta, float eps, T* __restrict__ y,
                              float* __restrict__ mean, float* __restrict__ rstd) {
  extern __shared__ float gb[];  // gamma [D], beta [D]
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, nvec = D / VEC;
  const float inv = 1.f / (float)D;
  const long long step = (long long)gridDim.x * (kThreads / 32);
  long long row = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  Vec<T, VEC> a[NV];
  auto load = [&](long long r) {
    const Vec<T, VEC>* xr = reinterpret_cast<const Vec<T, VEC>*>(x + r * D);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 32 * i < nvec) a[i] = xr[lane + 32 * i];
  };
  if (row < N) load(row);  // in flight while gamma and beta are staged
  for (int c = threadIdx.x; c < D; c += kThreads) {
    gb[c] = gamma ? gamma[c] : 1.f;
    gb[D + c] = beta ? beta[c] : 0.f;
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
    const float mu = s[0] * inv;
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
    const float rs = 1.f / sqrtf(s[0] * inv + eps);
    if (lane == 0) {
      if (mean) mean[row] = mu;
      if (rstd) rstd[row] = rs;
    }
    Vec<T, VEC>* yr = reinterpret_cast<Vec<T, VEC>*>(y + row * D);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 32 * i < nvec) {
        const Vec<float, VEC> g = reinterpret_cast<const Vec<float, VEC>*>(gb)[lane + 32 * i];
        const Vec<float, VEC> b = reinterpret_cast<const Vec<float, VEC>*>(gb + D)[lane + 32 * i];
        float f[VEC];
        unpack(a[i], f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] = fmaf((f[j] - mu) * rs, g.v[j], b.v[j]);
        yr[lane + 32 * i] = pack<T, VEC>(f);
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
  const float rs = 1.f / sqrtf(s[0] / (float)D + eps);
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

// Backward of rows of 129 to 1024 16-byte vectors: one persistent CTA per SM of GROUPS thread groups,
// each on rows of its own (while one waits at its barrier another computes).  A group's first thread
// streams its rows of x and dy into the group's shared-memory ring by 1-D TMA bulk copies, so that
// the next rows are in flight whatever the group does; the barrier that joins a row's two sums also
// says that the row has been read, and its stage is refilled after it.  A thread keeps gamma and the
// sums of dy h and dy of its NV vectors in registers over all rows.  At the end the groups' sums are
// added through shared memory, so that there is one row of partials per SM.
constexpr int kSite = 7 * 10000;
constexpr int kRingThreads = 512;

template <typename T, int NV, int GROUPS>
__global__ void __launch_bounds__(kRingThreads)
    layernorm_bwd_ring_kernel(const T* __restrict__ x, const T* __restrict__ dy, int N, int D,
                              const float* __restrict__ gamma, const float* __restrict__ mean,
                              const float* __restrict__ rstd, T* __restrict__ dx,
                              float* __restrict__ pg, float* __restrict__ pb, int stages, int* err,
                              unsigned long long limit_ns) {
  constexpr int VEC = 16 / sizeof(T);
  constexpr int MAXW = kRingThreads / 32 / GROUPS;  // warps of a group
  extern __shared__ __align__(128) uint8_t ring[];  // [GROUPS][stages][x row, dy row]
  __shared__ uint64_t full[GROUPS][kMaxRing];
  __shared__ float2 red[GROUPS][2][MAXW];
  const int threads = (int)blockDim.x / GROUPS, warps = threads / 32;
  const int grp = (int)threadIdx.x / threads, t = (int)threadIdx.x - grp * threads;
  const int warp = t >> 5, lane = t & 31;
  const uint32_t row_bytes = (uint32_t)D * sizeof(T);
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int g = 0; g < GROUPS; ++g)
      for (int i = 0; i < stages; ++i) mbar_init(&full[g][i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  // rows blockIdx.x + (k GROUPS + grp) gridDim.x, k = 0, 1, ...
  const long long row0 = blockIdx.x + (long long)grp * gridDim.x;
  const long long stride = (long long)gridDim.x * GROUPS;
  const int rows = row0 < N ? (int)((N - 1 - row0) / stride) + 1 : 0;
  uint8_t* mine = ring + (size_t)grp * stages * 2 * row_bytes;
  auto issue = [&](int k) {
    const int st = k % stages;
    const long long row = row0 + k * stride;
    uint8_t* dst = mine + (size_t)st * 2 * row_bytes;
    mbar_arrive_expect_tx(&full[grp][st], 2 * row_bytes);
    bulk_load(dst, x + row * D, row_bytes, &full[grp][st]);
    bulk_load(dst + row_bytes, dy + row * D, row_bytes, &full[grp][st]);
  };
  if (t == 0)
    for (int k = 0; k < rows && k < stages; ++k) issue(k);
  const int nvec = D / VEC;
  float ag[NV][VEC], ab[NV][VEC], gm[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      ag[i][j] = ab[i][j] = 0.f;
      const int v = t + i * threads;
      gm[i][j] = v < nvec ? (gamma ? gamma[v * VEC + j] : 1.f) : 0.f;
    }
  const float inv = 1.f / (float)D;
  float mu_next = 0.f, rs_next = 0.f;  // read one row ahead
  if (rows > 0) {
    mu_next = mean[row0];
    rs_next = rstd[row0];
  }
  bool ok = true;  // after an expired wait: no more waits, but every barrier
  for (int k = 0; k < rows; ++k) {
    const long long row = row0 + k * stride;
    const int st = k % stages;
    const float mu = mu_next, rs = rs_next;
    if (k + 1 < rows) {
      mu_next = mean[row + stride];
      rs_next = rstd[row + stride];
    }
    ok = ok && mbar_wait_bounded(&full[grp][st], (uint32_t)((k / stages) & 1), err, limit_ns,
                                 kSite + __LINE__);
    const Vec<T, VEC>* xr =
        reinterpret_cast<const Vec<T, VEC>*>(mine + (size_t)st * 2 * row_bytes);
    const Vec<T, VEC>* dr =
        reinterpret_cast<const Vec<T, VEC>*>(mine + (size_t)st * 2 * row_bytes + row_bytes);
    float h[NV][VEC], u[NV][VEC];
    float s0 = 0.f, s1 = 0.f;
    const float nmr = -mu * rs;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (t + i * threads < nvec) {
        float d[VEC];
        unpack(xr[t + i * threads], h[i]);
        unpack(dr[t + i * threads], d);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          h[i][j] = fmaf(h[i][j], rs, nmr);
          u[i][j] = d[j] * gm[i][j];
          s0 += u[i][j];
          s1 = fmaf(u[i][j], h[i][j], s1);
          ag[i][j] = fmaf(d[j], h[i][j], ag[i][j]);
          ab[i][j] += d[j];
        }
      }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      s0 += __shfl_xor_sync(0xffffffffu, s0, o);
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    }
    if (lane == 0) red[grp][k & 1][warp] = make_float2(s0, s1);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(threads) : "memory");
    if (t == 0 && k + stages < rows) issue(k + stages);  // every thread has read the stage
    s0 = s1 = 0.f;
    for (int w = 0; w < warps; ++w) {
      const float2 v = red[grp][k & 1][w];
      s0 += v.x;
      s1 += v.y;
    }
    const float c0 = -s0 * inv * rs, c1 = -s1 * inv * rs;
    Vec<T, VEC>* o = reinterpret_cast<Vec<T, VEC>*>(dx + row * D);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (t + i * threads < nvec) {
        float f[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] = fmaf(u[i][j], rs, fmaf(h[i][j], c1, c0));
        o[t + i * threads] = pack<T, VEC>(f);
      }
  }
  if (t == 0)  // no copy may be in flight when the CTA exits (passes at once but after a timeout)
    for (int k = rows > stages ? rows - stages : 0; k < rows; ++k)
      mbar_wait_bounded(&full[grp][k % stages], (uint32_t)((k / stages) & 1), err, limit_ns,
                        kSite + __LINE__);
  if (GROUPS > 1) {  // the other groups' sums through the ring's memory: dgamma [D], dbeta [D]
    static_assert(GROUPS <= 2, "two groups are added");
    float* sums = reinterpret_cast<float*>(ring);
    __syncthreads();
    if (grp == 1)
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (t + i * threads < nvec)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            sums[(t + i * threads) * VEC + j] = ag[i][j];
            sums[D + (t + i * threads) * VEC + j] = ab[i][j];
          }
    __syncthreads();
    if (grp == 1) return;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (t + i * threads < nvec)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          ag[i][j] += sums[(t + i * threads) * VEC + j];
          ab[i][j] += sums[D + (t + i * threads) * VEC + j];
        }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (t + i * threads < nvec) {
      const long long at = (long long)blockIdx.x * D + (t + i * threads) * VEC;
      if (pg) *reinterpret_cast<Vec<float, VEC>*>(pg + at) = pack<float, VEC>(ag[i]);
      if (pb) *reinterpret_cast<Vec<float, VEC>*>(pb + at) = pack<float, VEC>(ab[i]);
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

// The backward's ring form: rows of 129 to 1024 16-byte vectors.
bool bwd_ring(const NormShape& f, int D) { return f.vec > 1 && D / f.vec > 128 && D / f.vec <= 1024; }
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
  const bool ring = bwd_ring(f, D);
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

template <typename T, int VEC, int NV>
cudaError_t fwd_rows(const void* x, int N, int D, const float* gamma, const float* beta, float eps,
                     void* y, float* mean, float* rstd, cudaStream_t s) {
  long long ctas = ((long long)N + kThreads / 32 - 1) / (kThreads / 32);
  const long long cap = 2LL * sm_count();
  return launch_pdl(layernorm_fwd_rows_kernel<T, VEC, NV>, dim3((unsigned)(ctas < cap ? ctas : cap)),
                    dim3(kThreads), (size_t)D * 8, s, static_cast<const T*>(x), N, D, gamma, beta, eps,
                    static_cast<T*>(y), mean, rstd);
}

template <typename T, int NV, int GROUPS>
cudaError_t bwd_ring_launch(const void* x, const void* dy, int N, int D, const float* gamma,
                            const float* mean, const float* rstd, void* dx, float* pg, float* pb,
                            int parts, cudaStream_t s) {
  const size_t stage = 2 * (size_t)D * sizeof(T);
  const int threads = ring_shape(D / (16 / (int)sizeof(T))).threads;
  int stages = (int)((size_t)kRingBytes / (GROUPS * stage));
  if (stages > kMaxRing) stages = kMaxRing;
  auto k = layernorm_bwd_ring_kernel<T, NV, GROUPS>;
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [&] {
    attr = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  });
  if (attr != cudaSuccess) return attr;
  return launch_pdl(k, dim3(parts), dim3(GROUPS * threads), GROUPS * stages * stage, s,
                    static_cast<const T*>(x), static_cast<const T*>(dy), N, D, gamma, mean, rstd,
                    static_cast<T*>(dx), pg, pb, stages, device_error_word(), kWaitLimitNs);
}

template <typename T, int VEC>
cudaError_t fwd_pick(const NormShape& f, const void* x, int N, int D, const float* gamma,
                     const float* beta, float eps, void* y, float* mean, float* rstd,
                     cudaStream_t s) {
  // from a few rows per SM on, and up to 16 vectors per lane: a warp per row
  if constexpr (VEC > 1) {
    const int nvec = D / VEC;
    if (N >= 8 * sm_count() && nvec <= 512) {
      if (nvec <= 128) return fwd_rows<T, VEC, 4>(x, N, D, gamma, beta, eps, y, mean, rstd, s);
      if (nvec <= 256) return fwd_rows<T, VEC, 8>(x, N, D, gamma, beta, eps, y, mean, rstd, s);
      return fwd_rows<T, VEC, 16>(x, N, D, gamma, beta, eps, y, mean, rstd, s);
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
    if (bwd_ring(f, D)) {
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
