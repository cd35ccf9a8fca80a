// The end of a training step over many tensors: the global norm of the gradients, clipping by it, and
// the optimizer step with the clipping factor applied as the gradients are read.
//
//   norm = sqrt(sum g^2),  f = min(1, max_norm / (norm + 1e-6)),  g <- f g  or  Adam(q, f g, m, v)
//
// All bound by HBM (norm: 4 or 2 bytes per element; update: 28).  The tensors' table is a kernel
// parameter, so that the host arrays are free when the call returns and a captured graph keeps them.  The
// tensors, laid end to end in units of 16 bytes of gradient, are cut into equal shares, one per resident
// CTA: found by one binary search, then followed from tensor to tensor, so that many small tensors and few
// large ones cost the same and no CTA is left with a last round of its own.  Every sum has a fixed order.
// Norm of 0.92 GB in 226 tensors: 139 us (6.5 TB/s).  Step of 11.2 M parameters in 14 tensors: 44 us; of
// 360 M in 448, with the norm before it, 1.63 ms (11.5 GB at 7.0 TB/s).
//
#include <algorithm>
#include <type_traits>

#include "adam.cuh"
#include "common.cuh"
#include "kernels.h"

namespace poetx {
namespace {

constexpr int kThreads = 256;
constexpr int kTensors = 512;               // of one launch,
constexpr int kFewTensors = 48;             // or of a launch with a table of a tenth
constexpr long long kMaxCount = 1ll << 33;  // elements of a tensor
constexpr int kMaxParts = 8;                // CTAs per SM at most, whatever the kernel

// ARRAYS pointers per tensor (the gradient first).
template <int MAX, int ARRAYS>
struct Table {
  int n;
  long long start[MAX + 1];  // the tensors' first units (the last one of a tensor may be part of one)
  void* p[ARRAYS][MAX];
  long long count[MAX];
  uint8_t bf16[MAX];
};

// Calls f(tensor, first unit in it, whole units, elements of a part of a unit behind them) for each
// piece of the CTA's share.
template <int MAX, int ARRAYS, typename F>
__device__ __forceinline__ void for_share(const Table<MAX, ARRAYS>& t, F f) {
  const long long total = t.start[t.n];
  long long u = total * blockIdx.x / gridDim.x;
  const long long end = total * (blockIdx.x + 1) / gridDim.x;
  if (u >= end) return;
  int lo = 0, hi = t.n;  // the last tensor that begins at or before u
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.start[mid] <= u) lo = mid;
    else hi = mid;
  }
  for (int k = lo; u < end; ++k) {
    const int per = t.bf16[k] ? 8 : 4;
    const long long stop = min(end, t.start[k + 1]), first = u - t.start[k];
    const long long whole = min(t.count[k] / per, first + (stop - u));  // end of the whole units
    const bool last = stop == t.start[k + 1];
    f(k, first, (int)(whole - first), last ? (int)(t.count[k] % per) : 0);
    u = stop;
  }
}

// f = min(1, max_norm / (norm + 1e-6)), NaN where that is.
__device__ __forceinline__ float clip_factor(const float* norm, float max_norm) {
  if (!norm) return 1.f;
  const float f = max_norm / (*norm + 1e-6f);
  return f >= 1.f ? 1.f : f;
}

// The rounding error of s = a + b, exactly (Knuth's two-sum), for each of two.
__device__ __forceinline__ float2 lost_by(float2 a, float2 b, float2 s) {
  const float2 b0 = add2(s, neg2(a)), a0 = add2(s, neg2(b0));
  return add2(add2(a, neg2(a0)), add2(b, neg2(b0)));
}

// A sum in two numbers: what rounding took from the first is in the second.  What rounding takes from that is at
// most n^2 2^-50 of the sum over n adds: 2^-27 for the 2800 of a thread's share of 2^33 elements.  (64-bit adds run
// at two a cycle on an SM.)
struct Sum2 {
  float2 top = {0.f, 0.f}, rest = {0.f, 0.f};
  __device__ __forceinline__ void add(float2 v) {
    const float2 s = add2(top, v);
    rest = add2(rest, lost_by(top, v, s));
    top = s;
  }
};

// A thread's sum of squares.  The kUnroll vectors that it loads at a time give two fp32 sums of eight terms
// at most, whose sum (off by 9 x 2^-24 at most) a Sum2 takes up, so that the error is the same for few elements and
// for many.  Where the largest of a vector would lose its square to fp32's range (above 2^50, or below 2^-50
// and not zero), that vector goes into a 64-bit sum.  The others beside a largest of 2^-50 or more are below
// 2^-13 of it where their square leaves the normal range.
constexpr int kUnroll = 4;
struct Squares {
  float2 a = {0.f, 0.f}, b = {0.f, 0.f};  // since the last flush
  Sum2 sum;
  double wide = 0.0;
  template <int N>
  __device__ __forceinline__ void add(const float (&v)[N]) {
    float top = 0.f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      top = fmaxf(top, fabsf(v[i]));
      nan |= v[i] != v[i];
    }
    if ((top >= 0x1p-50f && top <= 0x1p50f) && !nan) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float2 x = make_float2(v[i], v[i + 1]), y = make_float2(v[i + 2], v[i + 3]);
        a = fma2(x, x, a);
        b = fma2(y, y, b);
      }
    } else if (top > 0.f || nan) {
#pragma unroll
      for (int i = 0; i < N; ++i) wide += (double)v[i] * (double)v[i];
    }
  }
  __device__ __forceinline__ void flush() {
    sum.add(add2(a, b));
    a = b = both(0.f);
  }
};

__device__ __forceinline__ void words(const uint4& w, float (&v)[4]) {
  v[0] = __uint_as_float(w.x);
  v[1] = __uint_as_float(w.y);
  v[2] = __uint_as_float(w.z);
  v[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void halves(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// The CTA's sum over its threads, on thread 0: two-number sums as well, and 64 bits where a thread had
// recourse to them.
__device__ __forceinline__ double block_sum(const Squares& s) {
  __shared__ float2 red[kThreads / 32];
  __shared__ double red_wide[kThreads / 32];
  // (both halves of a pair carry the same numbers from here on)
  Sum2 v{both(s.sum.top.x), both(s.sum.rest.x)};
  v.add(both(s.sum.top.y));
  v.rest = add2(v.rest, both(s.sum.rest.y));
  double w = s.wide;
  auto join = [&](int o) {
    const float top = __shfl_xor_sync(0xffffffffu, v.top.x, o);
    const float rest = __shfl_xor_sync(0xffffffffu, v.rest.x, o);
    v.add(both(top));
    v.rest = add2(v.rest, both(rest));
    if (__any_sync(0xffffffffu, w != 0.0)) w += __shfl_xor_sync(0xffffffffu, w, o);
  };
#pragma unroll
  for (int o = 16; o; o >>= 1) join(o);
  if ((threadIdx.x & 31) == 0) {
    red[threadIdx.x >> 5] = make_float2(v.top.x, v.rest.x);
    red_wide[threadIdx.x >> 5] = w;
  }
  __syncthreads();
  if (threadIdx.x >= 32) return 0.0;
  constexpr int W = kThreads / 32;
  const float2 mine = red[threadIdx.x % W];
  v = Sum2{both(mine.x), both(mine.y)};
  w = red_wide[threadIdx.x % W];
#pragma unroll
  for (int o = W / 2; o; o >>= 1) join(o);
  return ((double)v.top.x + (double)v.rest.x) + w;
}

// (Five CTAs per SM: with six the two-number sums spill and 0.92 GB take 149 us.)
template <int MAX>
__global__ void __launch_bounds__(kThreads, 5)
    norm_kernel(const __grid_constant__ Table<MAX, 1> t, double* part) {
  pdl_trigger();
  pdl_wait();
  Squares sq;
  for_share(t, [&](int k, long long first, int units, int rest) {
    const uint4* g = static_cast<const uint4*>(t.p[0][k]) + first;
    const bool half = t.bf16[k];
    constexpr int U = kUnroll;
    for (int i0 = threadIdx.x; i0 < units; i0 += U * kThreads) {
      uint4 w[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (i0 + j * kThreads < units) w[j] = g[i0 + j * kThreads];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (i0 + j * kThreads >= units) break;
        if (half) {
          float v[8];
          halves(w[j], v);
          sq.add(v);
        } else {
          float v[4];
          words(w[j], v);
          sq.add(v);
        }
      }
      sq.flush();
    }
    if ((int)threadIdx.x < rest) {  // the tensor's last elements
      const void* e = g + units;
      const float v[4] = {half ? __bfloat162float(static_cast<const __nv_bfloat16*>(e)[threadIdx.x])
                               : static_cast<const float*>(e)[threadIdx.x], 0.f, 0.f, 0.f};
      sq.add(v);
      sq.flush();
    }
  });
  const double s = block_sum(sq);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

constexpr int kJoinThreads = 128;
__global__ void __launch_bounds__(kJoinThreads) norm_join_kernel(const double* part, int n, float* norm) {
  __shared__ double red[kJoinThreads / 32];
  pdl_trigger();
  pdl_wait();
  double v = 0.0;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kJoinThreads) v += part[i];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) *norm = (float)sqrt((red[0] + red[1]) + (red[2] + red[3]));
}

template <int MAX>
__global__ void __launch_bounds__(kThreads, 6)
    clip_kernel(const __grid_constant__ Table<MAX, 1> t, float max_norm, const float* norm) {
  pdl_trigger();
  pdl_wait();
  const float f = clip_factor(norm, max_norm);
  if (f == 1.f) return;
  for_share(t, [&](int k, long long first, int units, int rest) {
    uint4* g = static_cast<uint4*>(t.p[0][k]) + first;
    const bool half = t.bf16[k];
    constexpr int U = 4;
    for (int i0 = threadIdx.x; i0 < units; i0 += U * kThreads) {
      uint4 w[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (i0 + j * kThreads < units) w[j] = g[i0 + j * kThreads];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (i0 + j * kThreads >= units) break;
        if (half) {
          float v[8];
          halves(w[j], v);
          w[j] = make_uint4(pack_bf16x2(f * v[0], f * v[1]), pack_bf16x2(f * v[2], f * v[3]),
                            pack_bf16x2(f * v[4], f * v[5]), pack_bf16x2(f * v[6], f * v[7]));
        } else {
          float v[4];
          words(w[j], v);
          w[j] = make_uint4(__float_as_uint(f * v[0]), __float_as_uint(f * v[1]),
                            __float_as_uint(f * v[2]), __float_as_uint(f * v[3]));
        }
        g[i0 + j * kThreads] = w[j];
      }
    }
    if ((int)threadIdx.x < rest) {
      if (half) {
        __nv_bfloat16* e = reinterpret_cast<__nv_bfloat16*>(g + units) + threadIdx.x;
        *e = __float2bfloat16_rn(f * __bfloat162float(*e));
      } else {
        reinterpret_cast<float*>(g + units)[threadIdx.x] *= f;
      }
    }
  });
}

template <int MAX>
__global__ void __launch_bounds__(kThreads, 4)
    adam_group_kernel(const __grid_constant__ Table<MAX, 4> t, AdamK h, float max_norm, const float* norm) {
  pdl_trigger();
  pdl_wait();
  const float f = clip_factor(norm, max_norm);
  for_share(t, [&](int k, long long first, int units, int rest) {
    const float4* g = static_cast<const float4*>(t.p[0][k]) + first;
    float4* q = static_cast<float4*>(t.p[1][k]) + first;
    float4* m = static_cast<float4*>(t.p[2][k]) + first;
    float4* v = static_cast<float4*>(t.p[3][k]) + first;
    constexpr int U = 2;
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < units; i0 += U * kThreads) {
      float4 gw[U], qw[U], mw[U], vw[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * kThreads;
        if (i < units) {
          gw[j] = g[i];
          qw[j] = q[i];
          mw[j] = m[i];
          vw[j] = v[i];
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * kThreads;
        if (i >= units) break;
        adam_one(qw[j].x, __fmul_rn(gw[j].x, f), mw[j].x, vw[j].x, h);
        adam_one(qw[j].y, __fmul_rn(gw[j].y, f), mw[j].y, vw[j].y, h);
        adam_one(qw[j].z, __fmul_rn(gw[j].z, f), mw[j].z, vw[j].z, h);
        adam_one(qw[j].w, __fmul_rn(gw[j].w, f), mw[j].w, vw[j].w, h);
        q[i] = qw[j];
        m[i] = mw[j];
        v[i] = vw[j];
      }
    }
    if ((int)threadIdx.x < rest) {
      const int i = 4 * units + threadIdx.x;
      adam_one(reinterpret_cast<float*>(q)[i], __fmul_rn(reinterpret_cast<const float*>(g)[i], f),
               reinterpret_cast<float*>(m)[i], reinterpret_cast<float*>(v)[i], h);
    }
  });
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The checks of n tensors' host arrays (ARRAYS of pointers): POETX_OK, or what is wrong.
template <int ARRAYS>
poetx_status check_arrays(void* const* const (&p)[ARRAYS], const poetx_dtype* dt, const long long* count,
                          int n) {
  if (n < 0) return POETX_ERR_ARG;
  if (n == 0) return POETX_OK;
  for (int a = 0; a < ARRAYS; ++a)
    if (!p[a]) return POETX_ERR_ARG;
  if (!count) return POETX_ERR_ARG;
  for (int i = 0; i < n; ++i) {
    if (count[i] < 0) return POETX_ERR_ARG;
    if (dt && dt[i] != POETX_F32 && dt[i] != POETX_BF16) return POETX_ERR_DTYPE;
    if (count[i] > kMaxCount) return POETX_ERR_SHAPE;
    for (int a = 0; a < ARRAYS; ++a) {
      if (count[i] > 0 && !p[a][i]) return POETX_ERR_ARG;
      if (!aligned16(p[a][i])) return POETX_ERR_ALIGN;
    }
  }
  return POETX_OK;
}

// The table of the next tensors from *at on (those without elements left out), at most MAX of them; false
// when none is left.
template <int MAX, int ARRAYS>
bool next_table(void* const* const (&p)[ARRAYS], const poetx_dtype* dt, const long long* count, int n,
                int* at, Table<MAX, ARRAYS>* t) {
  t->n = 0;
  t->start[0] = 0;
  while (*at < n && t->n < MAX) {
    const int i = (*at)++;
    const bool half = dt && dt[i] == POETX_BF16;
    if (!count[i]) continue;
    const int k = t->n++, per = half ? 8 : 4;
    for (int a = 0; a < ARRAYS; ++a) t->p[a][k] = p[a][i];
    t->count[k] = count[i];
    t->bf16[k] = half;
    t->start[k + 1] = t->start[k] + (count[i] + per - 1) / per;
  }
  return t->n > 0;
}

using Few = std::integral_constant<int, kFewTensors>;
using Many = std::integral_constant<int, kTensors>;

// CTAs of a kernel: one per kThreads units up to the resident ones, or, where `small` units are enough
// for a CTA, as many as there are such shares.  The norm, which only reads, runs at the copy's rate with
// equal shares for the resident CTAs (0.9 GB in 139 us).  The step, with seven streams, wants neighbouring
// CTAs at neighbouring addresses and a scheduler that hands out work as it is done: 360 million
// parameters (norm included) take 1.93 ms with resident shares, 1.67 with 1024 units, 1.63 with 512, the
// two vectors that a thread has in flight.
template <typename K>
int grid_of(K kernel, long long units, int small = 0) {
  static PerDevice<int> blocks;  // (per kernel: a type of its own)
  const int per_sm = blocks.get(current_device(), [&] {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, 0) != cudaSuccess) n = 1;
    return std::min(std::max(n, 1), kMaxParts);
  });
  const long long even = std::min<long long>((units + kThreads - 1) / kThreads,
                                             (long long)per_sm * sm_count());
  return (int)std::max(small ? units / small : 0, even);
}

}  // namespace
}  // namespace poetx

using namespace poetx;

extern "C" size_t poetx_grad_norm_workspace_bytes(int n) {
  if (n < 0) return 0;
  const long long launches = n / kTensors + 1;
  return align_up((size_t)launches * kMaxParts * sm_count() * sizeof(double), 256);
}

extern "C" poetx_status poetx_grad_norm(const void* const* g, const poetx_dtype* dt,
                                        const long long* count, int n, float* norm, void* ws,
                                        size_t ws_bytes, cudaStream_t stream) {
  void* const* const p[1] = {(void* const*)g};
  if (n > 0 && !dt) return POETX_ERR_ARG;
  POETX_TRY(check_arrays(p, dt, count, n));
  if (!norm || !ws) return POETX_ERR_ARG;
  if (!aligned4(norm) || !aligned16(ws)) return POETX_ERR_ALIGN;
  if (ws_bytes < poetx_grad_norm_workspace_bytes(n)) return POETX_ERR_WORKSPACE;
  double* part = static_cast<double*>(ws);
  int parts = 0;
  auto run = [&](auto kernel, auto max) -> poetx_status {
    Table<decltype(max)::value, 1> t;
    for (int at = 0; next_table(p, dt, count, n, &at, &t);) {
      const int grid = grid_of(kernel, t.start[t.n]);
      POETX_CUDA_TRY(launch_pdl(kernel, dim3(grid), dim3(kThreads), 0, stream, t, part + parts));
      POETX_CUDA_TRY(cudaGetLastError());
      after_launch(stream, ST_GRAD_NORM);
      parts += grid;
    }
    return POETX_OK;
  };
  POETX_TRY(n <= kFewTensors ? run(norm_kernel<kFewTensors>, Few{}) : run(norm_kernel<kTensors>, Many{}));
  POETX_CUDA_TRY(launch_pdl(norm_join_kernel, dim3(1), dim3(kJoinThreads), 0, stream, (const double*)part,
                            parts, norm));
  POETX_CUDA_TRY(cudaGetLastError());
  after_launch(stream, ST_GRAD_NORM);
  return POETX_OK;
}

extern "C" poetx_status poetx_grad_clip(void* const* g, const poetx_dtype* dt, const long long* count,
                                        int n, float max_norm, const float* norm, cudaStream_t stream) {
  void* const* const p[1] = {g};
  if (n > 0 && !dt) return POETX_ERR_ARG;
  POETX_TRY(check_arrays(p, dt, count, n));
  if (!(max_norm >= 0.f) || !norm) return POETX_ERR_ARG;
  if (!aligned4(norm)) return POETX_ERR_ALIGN;
  auto run = [&](auto kernel, auto max) -> poetx_status {
    Table<decltype(max)::value, 1> t;
    for (int at = 0; next_table(p, dt, count, n, &at, &t);) {
      POETX_CUDA_TRY(launch_pdl(kernel, dim3(grid_of(kernel, t.start[t.n])), dim3(kThreads), 0, stream, t,
                                max_norm, norm));
      POETX_CUDA_TRY(cudaGetLastError());
      after_launch(stream, ST_GRAD_NORM);
    }
    return POETX_OK;
  };
  return n <= kFewTensors ? run(clip_kernel<kFewTensors>, Few{}) : run(clip_kernel<kTensors>, Many{});
}

extern "C" poetx_status poetx_adam_group(float* const* q, const float* const* dq, float* const* m,
                                         float* const* v, const long long* count, int n,
                                         const poetx_adam* hp, float max_norm, const float* norm,
                                         cudaStream_t stream) {
  AdamK h;
  POETX_TRY(adam_params(hp, &h));
  void* const* const p[4] = {(void* const*)dq, (void* const*)q, (void* const*)m, (void* const*)v};
  POETX_TRY(check_arrays(p, nullptr, count, n));
  if (norm && !(max_norm >= 0.f)) return POETX_ERR_ARG;
  if (!aligned4(norm)) return POETX_ERR_ALIGN;
  auto run = [&](auto kernel, auto max) -> poetx_status {
    Table<decltype(max)::value, 4> t;
    for (int at = 0; next_table(p, nullptr, count, n, &at, &t);) {
      POETX_CUDA_TRY(launch_pdl(kernel, dim3(grid_of(kernel, t.start[t.n], 512)), dim3(kThreads), 0, stream,
                                t, h, max_norm, norm));
      POETX_CUDA_TRY(cudaGetLastError());
      after_launch(stream, ST_OPTIM);
    }
    return POETX_OK;
  };
  return n <= kFewTensors ? run(adam_group_kernel<kFewTensors>, Few{})
                          : run(adam_group_kernel<kTensors>, Many{});
}
