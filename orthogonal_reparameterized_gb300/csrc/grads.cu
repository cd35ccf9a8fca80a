// The end of a training step over many tensors: the global norm of the gradients, clipping by it, and
// the optimizer step with the clipping factor applied as the gradients are read.
//
//   norm = sqrt(sum g^2),  f = min(1, max_norm / (norm + 1e-6)),  g <- f g  or  Adam(q, f g, m, v)
//
// All bound by HBM (norm: 4 or 2 bytes per element; update: 28).  The tensors' table is a kernel
// parameter, so that the host arrays are free when the call returns and a captured graph keeps them.  The
// tensors are cut into chunks of 16 KB of gradient; a CTA takes a contiguous range of all chunks (found by
// one binary search, then followed), so that many small tensors and few large ones cost the same.  Every
// sum has a fixed order.
#include <algorithm>

#include "adam.cuh"
#include "common.cuh"
#include "kernels.h"

namespace poetx {
namespace {

constexpr int kThreads = 256;
constexpr int kTensors = 512;        // of one launch
constexpr int kChunkBytes = 16384;   // of gradient: four 16-byte loads per thread
constexpr int kNormCtasPerSm = 8;
constexpr long long kMaxCount = 1ll << 33;  // elements of a tensor: a launch's chunks stay below 2^31

// ARRAYS pointers per tensor (the gradient first).
template <int MAX, int ARRAYS>
struct Table {
  int n;
  int start[MAX + 1];  // first chunk of each tensor, start[n] the number of chunks
  void* p[ARRAYS][MAX];
  long long count[MAX];
  uint8_t bf16[MAX];
};

__device__ __forceinline__ int find_tensor(const int* start, int n, int chunk) {
  int lo = 0, hi = n;  // the last tensor that begins at or before the chunk
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// f = min(1, max_norm / (norm + 1e-6)), NaN where that is.
__device__ __forceinline__ float clip_factor(const float* norm, float max_norm) {
  if (!norm) return 1.f;
  const float f = max_norm / (*norm + 1e-6f);
  return f >= 1.f ? 1.f : f;
}

// Squares of eight (four) neighbouring values into the thread's fp32 sums, or, where the largest would
// lose them to fp32's range (above 2^50, or below 2^-50 and not zero), into its 64-bit one.  The others
// beside a largest of 2^-50 or more are below 2^-13 of it where their square leaves the normal range.
struct Squares {
  float2 a = {0.f, 0.f}, b = {0.f, 0.f};
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
  __device__ __forceinline__ double sum() const {
    return ((double)a.x + (double)a.y) + ((double)b.x + (double)b.y) + wide;
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

// The CTA's sum over its threads, on thread 0, in a fixed order.
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < (int)blockDim.x / 32; ++w) s += red[w];
  return s;
}

__global__ void __launch_bounds__(kThreads)
    norm_kernel(const __grid_constant__ Table<kTensors, 1> t, double* part) {
  __shared__ double red[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int chunks = t.start[t.n];
  const int c0 = (int)((long long)chunks * blockIdx.x / gridDim.x);
  const int c1 = (int)((long long)chunks * (blockIdx.x + 1) / gridDim.x);
  Squares sq;
  int k = c0 < c1 ? find_tensor(t.start, t.n, c0) : 0;
  for (int c = c0; c < c1; ++c) {
    while (c >= t.start[k + 1]) ++k;
    const bool half = t.bf16[k];
    const int per = half ? kChunkBytes / 2 : kChunkBytes / 4;  // elements of a chunk
    const long long e0 = (long long)(c - t.start[k]) * per;
    const int n = (int)min((long long)per, t.count[k] - e0);
    const uint8_t* g = static_cast<const uint8_t*>(t.p[0][k]) + e0 * (half ? 2 : 4);
    const int vecs = n / (half ? 8 : 4);
    uint4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = threadIdx.x + j * kThreads;
      if (i < vecs) w[j] = reinterpret_cast<const uint4*>(g)[i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if ((int)threadIdx.x + j * kThreads < vecs) {
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
    const int done = vecs * (half ? 8 : 4);
    if ((int)threadIdx.x < n - done) {  // the tensor's last elements
      const int i = done + threadIdx.x;
      const float v[4] = {half ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(g)[i])
                               : reinterpret_cast<const float*>(g)[i], 0.f, 0.f, 0.f};
      sq.add(v);
    }
  }
  const double s = block_sum(sq.sum(), red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ void __launch_bounds__(1024) norm_join_kernel(const double* part, int n, float* norm) {
  __shared__ double red[32];
  pdl_trigger();
  pdl_wait();
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) v += part[i];
  const double s = block_sum(v, red);
  if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

__global__ void __launch_bounds__(kThreads)
    clip_kernel(const __grid_constant__ Table<kTensors, 1> t, float max_norm, const float* norm) {
  pdl_trigger();
  pdl_wait();
  const float f = clip_factor(norm, max_norm);
  if (f == 1.f) return;
  const int chunks = t.start[t.n];
  const int c0 = (int)((long long)chunks * blockIdx.x / gridDim.x);
  const int c1 = (int)((long long)chunks * (blockIdx.x + 1) / gridDim.x);
  int k = c0 < c1 ? find_tensor(t.start, t.n, c0) : 0;
  for (int c = c0; c < c1; ++c) {
    while (c >= t.start[k + 1]) ++k;
    const bool half = t.bf16[k];
    const int per = half ? kChunkBytes / 2 : kChunkBytes / 4;
    const long long e0 = (long long)(c - t.start[k]) * per;
    const int n = (int)min((long long)per, t.count[k] - e0);
    uint8_t* g = static_cast<uint8_t*>(t.p[0][k]) + e0 * (half ? 2 : 4);
    const int vecs = n / (half ? 8 : 4);
    uint4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = threadIdx.x + j * kThreads;
      if (i < vecs) w[j] = reinterpret_cast<const uint4*>(g)[i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = threadIdx.x + j * kThreads;
      if (i >= vecs) break;
      if (half) {
        float v[8];
        halves(w[j], v);
        reinterpret_cast<uint4*>(g)[i] =
            make_uint4(pack_bf16x2(f * v[0], f * v[1]), pack_bf16x2(f * v[2], f * v[3]),
                       pack_bf16x2(f * v[4], f * v[5]), pack_bf16x2(f * v[6], f * v[7]));
      } else {
        float v[4];
        words(w[j], v);
        reinterpret_cast<float4*>(g)[i] = make_float4(f * v[0], f * v[1], f * v[2], f * v[3]);
      }
    }
    const int done = vecs * (half ? 8 : 4);
    if ((int)threadIdx.x < n - done) {
      const int i = done + threadIdx.x;
      if (half) {
        __nv_bfloat16* e = reinterpret_cast<__nv_bfloat16*>(g) + i;
        *e = __float2bfloat16_rn(f * __bfloat162float(*e));
      } else {
        reinterpret_cast<float*>(g)[i] *= f;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    adam_group_kernel(const __grid_constant__ Table<kTensors, 4> t, AdamK h, float max_norm,
                      const float* norm) {
  pdl_trigger();
  pdl_wait();
  const float f = clip_factor(norm, max_norm);
  const int chunks = t.start[t.n];
  const int c0 = (int)((long long)chunks * blockIdx.x / gridDim.x);
  const int c1 = (int)((long long)chunks * (blockIdx.x + 1) / gridDim.x);
  int k = c0 < c1 ? find_tensor(t.start, t.n, c1 - 1) : 0;
  for (int c = c1 - 1; c >= c0; --c) {  // (backwards: the norm has left each CTA's last chunks in L2)
    while (c < t.start[k]) --k;
    const long long e0 = (long long)(c - t.start[k]) * (kChunkBytes / 4);
    const int n = (int)min((long long)(kChunkBytes / 4), t.count[k] - e0);
    const float* g = static_cast<const float*>(t.p[0][k]) + e0;
    float* q = static_cast<float*>(t.p[1][k]) + e0;
    float* m = static_cast<float*>(t.p[2][k]) + e0;
    float* v = static_cast<float*>(t.p[3][k]) + e0;
    const int vecs = n / 4;
    constexpr int U = 2;
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < vecs; i0 += U * kThreads) {
      float4 gw[U], qw[U], mw[U], vw[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * kThreads;
        if (i < vecs) {
          gw[j] = reinterpret_cast<const float4*>(g)[i];
          qw[j] = reinterpret_cast<const float4*>(q)[i];
          mw[j] = reinterpret_cast<const float4*>(m)[i];
          vw[j] = reinterpret_cast<const float4*>(v)[i];
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * kThreads;
        if (i >= vecs) break;
        adam_one(qw[j].x, __fmul_rn(gw[j].x, f), mw[j].x, vw[j].x, h);
        adam_one(qw[j].y, __fmul_rn(gw[j].y, f), mw[j].y, vw[j].y, h);
        adam_one(qw[j].z, __fmul_rn(gw[j].z, f), mw[j].z, vw[j].z, h);
        adam_one(qw[j].w, __fmul_rn(gw[j].w, f), mw[j].w, vw[j].w, h);
        reinterpret_cast<float4*>(q)[i] = qw[j];
        reinterpret_cast<float4*>(m)[i] = mw[j];
        reinterpret_cast<float4*>(v)[i] = vw[j];
      }
    }
    if ((int)threadIdx.x < n - 4 * vecs) {
      const int i = 4 * vecs + threadIdx.x;
      adam_one(q[i], __fmul_rn(g[i], f), m[i], v[i], h);
    }
  }
}

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

long long chunks_of(long long count, bool half) {
  const long long per = half ? kChunkBytes / 2 : kChunkBytes / 4;
  return (count + per - 1) / per;
}

// The table of the next tensors from *at on (those without elements left out), at most kTensors of them;
// false when none is left.
template <int ARRAYS>
bool next_table(void* const* const (&p)[ARRAYS], const poetx_dtype* dt, const long long* count, int n,
                int* at, Table<kTensors, ARRAYS>* t) {
  t->n = 0;
  t->start[0] = 0;
  while (*at < n && t->n < kTensors) {
    const int i = (*at)++;
    const bool half = dt && dt[i] == POETX_BF16;
    const long long c = chunks_of(count[i], half);
    if (!c) continue;
    const int k = t->n++;
    for (int a = 0; a < ARRAYS; ++a) t->p[a][k] = p[a][i];
    t->count[k] = count[i];
    t->bf16[k] = half;
    t->start[k + 1] = t->start[k] + (int)c;
  }
  return t->n > 0;
}

int grid_of(int chunks, int per_sm) { return std::min(chunks, per_sm * sm_count()); }

}  // namespace
}  // namespace poetx

using namespace poetx;

extern "C" size_t poetx_grad_norm_workspace_bytes(int n) {
  if (n < 0) return 0;
  const long long launches = n / kTensors + 1;
  return align_up((size_t)launches * kNormCtasPerSm * sm_count() * sizeof(double), 256);
}

extern "C" poetx_status poetx_grad_norm(const void* const* g, const poetx_dtype* dt,
                                        const long long* count, int n, float* norm, void* ws,
                                        size_t ws_bytes, cudaStream_t stream) {
  void* const* const p[1] = {(void* const*)g};
  if (n > 0 && !dt) return POETX_ERR_ARG;
  POETX_TRY(check_arrays(p, dt, count, n));
  if (!norm || !ws) return POETX_ERR_ARG;
  if (!aligned16(norm) || !aligned16(ws)) return POETX_ERR_ALIGN;
  if (ws_bytes < poetx_grad_norm_workspace_bytes(n)) return POETX_ERR_WORKSPACE;
  double* part = static_cast<double*>(ws);
  int parts = 0, at = 0;
  Table<kTensors, 1> t;
  while (next_table(p, dt, count, n, &at, &t)) {
    const int grid = grid_of(t.start[t.n], kNormCtasPerSm);
    POETX_CUDA_TRY(launch_pdl(norm_kernel, dim3(grid), dim3(kThreads), 0, stream, t, part + parts));
    POETX_CUDA_TRY(cudaGetLastError());
    after_launch(stream, ST_GRAD_NORM);
    parts += grid;
  }
  POETX_CUDA_TRY(launch_pdl(norm_join_kernel, dim3(1), dim3(1024), 0, stream, (const double*)part, parts,
                            norm));
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
  if (!aligned16(norm)) return POETX_ERR_ALIGN;
  int at = 0;
  Table<kTensors, 1> t;
  while (next_table(p, dt, count, n, &at, &t)) {
    POETX_CUDA_TRY(launch_pdl(clip_kernel, dim3(grid_of(t.start[t.n], kNormCtasPerSm)), dim3(kThreads), 0,
                              stream, t, max_norm, norm));
    POETX_CUDA_TRY(cudaGetLastError());
    after_launch(stream, ST_GRAD_NORM);
  }
  return POETX_OK;
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
  if (!aligned16(norm)) return POETX_ERR_ALIGN;
  int at = 0;
  Table<kTensors, 4> t;
  while (next_table(p, nullptr, count, n, &at, &t)) {
    POETX_CUDA_TRY(launch_pdl(adam_group_kernel, dim3(grid_of(t.start[t.n], 8)), dim3(kThreads), 0,
                              stream, t, h, max_norm, norm));
    POETX_CUDA_TRY(cudaGetLastError());
    after_launch(stream, ST_OPTIM);
  }
  return POETX_OK;
}
