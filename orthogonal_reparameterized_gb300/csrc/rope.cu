// Queries and keys of a transformer block: the root-mean-square norm of each head and the rotation of
// its pairs by the token's positions, forward and backward, in one pass over the data.
//
//   n = x rstd gamma, rstd = 1 / sqrt(mean(x^2) + eps)      (or n = x)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = pos[axis_i] inv_freq_i
//   backward: dn = the rotation of dy by -t, u = dn gamma, h = x rstd,
//             dx = rstd (u - h mean(u h)),  dgamma = sum dn h
//
// Bound by HBM: every element is read once and written once.  A group of G lanes (a power of two) holds
// one head: lane c its c-th chunk, CH pairs in two vectors of CH elements, so that both elements of a
// pair, their angle and their gamma are in one lane's registers whatever the pairing.  All heads of a token
// use the same angles: a lane makes those of its CH pairs once per token and keeps them over the heads.
//
// The angle is reduced in 64-bit fixed point: with f = inv_freq / 2 pi in units of 2^-64 turns (modulo a
// turn), pos * f modulo 2^64 is the angle modulo a turn, exact to 2^-32 turns at any int32 position (an
// fp32 product of position and frequency has lost the angle's second decimal at position 100000).
#include <mutex>

#include "common.cuh"
#include "kernels.h"

namespace poetx {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxHalf = 256;   // pairs of a head
constexpr int kCtasPerSm = 2;
constexpr int kMaxAxes = 8;

struct Side {
  const void* x;
  const void* dy;
  void* y;
  const float* gamma;
  float* part;              // backward: [ctas][dh] partial sums of dgamma (nullable)
  long long xp, dyp, yp;
  int H;
  int hs, parts;            // heads of a task, tasks of a token
  int ctas;
  long long tasks;
};
struct RopeArgs {
  Side s[2];
  const int32_t* pos;
  const float* inv_freq;
  const int32_t* axis;
  int N, axes;
  int dh, half;
  int G;                    // lanes of a head
  float eps;
};

template <int CH>
__device__ __forceinline__ void widen(const uint32_t (&r)[CH / 2], float* v, __nv_bfloat16) {
#pragma unroll
  for (int i = 0; i < CH / 2; ++i) {
    v[2 * i] = __uint_as_float(r[i] << 16);
    v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
  }
}
template <int CH>
__device__ __forceinline__ void widen(const uint32_t (&r)[CH], float* v, float) {
#pragma unroll
  for (int i = 0; i < CH; ++i) v[i] = __uint_as_float(r[i]);
}

// One chunk as it lies in memory: two vectors of CH elements.
template <typename T, int CH>
struct Chunk {
  static constexpr int WORDS = CH * (int)sizeof(T) / 4;
  uint32_t r[2][WORDS];
  __device__ __forceinline__ void load(const T* p, int o0, int o1) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const T* q = p + (k ? o1 : o0);
      if constexpr (WORDS == 2) {
        const uint2 w = *reinterpret_cast<const uint2*>(q);
        r[k][0] = w.x;
        r[k][1] = w.y;
      } else {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4) {
          const uint4 w = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(q) + i);
          r[k][i] = w.x;
          r[k][i + 1] = w.y;
          r[k][i + 2] = w.z;
          r[k][i + 3] = w.w;
        }
      }
    }
  }
  __device__ __forceinline__ void get(float (&v)[2 * CH]) const {
    widen<CH>(r[0], v, T());
    widen<CH>(r[1], v + CH, T());
  }
  __device__ __forceinline__ void put(const float (&v)[2 * CH]) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < WORDS; ++i)
        r[k][i] = sizeof(T) == 2 ? pack_bf16x2(v[k * CH + 2 * i], v[k * CH + 2 * i + 1])
                                 : __float_as_uint(v[k * CH + i]);
  }
  __device__ __forceinline__ void store(T* p, int o0, int o1) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      T* q = p + (k ? o1 : o0);
      if constexpr (WORDS == 2) {
        *reinterpret_cast<uint2*>(q) = make_uint2(r[k][0], r[k][1]);
      } else {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4)
          *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(q) + i) =
              make_uint4(r[k][i], r[k][i + 1], r[k][i + 2], r[k][i + 3]);
      }
    }
  }
};

template <typename T, int CH, bool INTER, bool NORM, bool BWD>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ unsigned long long turn[kMaxHalf];  // inv_freq / 2 pi, in 2^-64 turns
  __shared__ int ax[kMaxHalf];                   // the pair's axis, -1: NaN
  __shared__ float red[BWD && NORM ? kWarps * 2 * CH * 32 : 1];
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t < a.half) {
    const float f = a.inv_freq[t];
    const int axis = a.axis ? a.axis[t] : 0;
    double w = (double)f * 0.15915494309189533577;  // 1 / 2 pi
    w -= floor(w);
    turn[t] = w < 1.0 ? (unsigned long long)(w * 18446744073709551616.0) : 0ull;
    ax[t] = isfinite(f) && axis >= 0 && axis < a.axes ? axis : -1;
  }
  __syncthreads();
  const int which = (int)blockIdx.x >= a.s[0].ctas;
  const Side& s = a.s[which];
  const int cta = (int)blockIdx.x - (which ? a.s[0].ctas : 0);
  const int G = a.G, c = lane & (G - 1), sub = lane / G, HW = 32 / G;
  const int pr = a.half / CH;  // rotated chunks
  const bool mine = c < a.dh / (2 * CH), rot = c < pr;
  const int tail = 2 * a.half + 2 * CH * (c - pr);
  const int o0 = rot ? (INTER ? 2 * CH * c : CH * c) : tail;
  const int o1 = rot && !INTER ? a.half + CH * c : o0 + CH;
  float gm[2 * CH], dg[2 * CH];
#pragma unroll
  for (int i = 0; i < 2 * CH; ++i) {
    gm[i] = NORM && mine && s.gamma ? s.gamma[(i < CH ? o0 : o1 - CH) + i] : 1.f;
    dg[i] = 0.f;
  }
  const float inv_dh = 1.f / (float)a.dh;
  const T* const x = static_cast<const T*>(s.x);
  const T* const dy = static_cast<const T*>(s.dy);
  T* const y = static_cast<T*>(s.y);

  for (long long task = (long long)cta * kWarps + warp; task < s.tasks;
       task += (long long)s.ctas * kWarps) {
    const int token = s.parts == 1 ? (int)task : (int)(task / s.parts);
    const int part = s.parts == 1 ? 0 : (int)(task - (long long)token * s.parts);
    float cs[CH], sn[CH];
    if (rot) {
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int k = ax[CH * c + j];
        const int p = k < 0 ? 0 : a.pos[(long long)k * a.N + token];
        const unsigned long long ang = (unsigned long long)(long long)p * turn[CH * c + j];
        const float h = (float)(int)(ang >> 32) * 0x1p-32f;  // turns, in [-1/2, 1/2]
        // bf16: the hardware's sine and cosine, within 2^-21 on (-pi, pi), far below the result's
        // rounding
        if (sizeof(T) == 2) __sincosf(h * 6.28318530717958647692f, &sn[j], &cs[j]);
        else sincospif(2.f * h, &sn[j], &cs[j]);
        if (k < 0) cs[j] = sn[j] = __int_as_float(0x7fc00000);
      }
    }
    const int h_end = min(s.H, (part + 1) * s.hs);
    constexpr int U = BWD && NORM ? 2 : 4;  // heads in flight per group
    for (int h0 = part * s.hs; h0 < h_end; h0 += U * HW) {
      Chunk<T, CH> rx[U], ry[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int h = h0 + k * HW + sub;
        if (mine && h < h_end) {
          if (!BWD || NORM) rx[k].load(x + (long long)token * s.xp + (long long)h * a.dh, o0, o1);
          if (BWD) ry[k].load(dy + (long long)token * s.dyp + (long long)h * a.dh, o0, o1);
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (h0 + k * HW >= h_end) break;  // (the same for the whole warp)
        const int h = h0 + k * HW + sub;
        const bool on = mine && h < h_end;
        float v[2 * CH], d[2 * CH];
#pragma unroll
        for (int i = 0; i < 2 * CH; ++i) v[i] = d[i] = 0.f;
        if (on) {
          if (!BWD || NORM) rx[k].get(v);
          if (BWD) ry[k].get(d);
        }
        auto rotate = [&](float (&w)[2 * CH], float sign) {
          if (!rot) return;
#pragma unroll
          for (int j = 0; j < CH; ++j) {
            const int i0 = INTER ? 2 * j : j, i1 = INTER ? 2 * j + 1 : CH + j;
            const float p = w[i0], q = w[i1], si = sign * sn[j];
            w[i0] = p * cs[j] - q * si;
            w[i1] = p * si + q * cs[j];
          }
        };
        if (BWD) rotate(d, -1.f);
        float ss = 0.f, su = 0.f;
        if (NORM) {
#pragma unroll
          for (int i = 0; i < 2 * CH; ++i) {
            ss = fmaf(v[i], v[i], ss);
            if (BWD) su = fmaf(d[i] * gm[i], v[i], su);
          }
          for (int o = G / 2; o; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (BWD) su += __shfl_xor_sync(0xffffffffu, su, o);
          }
          const float rstd = 1.f / sqrtf(ss * inv_dh + a.eps);
          if (!BWD) {
#pragma unroll
            for (int i = 0; i < 2 * CH; ++i) v[i] = v[i] * rstd * gm[i];
          } else {
            const float m = su * rstd * inv_dh;
#pragma unroll
            for (int i = 0; i < 2 * CH; ++i) {
              const float hh = v[i] * rstd;
              if (on) dg[i] = fmaf(d[i], hh, dg[i]);
              d[i] = rstd * (d[i] * gm[i] - hh * m);
            }
          }
        }
        if (!BWD) rotate(v, 1.f);
        if (on) {
          Chunk<T, CH> o;
          o.put(BWD ? d : v);
          o.store(y + (long long)token * s.yp + (long long)h * a.dh, o0, o1);
        }
      }
    }
  }
  if (BWD && NORM && s.part) {  // the CTA's sums of dgamma, in the order of warps and lanes
#pragma unroll
    for (int i = 0; i < 2 * CH; ++i) red[(warp * 2 * CH + i) * 32 + lane] = dg[i];
    __syncthreads();
    for (int e = t; e < 2 * CH * G; e += kThreads) {
      const int i = e / G, cc = e - i * G;
      if (cc >= a.dh / (2 * CH)) continue;
      float sum = 0.f;
      for (int w = 0; w < kWarps; ++w)
        for (int l = cc; l < 32; l += G) sum += red[(w * 2 * CH + i) * 32 + l];
      const bool r = cc < pr;
      const int tl = 2 * a.half + 2 * CH * (cc - pr);
      const int b0 = r ? (INTER ? 2 * CH * cc : CH * cc) : tl;
      const int b1 = r && !INTER ? a.half + CH * cc : b0 + CH;
      s.part[(long long)cta * a.dh + (i < CH ? b0 + i : b1 + i - CH)] = sum;
    }
  }
}

// dgamma of both sides: the CTAs' partial sums, 32 columns per block, added in a fixed order.
constexpr int kSumRows = 16;
struct RopeSum {
  const float* part[2];
  int ctas[2];
  float* out[2];
};
__global__ void __launch_bounds__(32 * kSumRows) rope_sum_kernel(const RopeSum p, int dh, int accumulate) {
  __shared__ float sm[kSumRows][32];
  pdl_trigger();
  pdl_wait();
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5, k = blockIdx.y;
  float* out = p.out[k];
  if (!out) return;
  float sum = 0.f;
  if (col < dh)
    for (int i = r; i < p.ctas[k]; i += kSumRows) sum += p.part[k][(long long)i * dh + col];
  sm[r][threadIdx.x & 31] = sum;
  __syncthreads();
  if (r == 0 && col < dh) {
    sum = sm[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kSumRows; ++i) sum += sm[i][threadIdx.x];
    out[col] = accumulate ? out[col] + sum : sum;
  }
}

bool rope_ok(const poetx_rope* r) {
  if (r->head_dim < 8 || r->rot_dim < 8 || r->head_dim % 8 || r->rot_dim % 8 ||
      r->rot_dim > r->head_dim)
    return false;
  const bool wide = r->head_dim % 16 == 0 && r->rot_dim % 16 == 0;
  return r->head_dim <= (wide ? 512 : 256) && r->axes >= 1 && r->axes <= kMaxAxes;
}

template <typename T, int CH, bool BWD>
cudaError_t rope_launch(const RopeArgs& a, bool inter, bool norm, cudaStream_t s) {
  const dim3 grid(a.s[0].ctas + a.s[1].ctas), block(kThreads);
  if (inter)
    return norm ? launch_pdl(rope_kernel<T, CH, true, true, BWD>, grid, block, 0, s, a)
                : launch_pdl(rope_kernel<T, CH, true, false, BWD>, grid, block, 0, s, a);
  return norm ? launch_pdl(rope_kernel<T, CH, false, true, BWD>, grid, block, 0, s, a)
              : launch_pdl(rope_kernel<T, CH, false, false, BWD>, grid, block, 0, s, a);
}

// A side's tasks: whole tokens where they give every warp some, else a token's heads in parts.
void rope_tasks(Side* s, int N, int HW, int warps) {
  const int most = ceil_div(s->H, HW), want = ceil_div(warps, N);
  const int parts = want < most ? want : most;
  s->hs = ceil_div(ceil_div(s->H, parts), HW) * HW;
  s->parts = ceil_div(s->H, s->hs);
  s->tasks = (long long)N * s->parts;
}

template <bool BWD>
poetx_status rope_run(const poetx_rope* r, poetx_dtype dt, const int32_t* pos, int N,
                      const poetx_heads* q, const poetx_heads* k, int accumulate, void* ws,
                      size_t ws_bytes, cudaStream_t stream) {
  if (!r || (!q && !k) || N < 0 || (r->norm && !(r->eps >= 0.f))) return POETX_ERR_ARG;
  if (dt != POETX_F32 && dt != POETX_BF16) return POETX_ERR_DTYPE;
  if (!rope_ok(r)) return POETX_ERR_SHAPE;
  auto aligned4 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; };
  if (!aligned4(pos) || !aligned4(r->inv_freq) || !aligned4(r->axis) || (BWD && !aligned16(ws)))
    return POETX_ERR_ALIGN;
  const poetx_heads* side[2] = {q, k};
  bool sums = false, any = false;
  for (const poetx_heads* h : side) {
    if (!h) continue;
    if (h->heads < 0) return POETX_ERR_ARG;
    if (h->heads == 0) continue;
    any = true;
    const long long row = (long long)h->heads * r->head_dim;
    const bool reads_x = !BWD || r->norm;
    if ((reads_x && (h->x_pitch < row || h->x_pitch % 8)) || h->y_pitch < row || h->y_pitch % 8 ||
        (BWD && (h->dy_pitch < row || h->dy_pitch % 8)))
      return POETX_ERR_SHAPE;
    if (!aligned16(h->x) || !aligned16(h->y) || !aligned16(h->gamma) ||
        (BWD && (!aligned16(h->dy) || !aligned16(h->dgamma))))
      return POETX_ERR_ALIGN;
    if (N > 0 && ((reads_x && !h->x) || !h->y || (BWD && !h->dy))) return POETX_ERR_ARG;
    if (BWD && r->norm && h->dgamma) sums = true;
  }
  if (sums && N > 0) {
    if (!ws) return POETX_ERR_ARG;
    if (ws_bytes < poetx_qk_rope_bwd_workspace_bytes(r)) return POETX_ERR_WORKSPACE;
  }
  if (N == 0 || !any) {
    if (sums && !accumulate)
      for (const poetx_heads* h : side)
        if (h && h->heads && h->dgamma)
          POETX_CUDA_TRY(cudaMemsetAsync(h->dgamma, 0, (size_t)r->head_dim * 4, stream));
    return POETX_OK;
  }
  if (!pos || !r->inv_freq) return POETX_ERR_ARG;

  const int CH = r->head_dim % 16 == 0 && r->rot_dim % 16 == 0 ? 8 : 4;
  RopeArgs a{};
  a.pos = pos;
  a.inv_freq = r->inv_freq;
  a.axis = r->axis;
  a.N = N;
  a.axes = r->axes;
  a.dh = r->head_dim;
  a.half = r->rot_dim / 2;
  a.eps = r->eps;
  a.G = 1;
  while (a.G * 2 * CH < a.dh) a.G *= 2;
  const int max_ctas = kCtasPerSm * sm_count();
  const int heads = (q ? q->heads : 0) + (k ? k->heads : 0);
  float* part = static_cast<float*>(ws);
  RopeSum rs{};
  for (int i = 0; i < 2; ++i) {
    const poetx_heads* h = side[i];
    if (!h || h->heads == 0) continue;
    Side& s = a.s[i];
    s.x = h->x;
    s.dy = BWD ? h->dy : nullptr;
    s.y = h->y;
    s.gamma = h->gamma;
    s.xp = h->x_pitch;
    s.dyp = h->dy_pitch;
    s.yp = h->y_pitch;
    s.H = h->heads;
    // the CTAs in proportion to the sides' heads
    int ctas = (int)((long long)max_ctas * s.H / heads);
    if (ctas < 1) ctas = 1;
    rope_tasks(&s, N, 32 / a.G, ctas * kWarps);
    const int need = ceil_div(s.tasks, kWarps);
    s.ctas = need < ctas ? need : ctas;
    if (BWD && r->norm && h->dgamma) {
      s.part = part;
      rs.part[i] = part;
      rs.ctas[i] = s.ctas;
      rs.out[i] = h->dgamma;
      part += (size_t)s.ctas * a.dh;
    }
  }
  const bool inter = r->interleaved != 0, norm = r->norm != 0;
  cudaError_t e;
  if (dt == POETX_BF16)
    e = CH == 8 ? rope_launch<__nv_bfloat16, 8, BWD>(a, inter, norm, stream)
                : rope_launch<__nv_bfloat16, 4, BWD>(a, inter, norm, stream);
  else
    e = CH == 8 ? rope_launch<float, 8, BWD>(a, inter, norm, stream)
                : rope_launch<float, 4, BWD>(a, inter, norm, stream);
  POETX_CUDA_TRY(e);
  POETX_CUDA_TRY(cudaGetLastError());
  after_launch(stream, ST_ROPE);
  if (sums) {
    POETX_CUDA_TRY(launch_pdl(rope_sum_kernel, dim3((a.dh + 31) / 32, 2), dim3(32 * kSumRows), 0, stream,
                              rs, a.dh, accumulate));
    POETX_CUDA_TRY(cudaGetLastError());
    after_launch(stream, ST_ROPE);
  }
  return POETX_OK;
}

}  // namespace
}  // namespace poetx

using namespace poetx;

extern "C" poetx_status poetx_qk_rope_fwd(const poetx_rope* r, poetx_dtype dt, const int32_t* pos, int N,
                                          const poetx_heads* q, const poetx_heads* k,
                                          cudaStream_t stream) {
  return rope_run<false>(r, dt, pos, N, q, k, 0, nullptr, 0, stream);
}

extern "C" size_t poetx_qk_rope_bwd_workspace_bytes(const poetx_rope* r) {
  if (!r || !rope_ok(r)) return 0;
  return align_up((size_t)(kCtasPerSm * sm_count() + 2) * r->head_dim * sizeof(float), 256);
}

extern "C" poetx_status poetx_qk_rope_bwd(const poetx_rope* r, poetx_dtype dt, const int32_t* pos, int N,
                                          const poetx_heads* q, const poetx_heads* k, int accumulate,
                                          void* ws, size_t ws_bytes, cudaStream_t stream) {
  return rope_run<true>(r, dt, pos, N, q, k, accumulate, ws, ws_bytes, stream);
}
