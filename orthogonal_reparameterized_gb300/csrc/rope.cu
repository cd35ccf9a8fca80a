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
// use the same angles: a lane makes those of its CH pairs once per token and keeps them over the heads,
// multiplied by gamma where that saves instructions.  What is in flight waits in shared memory: each
// thread copies the chunks of its own next heads there asynchronously (one or two ahead) and is the only
// one to read them, so that no barrier is needed.
//
// 8192 x (32 + 8) heads of 128 in bf16: 168 MB in 32.6 us (5.1 TB/s; at 65536 tokens 6.0; without the norm
// 30.2), 4096 in fp32 the same bytes in 29.5 us; backward 4096 x (40 + 40) heads 252 MB in 45.4 us
// (5.5 TB/s).  What bounds it besides HBM is a launch's ramp and latency: some 200 instructions per warp
// and four heads, 0.55 issued per cycle and quarter of an SM.
//
// The angle is reduced in 64-bit fixed point: with f = inv_freq / 2 pi in units of 2^-64 turns (modulo a
// turn), pos * f modulo 2^64 is the angle modulo a turn, to 2^-32 turns at any int32 position for |inv_freq| <=
// 2 pi (an fp32 product of position and frequency has lost the angle's second decimal at position 100000).
// Its rounding to fp32 is up to 2^-26 turns, 9e-8 radians.

#include "common.cuh"
#include "kernels.h"

namespace poetx {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxHalf = 256;   // pairs of a head
constexpr int ctas_per_sm(int CH, bool both) { return (CH == 8 ? 3 : 4) - both; }  // (by registers)
// Items that a thread has in flight, by the pairs of a lane.  (More are slower: with 8192 x 40 heads of 128
// one takes 32.7 us, two 34.1, eight 35.2; at 65536 tokens 221 and 254; backward in bf16 one 50.6, two 45.3,
// four 48, in fp32 one 46.2, two 48.1.)
constexpr int ring_slots(int CH, bool both) { return both && CH == 8 ? 2 : 1; }
constexpr int kMostCtas = 3;  // per SM with dgamma's partial sums
constexpr int kMaxAxes = 8;

struct Side {
  const void* x;
  const void* dy;
  void* y;
  const float* gamma;
  float* part;              // backward: [ctas][dh] partial sums of dgamma (nullable)
  long long xp, dyp, yp;
  int H;
  int per_token;            // items of a token: an item is what a warp does at a time, 32 / G heads
  int ctas;
  int share, extra;         // items of a warp; the first `extra` warps have one more
  bool wide;                // the items' numbers take 64 bits
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

// f / 2 pi in units of 2^-64 turns, modulo a turn, to one such unit for |f| <= 2 pi: 1 / 2 pi in two doubles,
// the first's product with its rounding error (one double alone is 2^-53 turns off, which a position of 2^31
// makes 2^-22).  The magnitude's whole turns leave the first product without rounding; the sign comes last.
__device__ __forceinline__ unsigned long long turns_of(float f) {
  const double a = fabs((double)f), inv_hi = 0x1.45f306dc9c883p-3, inv_lo = -0x1.6b01ec5417056p-57;
  const double p = a * inv_hi, e = fma(a, inv_lo, fma(a, inv_hi, -p));
  // (e is below 2^-50 turns for such f; whole turns of a larger one leave it without rounding too)
  const unsigned long long t = __double2ull_rn((p - floor(p)) * 0x1p64) +
                               (unsigned long long)__double2ll_rn((e - rint(e)) * 0x1p64);
  return f < 0.f ? 0ull - t : t;
}

// A lane's chunk of one head in one array: CH first and CH second elements of its pairs.
template <typename T, int CH, bool INTER>
struct Chunk {
  static constexpr int BYTES = 2 * CH * (int)sizeof(T);
  static constexpr int UNIT = BYTES / 2 < 16 ? BYTES / 2 : 16;  // bytes of one copy
  static constexpr int UNITS = BYTES / UNIT, WORDS = BYTES / 4;
  // slot: the chunk's first unit of this thread; units are kThreads * UNIT apart (no bank conflicts)
  // (`far`: elements from the first to the second vector of the chunk)
  static __device__ __forceinline__ void fetch(uint32_t slot, const T* at, int far) {
#pragma unroll
    for (int k = 0; k < UNITS; ++k)
      copy_async<UNIT>(slot + k * kThreads * UNIT,
                       reinterpret_cast<const char*>(k < UNITS / 2 ? at : at + far) +
                           (k % (UNITS / 2)) * UNIT);
  }
  static __device__ __forceinline__ void read(const char* slot, uint32_t (&r)[WORDS]) {
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
      const char* at = slot + k * kThreads * UNIT;
      if constexpr (UNIT == 8) {
        const uint2 w = *reinterpret_cast<const uint2*>(at);
        r[2 * k] = w.x;
        r[2 * k + 1] = w.y;
      } else {
        const uint4 w = *reinterpret_cast<const uint4*>(at);
        r[4 * k] = w.x;
        r[4 * k + 1] = w.y;
        r[4 * k + 2] = w.z;
        r[4 * k + 3] = w.w;
      }
    }
  }
  // words as they lie in memory <-> the pairs' first and second elements, two by two
  static __device__ __forceinline__ void split(const uint32_t (&r)[WORDS], float2 (&a)[CH / 2],
                                               float2 (&b)[CH / 2]) {
    float v[2 * CH];
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      if constexpr (sizeof(T) == 2) {
        v[2 * i] = __uint_as_float(r[i] << 16);
        v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
      } else {
        v[i] = __uint_as_float(r[i]);
      }
    }
    pairs(v, a, b);
  }
  static __device__ __forceinline__ void pairs(const float (&v)[2 * CH], float2 (&a)[CH / 2],
                                               float2 (&b)[CH / 2]) {
#pragma unroll
    for (int j = 0; j < CH / 2; ++j) {
      a[j] = INTER ? make_float2(v[4 * j], v[4 * j + 2]) : make_float2(v[2 * j], v[2 * j + 1]);
      b[j] = INTER ? make_float2(v[4 * j + 1], v[4 * j + 3])
                   : make_float2(v[CH + 2 * j], v[CH + 2 * j + 1]);
    }
  }
  static __device__ __forceinline__ void store(T* to, int far, const float2 (&a)[CH / 2],
                                               const float2 (&b)[CH / 2]) {
    float v[2 * CH];
#pragma unroll
    for (int j = 0; j < CH / 2; ++j) {
      v[INTER ? 4 * j : 2 * j] = a[j].x;
      v[INTER ? 4 * j + 2 : 2 * j + 1] = a[j].y;
      v[INTER ? 4 * j + 1 : CH + 2 * j] = b[j].x;
      v[INTER ? 4 * j + 3 : CH + 2 * j + 1] = b[j].y;
    }
    uint32_t r[WORDS];
#pragma unroll
    for (int i = 0; i < WORDS; ++i)
      r[i] = sizeof(T) == 2 ? pack_bf16x2(v[2 * i], v[2 * i + 1]) : __float_as_uint(v[i]);
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
      char* at = reinterpret_cast<char*>(k < UNITS / 2 ? to : to + far) + (k % (UNITS / 2)) * UNIT;
      if constexpr (UNIT == 8)
        *reinterpret_cast<uint2*>(at) = make_uint2(r[2 * k], r[2 * k + 1]);
      else
        *reinterpret_cast<uint4*>(at) = make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
    }
  }
};
// Where a warp is in its items: how many are left, the token and the first head of the next one, and the
// thread's own chunk there in up to two arrays.
template <typename T>
struct Cursor {
  int left, token, h0;
  const T *p0, *p1;
};

// Sums over the G lanes of a head.
template <int n>
__device__ __forceinline__ void group_sum(float (&v)[n], int G) {
  auto add = [&](int o) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  };
  if (G == 8) {  // (most heads: 128 wide, or 64 in chunks of four pairs)
    add(4);
    add(2);
    add(1);
  } else {
    for (int o = G / 2; o; o >>= 1) add(o);
  }
}

template <typename T, int CH, bool INTER, bool NORM, bool BWD>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(CH, NORM && BWD))
    rope_kernel(const __grid_constant__ RopeArgs a) {
  using C = Chunk<T, CH, INTER>;
  constexpr bool BOTH = BWD && NORM;  // both x and dy are read
  constexpr int HEAD = C::BYTES * kThreads, SLOT = (BOTH ? 2 : 1) * HEAD;
  constexpr int SLOTS = ring_slots(CH, BOTH);
  constexpr int N2 = CH / 2;
  // [slot][array][unit][thread], then each warp's cosines and sines of its token [half]
  extern __shared__ __align__(16) char ring[];
  __shared__ unsigned long long turn[kMaxHalf];  // the frequencies in 2^-64 turns
  __shared__ int ax[kMaxHalf];                   // the pair's axis, -1: NaN
  __shared__ __align__(16) float gsm[NORM ? 2 * kMaxHalf : 4];
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const float freq = t < a.half ? a.inv_freq[t] : 0.f;
  const int axis = t < a.half && a.axis ? a.axis[t] : 0;
  const int which = (int)blockIdx.x >= a.s[0].ctas;
  const Side& s = a.s[which];
  const int cta = (int)blockIdx.x - (which ? a.s[0].ctas : 0);
  const int G = a.G, c = lane & (G - 1), sub = lane / G, HW = 32 / G, dh = a.dh, H = s.H;
  const int pr = a.half / CH;  // rotated chunks
  const bool mine = c < dh / (2 * CH), rot = c < pr;
  // its two vectors, half of the rotated (of the other) elements apart, so that the lanes of a head read
  // and write whole lines whatever the pairing (interleaved pairs in neighbouring vectors: 49 us, not 37)
  const int o0 = rot ? CH * c : 2 * a.half + CH * (c - pr);
  const int far = rot ? a.half : dh / 2 - a.half, ahead_by = HW * dh;
  const uint32_t ring_at = smem_u32(ring) + t * C::UNIT;
  char* const my_ring = ring + t * C::UNIT;
  float2* const angles = reinterpret_cast<float2*>(ring + SLOTS * SLOT) + warp * a.half;

  const T* const in0 = static_cast<const T*>(BWD && !NORM ? s.dy : s.x);
  const T* const in1 = BOTH ? static_cast<const T*>(s.dy) : nullptr;
  const long long pitch0 = BWD && !NORM ? s.dyp : s.xp;
  T* const y = static_cast<T*>(s.y);
  const int own = sub * dh + o0;  // the thread's chunk in the heads of an item
  // The warp's items: an equal share of all, one after the other, whatever tokens they belong to.
  Cursor<T> at, ahead;  // the heads being computed, the heads being fetched
  {
    const int w = cta * kWarps + warp;
    const long long first = (long long)w * s.share + min(w, s.extra);
    at.left = s.share + (w < s.extra);
    at.token = s.wide ? (int)(first / s.per_token) : (int)((uint32_t)first / (uint32_t)s.per_token);
    at.h0 = (int)(first - (long long)at.token * s.per_token) * HW;
    ahead = at;
    at.p0 = y + at.token * s.yp + (at.h0 * dh + own);
    ahead.p0 = in0 + at.token * pitch0 + (at.h0 * dh + own);
    ahead.p1 = BOTH ? in1 + at.token * s.dyp + (at.h0 * dh + own) : nullptr;
  }
  auto fetch = [&](int slot) {
    if (ahead.left > 0) {
      if (mine && ahead.h0 + sub < H) {
        C::fetch(ring_at + slot * SLOT, ahead.p0, far);
        if (BOTH) C::fetch(ring_at + slot * SLOT + HEAD, ahead.p1, far);
      }
      --ahead.left;
      ahead.h0 += HW;
      ahead.p0 += ahead_by;
      if (BOTH) ahead.p1 += ahead_by;
      if (ahead.h0 >= H) {
        ahead.h0 = 0;
        ++ahead.token;
        ahead.p0 = in0 + ahead.token * pitch0 + own;
        if (BOTH) ahead.p1 = in1 + ahead.token * s.dyp + own;
      }
    }
    copy_commit();
  };
#pragma unroll 1
  for (int i = 0; i < SLOTS; ++i) fetch(i);
  if (t < a.half) {
    turn[t] = turns_of(freq);
    ax[t] = isfinite(freq) && axis >= 0 && axis < a.axes ? axis : -1;
  }
  if (!mine)  // lanes beyond the head's width: zeros in the sums
    for (int i = 0; i < SLOTS * SLOT / (kThreads * C::UNIT); ++i) {
      if (C::UNIT == 8) *reinterpret_cast<uint2*>(my_ring + i * kThreads * C::UNIT) = make_uint2(0u, 0u);
      else *reinterpret_cast<uint4*>(my_ring + i * kThreads * C::UNIT) = make_uint4(0u, 0u, 0u, 0u);
    }
  if (NORM)
    for (int i = t; i < dh; i += kThreads) gsm[i] = s.gamma ? s.gamma[i] : 1.f;
  const float inv_dh = 1.f / (float)dh;
  __syncthreads();
  // gamma of the pairs' first and second elements (the forward reads it once per token)
  auto gamma2 = [&](float2 (&p)[N2], float2 (&q)[N2]) {
    float v[2 * CH];
    if (NORM && mine) {
#pragma unroll
      for (int i = 0; i < CH; i += 4) {
        const float4 w = *reinterpret_cast<const float4*>(gsm + o0 + i);
        const float4 z = *reinterpret_cast<const float4*>(gsm + o0 + far + i);
        v[i] = w.x, v[i + 1] = w.y, v[i + 2] = w.z, v[i + 3] = w.w;
        v[CH + i] = z.x, v[CH + i + 1] = z.y, v[CH + i + 2] = z.z, v[CH + i + 3] = z.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2 * CH; ++i) v[i] = 1.f;
    }
    C::pairs(v, p, q);
  };
  float2 ga[N2], gb[N2], dga[N2], dgb[N2];
  if (BOTH) {
    gamma2(ga, gb);
#pragma unroll
    for (int j = 0; j < N2; ++j) dga[j] = dgb[j] = both(0.f);
  }
  float2 cs[N2], sn[N2];  // of the token's angles
  // forward with the norm: gamma_a cos, -gamma_b sin, gamma_a sin, gamma_b cos
  float2 fa[N2], fb[N2], fc[N2], fd[N2];
  // the positions of the token, lane i those of axis i (read while the token before is worked on)
  int pos = lane < a.axes && at.left > 0 ? a.pos[(long long)lane * a.N + at.token] : 0;
  bool fresh = true;
  int slot = 0;
#pragma unroll 1
  for (; at.left > 0; --at.left) {
    if (fresh) {  // the token's angles, each made once by the warp
      __syncwarp();
      for (int i0 = 0; i0 < a.half; i0 += 32) {
        const int i = i0 + lane, k = i < a.half ? ax[i] : -1;
        const int p = __shfl_sync(0xffffffffu, pos, k < 0 ? 0 : k);
        if (i >= a.half) break;
        const unsigned long long ang = (unsigned long long)(long long)p * turn[i];
        // turns, in [-1/2, 1/2]: rounded to 2^-32, then to fp32
        const float h = (float)(int)((ang + (1ull << 31)) >> 32) * 0x1p-32f;
        float sv, cv;
        // bf16: the hardware's sine and cosine, within 2^-21 on (-pi, pi), far below the result's
        // rounding
        if (sizeof(T) == 2) __sincosf(h * 6.28318530717958647692f, &sv, &cv);
        else sincospif(2.f * h, &sv, &cv);
        if (k < 0) cv = sv = __int_as_float(0x7fc00000);
        angles[i] = make_float2(cv, sv);
      }
      if (lane < a.axes && at.token + 1 < a.N) pos = a.pos[(long long)lane * a.N + at.token + 1];
      __syncwarp();
      if (rot) {
#pragma unroll
        for (int j = 0; j < N2; ++j) {
          const int i = !INTER ? CH * c + 2 * j : CH / 2 * c + 2 * j + (j < N2 / 2 ? 0 : (a.half - CH) / 2);
          const float4 w = *reinterpret_cast<const float4*>(angles + i);
          cs[j] = make_float2(w.x, w.z);
          sn[j] = make_float2(w.y, w.w);
        }
      } else if (NORM && !BWD) {
#pragma unroll
        for (int j = 0; j < N2; ++j) cs[j] = both(1.f), sn[j] = both(0.f);
      }
      if (NORM && !BWD) {
        float2 p[N2], q[N2];
        gamma2(p, q);
#pragma unroll
        for (int j = 0; j < N2; ++j) {
          fa[j] = mul2(p[j], cs[j]);
          fb[j] = mul2(q[j], neg2(sn[j]));
          fc[j] = mul2(p[j], sn[j]);
          fd[j] = mul2(q[j], cs[j]);
        }
      }
    }
    copy_wait<SLOTS - 1>();
    float2 xa[N2], xb[N2];  // x (backward without the norm: dy)
    float2 da[N2], db[N2];  // the gradient of the rotated head, then of the normalised one
    {
      uint32_t r[C::WORDS];
      C::read(my_ring + slot * SLOT, r);
      C::split(r, xa, xb);
      if (BOTH) {
        C::read(my_ring + slot * SLOT + HEAD, r);
        C::split(r, da, db);
      }
    }
    float sum[BOTH ? 2 : 1];  // of x^2, and of u x
    if (NORM) {
      float2 sq = mul2(xa[0], xa[0]), sr = mul2(xb[0], xb[0]);
#pragma unroll
      for (int j = 1; j < N2; ++j) {
        sq = fma2(xa[j], xa[j], sq);
        sr = fma2(xb[j], xb[j], sr);
      }
      sq = add2(sq, sr);
      sum[0] = sq.x + sq.y;
    }
    if (BWD && rot) {
#pragma unroll
      for (int j = 0; j < N2; ++j) {
        const float2 p = BOTH ? da[j] : xa[j], q = BOTH ? db[j] : xb[j];
        da[j] = fma2(q, sn[j], mul2(p, cs[j]));
        db[j] = fma2(q, cs[j], mul2(p, neg2(sn[j])));
      }
    } else if (BWD && !NORM) {
#pragma unroll
      for (int j = 0; j < N2; ++j) {
        da[j] = xa[j];
        db[j] = xb[j];
      }
    }
    if constexpr (BOTH) {
      float2 sd = mul2(mul2(da[0], ga[0]), xa[0]), se = mul2(mul2(db[0], gb[0]), xb[0]);
#pragma unroll
      for (int j = 1; j < N2; ++j) {
        sd = fma2(mul2(da[j], ga[j]), xa[j], sd);
        se = fma2(mul2(db[j], gb[j]), xb[j], se);
      }
      sd = add2(sd, se);
      sum[1] = sd.x + sd.y;
    }
    fetch(slot);  // into the slot just read
    if (NORM) group_sum(sum, G);
    const float2 rstd = both(NORM ? rsqrtf(sum[0] * inv_dh + a.eps) : 1.f);
    const bool on = mine && at.h0 + sub < H;
    T* const out = const_cast<T*>(at.p0);
    if constexpr (!BWD) {
      if (rot) {
#pragma unroll
        for (int j = 0; j < N2; ++j) {
          const float2 p = xa[j], q = xb[j];
          if (NORM) {
            xa[j] = mul2(fma2(q, fb[j], mul2(p, fa[j])), rstd);
            xb[j] = mul2(fma2(q, fd[j], mul2(p, fc[j])), rstd);
          } else {
            xa[j] = fma2(q, neg2(sn[j]), mul2(p, cs[j]));
            xb[j] = fma2(q, cs[j], mul2(p, sn[j]));
          }
        }
      } else if (NORM) {  // (no product with a zero sine: the partner may be infinite)
#pragma unroll
        for (int j = 0; j < N2; ++j) {
          xa[j] = mul2(mul2(xa[j], fa[j]), rstd);
          xb[j] = mul2(mul2(xb[j], fd[j]), rstd);
        }
      }
      if (on) C::store(out, far, xa, xb);
    } else if (on) {
      if constexpr (NORM) {
        const float2 m = both(-sum[1] * rstd.x * inv_dh);
#pragma unroll
        for (int j = 0; j < N2; ++j) {
          const float2 ha = mul2(xa[j], rstd), hb = mul2(xb[j], rstd);
          dga[j] = fma2(da[j], ha, dga[j]);
          dgb[j] = fma2(db[j], hb, dgb[j]);
          da[j] = mul2(fma2(ha, m, mul2(da[j], ga[j])), rstd);
          db[j] = mul2(fma2(hb, m, mul2(db[j], gb[j])), rstd);
        }
      }
      C::store(out, far, da, db);
    }
    if (++slot == SLOTS) slot = 0;
    at.h0 += HW;
    at.p0 += ahead_by;
    fresh = at.h0 >= H;
    if (fresh) {
      at.h0 = 0;
      ++at.token;
      at.p0 = y + at.token * s.yp + own;
    }
  }
  if (BOTH && s.part) {  // the CTA's sums of dgamma, in the order of warps and lanes
    copy_wait<0>();
    __syncthreads();
    float* red = reinterpret_cast<float*>(ring);  // [warp][element of the chunk][lane]
#pragma unroll
    for (int j = 0; j < N2; ++j) {
      const float v[4] = {dga[j].x, dga[j].y, dgb[j].x, dgb[j].y};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        red[(warp * 2 * CH + (k < 2 ? 2 * j + k : CH + 2 * j + k - 2)) * 32 + lane] = v[k];
    }
    __syncthreads();
    for (int e = t; e < 2 * CH * G; e += kThreads) {
      const int i = e / G, cc = e - i * G;
      if (cc >= dh / (2 * CH)) continue;
      float sum = 0.f;
      for (int w = 0; w < kWarps; ++w)
        for (int l = cc; l < 32; l += G) sum += red[(w * 2 * CH + i) * 32 + l];
      const bool r = cc < pr;
      const int b0 = r ? CH * cc : 2 * a.half + CH * (cc - pr), b1 = b0 + (r ? a.half : dh / 2 - a.half);
      const int j = i < CH ? i : i - CH;  // pair of the chunk
      const int el = INTER ? (j < CH / 2 ? b0 : b1 - CH) + 2 * j + (i >= CH) : (i < CH ? b0 : b1) + j;
      s.part[(long long)cta * dh + el] = sum;
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

constexpr int rope_smem(int esz, int CH, bool both, int half) {
  const int ring = ring_slots(CH, both) * (both ? 2 : 1) * 2 * CH * esz * kThreads;
  const int red = both ? kWarps * 2 * CH * 32 * 4 : 0;
  return (ring > red ? ring : red) + kWarps * half * (int)sizeof(float2);
}
// CTAs that an SM holds: by the kernels' registers, and by shared memory (with 5 KB of tables each).
int rope_ctas(int esz, int CH, bool both, int half) {
  const int by_smem = 227 * 1024 / (rope_smem(esz, CH, both, half) + 6 * 1024);
  const int by_regs = ctas_per_sm(CH, both);
  return by_smem < by_regs ? by_smem : by_regs;
}

template <typename T, int CH, bool INTER, bool NORM, bool BWD>
cudaError_t rope_launch1(const RopeArgs& a, cudaStream_t s) {
  auto k = rope_kernel<T, CH, INTER, NORM, BWD>;
  static PerDevice<cudaError_t> attr;
  const cudaError_t e = allow_smem(attr, k, rope_smem(sizeof(T), CH, BWD && NORM, kMaxHalf));
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(a.s[0].ctas + a.s[1].ctas), dim3(kThreads),
                    rope_smem(sizeof(T), CH, BWD && NORM, a.half), s, a);
}
template <typename T, int CH, bool BWD>
cudaError_t rope_launch(const RopeArgs& a, bool inter, bool norm, cudaStream_t s) {
  if (inter)
    return norm ? rope_launch1<T, CH, true, true, BWD>(a, s) : rope_launch1<T, CH, true, false, BWD>(a, s);
  return norm ? rope_launch1<T, CH, false, true, BWD>(a, s) : rope_launch1<T, CH, false, false, BWD>(a, s);
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
    if (row > (1ll << 30)) return POETX_ERR_SHAPE;
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

  // a lane's vectors of 16 bytes, bf16 or fp32, where the widths allow (fp32 in vectors of 32 bytes, of
  // which each access takes half: 43 us for 29.8 at 4096 x 40 heads of 128)
  const bool wide = r->head_dim % 16 == 0 && r->rot_dim % 16 == 0;
  const int CH = wide && (dt == POETX_BF16 || r->head_dim > 256) ? 8 : 4;
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
  const int max_ctas = rope_ctas((int)dtype_size(dt), CH, BWD && r->norm, a.half) * sm_count();
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
    s.per_token = ceil_div(s.H, 32 / a.G);
    const long long items = (long long)N * s.per_token, need = (items + kWarps - 1) / kWarps;
    s.ctas = need < ctas ? (int)need : ctas;
    s.share = (int)(items / (s.ctas * kWarps));
    s.extra = (int)(items % (s.ctas * kWarps));
    s.wide = items > 0x7fffffffLL;
    if (BWD && r->norm && h->dgamma) {
      s.part = part;
      rs.part[i] = part;
      rs.ctas[i] = s.ctas;
      rs.out[i] = h->dgamma;
      part += (size_t)s.ctas * a.dh;
    }
  }
  if (rs.out[0] && rs.out[0] == rs.out[1]) {  // one gamma for both: k's partial sums follow q's
    rs.ctas[0] += rs.ctas[1];
    rs.out[1] = nullptr;
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
  return align_up((size_t)(kMostCtas * sm_count() + 2) * r->head_dim * sizeof(float), 256);
}

extern "C" poetx_status poetx_qk_rope_bwd(const poetx_rope* r, poetx_dtype dt, const int32_t* pos, int N,
                                          const poetx_heads* q, const poetx_heads* k, int accumulate,
                                          void* ws, size_t ws_bytes, cudaStream_t stream) {
  return rope_run<true>(r, dt, pos, N, q, k, accumulate, ws, ws_bytes, stream);
}
