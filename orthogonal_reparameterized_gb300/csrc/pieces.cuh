// fp32 values as three bf16 pieces, whose products on the tensor cores keep fp32's accuracy.
#pragma once

#include "common.cuh"

namespace poetx {

// Products of two bf16 pieces of dz with W or x: the second piece holds rests of either sign and zeros, so that
// where W or x is infinite its product is NaN or of the wrong sign, and the first piece's alone, an infinity or
// NaN, is the result.  (It is finite only where no factor was infinite.)
__device__ __forceinline__ float with_rest(float first, float rest) {
  return isfinite(first) ? first + rest : first;
}
// dW's sum is over both pieces.  An infinity of x meets every feature's dz, so that its column of dW is infinite or
// NaN in every row: a warp looks at one row of its staged 32 rows x 128 columns (two boxes of 64 columns with
// 128-byte swizzle, `box` bytes apart), each lane at four columns.  (Looking at every result cost the gradients of
// 33 rows 3 %.)
__device__ __forceinline__ bool staged_not_finite(const uint8_t* stg, int box, int lane) {
  const uint2 w =
      *reinterpret_cast<const uint2*>(stg + lane / 16 * box + ((lane % 16 / 2) << 4) + (lane & 1) * 8);
  const uint32_t top = __vmaxs2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
  return __any_sync(0xffffffffu, (top & 0xffffu) >= 0x7f80u || top >> 16 >= 0x7f80u);
}
// Then the warp looks for infinities in those columns of x, `col` on of D, eight at a time (dz's own infinities and
// NaN are in dW already: a step that has blown up must not end in this).  In a column with one, each lane
// (`mine`: its row is dW's) takes its result, and where that is NaN puts scale * the sum over the tokens of the
// first piece of dz (z + n pitch) by x (+ old) in its place.
__device__ __forceinline__ void first_piece_again(uint8_t* stg, int box, int lane, bool mine,
                                                  const __nv_bfloat16* z, long long pitch,
                                                  const __nv_bfloat16* x, int N, int D, int col, float scale,
                                                  const __nv_bfloat16* old) {
#pragma unroll 1
  for (int c8 = 0; c8 < 128 && col + c8 < D; c8 += 8) {
    uint32_t inf = 0;
#pragma unroll 1
    for (int n = lane; n < N; n += 32) {
      const uint4 w = *reinterpret_cast<const uint4*>(x + (long long)n * D + col + c8);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        inf |= ((u[i] & 0x7fffu) == 0x7f80u ? 1u : 0u) << (2 * i) |
               ((u[i] & 0x7fff0000u) == 0x7f800000u ? 2u : 0u) << (2 * i);
    }
#pragma unroll 1
    for (inf = __reduce_or_sync(0xffffffffu, inf); inf; inf &= inf - 1) {
      const int c = c8 + __ffs(inf) - 1;
      __nv_bfloat16* const at =
          reinterpret_cast<__nv_bfloat16*>(stg + c / 64 * box + lane * 128 + (((c % 64 / 8) ^ (lane & 7)) << 4)) +
          c % 8;
      if (!mine || !isnan(__bfloat162float(*at))) continue;
      float s = 0.f;
#pragma unroll 8
      for (int n = 0; n < N; ++n)
        s = fmaf(__bfloat162float(z[n * pitch]), __bfloat162float(x[(long long)n * D + col + c]), s);
      s *= scale;
      if (old) s += __bfloat162float(old[col + c]);
      *at = __float2bfloat16_rn(s);
    }
  }
}

// Three bf16 pieces of v, whose sum it is.  An infinity goes into the third: the products take the third piece
// with the other operand's first alone, so that it meets each number once, with that number's own sign (inf - inf
// in the split and inf times a rest of either sign would make NaN of a plain infinity).  Its first piece is its sign
// as a 1, for an infinity of the other operand: zero would make NaN of inf times inf.  A NaN is the third piece
// with zeros before it.  A finite value that would round to infinity is cut off at bf16's largest.
constexpr float kBf16Max = 0x1.fep127f;
template <bool CHECK = true>
__device__ __forceinline__ void split3(float v, __nv_bfloat16 (&o)[3]) {
  o[0] = __float2bfloat16_rn(v);
  if (CHECK && !(fabsf(v) <= kBf16Max)) {
    if (!isfinite(v)) {
      o[0] = __float2bfloat16_rn(isnan(v) ? 0.f : copysignf(1.f, v));
      o[1] = __float2bfloat16_rn(0.f);
      o[2] = __float2bfloat16_rn(v);
      return;
    }
    o[0] = __float2bfloat16_rz(v);
  }
  v -= __bfloat162float(o[0]);
  o[1] = __float2bfloat16_rn(v);
  v -= __bfloat162float(o[1]);
  o[2] = __float2bfloat16_rn(v);
}

// The pieces of four neighbouring values, to d[0], d[1] and d[2].
__device__ __forceinline__ void store3(float4 w, __nv_bfloat16* const (&d)[3]) {
  __nv_bfloat16 o[4][3];
  if (fabsf(w.x) + fabsf(w.y) + fabsf(w.z) + fabsf(w.w) <= kBf16Max) {  // (false for a NaN)
    split3<false>(w.x, o[0]);
    split3<false>(w.y, o[1]);
    split3<false>(w.z, o[2]);
    split3<false>(w.w, o[3]);
  } else {
    split3(w.x, o[0]);
    split3(w.y, o[1]);
    split3(w.z, o[2]);
    split3(w.w, o[3]);
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const __nv_bfloat162 lo = __halves2bfloat162(o[0][k], o[1][k]);
    const __nv_bfloat162 hi = __halves2bfloat162(o[2][k], o[3][k]);
    *reinterpret_cast<uint2*>(d[k]) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                 *reinterpret_cast<const uint32_t*>(&hi));
  }
}

// Two fp32 arrays (of quads * 4 values; the second may be empty) and where their pieces go.
struct SplitArray {
  const float4* src;
  long long quads;
  __nv_bfloat16* dst[3];
};
inline SplitArray split_of(const float* src, long long count, uint8_t* dst, size_t step) {
  SplitArray a{reinterpret_cast<const float4*>(src), count / 4, {}};
  for (int j = 0; j < 3; ++j) a.dst[j] = reinterpret_cast<__nv_bfloat16*>(dst + j * step);
  return a;
}

// The pieces of both arrays, the share of thread `t` of `step`.
__device__ __forceinline__ void split_arrays(const SplitArray& a, const SplitArray& b, long long t,
                                             long long step) {
  constexpr int U = 4;  // loads in flight per thread
  const long long n = a.quads + b.quads;
  for (long long i0 = t; i0 < n; i0 += U * step) {
    float4 w[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const long long i = i0 + k * step;
      if (i < n) w[k] = i < a.quads ? a.src[i] : b.src[i - a.quads];
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const long long i = i0 + k * step;
      if (i >= n) break;
      const bool first = i < a.quads;
      const long long at = 4 * (first ? i : i - a.quads);
      __nv_bfloat16* d[3];
#pragma unroll
      for (int j = 0; j < 3; ++j) d[j] = (first ? a.dst[j] : b.dst[j]) + at;
      store3(w[k], d);
    }
  }
}

}  // namespace poetx
