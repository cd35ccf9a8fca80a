// The gated feed-forward block (ffn.cu) for so few rows that its time is W's way through the SMs, on the CUDA
// cores (fp32, and the forward of one to four bf16 rows):
//
//   forward:    z = x W^T, then h = a(g) u, or dz = [dh u a'(g) | dh a(g)] from the sums
//   gradients:  dx = dz W,  dW = dz^T x
//
// Forward: a warp has the gate and value rows of two features, its lanes every 32nd float4 of them, and
// multiplies them with up to eight tokens' x from shared memory (or L1); more tokens are further warps of the
// same CTA (up to 32; beyond that further CTAs), which find W's lines in L1.  The sums of a warp's 4 x 8
// products are joined by halving: in each of five steps a lane gives half of its sums away and keeps the
// other half, so that 31 shuffles leave one sum per lane.  One row of 4096 x 14336: 470 MB in 66.8 us (7.0
// TB/s), eight 70 us; sixteen of 2048 x 5632 28.5 us (92 MB: shared memory bounds it, 128 bytes of x for each
// of W's 64 that are copied in and read; the tensor cores with W in three pieces 124 us).
//
// Gradients: both products in one pass over W's rows, which reads a row and writes the same row of dW.  A
// lane has four columns with x's values and dx's sums for every token in registers, a warp an equal share of
// the rows, and a row costs 2 N multiply-adds per column and no exchange; dz's values come from shared
// memory, where the warp lays those of its next eight rows.  Each thread copies its own bytes of the next
// eight rows ahead (with a ring of registers instead sixteen rows took 92 us, not 48: a wait for one of
// several loads in flight is a wait for all of them).  The warps' sums of dx are joined in shared memory, the
// CTAs' by the head's kernel for partial sums.  Sixteen rows of 2048 x 5632: 48 us (115 on the tensor cores).
#include <algorithm>

#include "common.cuh"
#include "gated.cuh"
#include "kernels.h"

namespace poetx {
namespace {

// ---------------------------------------------------------------- forward
// Warps of a CTA.  RING: all of x is in the shared memory of one CTA per SM, and so many steps of 128 columns
// of a warp's rows of W are on their way there; 0: a warp reads both through L1.
constexpr int fwd_warps(int ring) { return ring ? 12 : 4; }
constexpr int kGroup = 8;  // tokens of a warp at most
constexpr int kBlock = 32;  // tokens of a CTA at most
constexpr int kStepBytes = 4 * 512;  // a warp's 128 columns of four rows
constexpr size_t ring_bytes(int ring) { return (size_t)fwd_warps(ring) * ring * kStepBytes; }
constexpr size_t x_room(int ring) { return 226 * 1024 - ring_bytes(ring); }

struct FwdArgs {
  RowsForward c;
  int groups;  // of a block's tokens, at most four
  int x_bytes;  // of a block (RING)
  Act act;
};

// 16 bytes of a bf16 row in pairs of columns.
__device__ __forceinline__ void unpack(const uint4& w, float2 (&v)[4]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}

// Two features' sums for the group's tokens.
template <typename T, int NT, int RING>
__device__ __forceinline__ void rows_fwd_unit(const RowsForward& c, Act act, int f0, int n0, int lane,
                                              const float4* x_here, const uint8_t* ring) {
  static_assert(sizeof(T) == 4 || RING == 0, "bf16: through L1");
  float2 acc[4][NT] = {};
  if constexpr (RING > 0) {
    const int quads = c.D / 4;
    // the lane's columns are lane * 4 and every 128th from there; it copies its own bytes and reads them itself
    const int steps = (quads - lane + 31) / 32;
    const uint32_t ring_at = smem_u32(ring);
    const float4* const g = static_cast<const float4*>(c.W) + (long long)f0 * quads + lane;
    const float4* const u = g + (long long)c.F * quads;
    auto request = [&](int k) {  // two gate rows, two value rows
      if (k < steps) {
        const uint32_t at = ring_at + k % RING * kStepBytes;
        copy_async<16>(at, g + 32 * k);
        copy_async<16>(at + 512, g + 32 * k + quads);
        copy_async<16>(at + 1024, u + 32 * k);
        copy_async<16>(at + 1536, u + 32 * k + quads);
      }
      copy_commit();
    };
#pragma unroll
    for (int k = 0; k < RING - 1; ++k) request(k);
    int x_at[NT];  // (a token beyond the last: the last one's, and its sums are not stored)
#pragma unroll
    for (int n = 0; n < NT; ++n) x_at[n] = min(n0 + n, c.N - 1) * quads + lane;
    for (int k = 0; k < steps; ++k) {
      request(k + RING - 1);
      copy_wait<RING - 1>();
      float4 wv[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        wv[r] = *reinterpret_cast<const float4*>(ring + k % RING * kStepBytes + 512 * r);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float4 xv = x_here[x_at[n] + 32 * k];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          acc[r][n] = fma2(make_float2(wv[r].x, wv[r].y), make_float2(xv.x, xv.y), acc[r][n]);
          acc[r][n] = fma2(make_float2(wv[r].z, wv[r].w), make_float2(xv.z, xv.w), acc[r][n]);
        }
      }
    }
    copy_wait<0>();
  } else if constexpr (sizeof(T) == 4) {
    const int quads = c.D / 4;
    const float4* w[4];  // two gate rows, two value rows
#pragma unroll
    for (int r = 0; r < 4; ++r)
      w[r] = static_cast<const float4*>(c.W) + (long long)(f0 + (r & 1) + (r >> 1) * c.F) * quads;
    const float4* x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
      x[n] = static_cast<const float4*>(c.x) + (long long)min(n0 + n, c.N - 1) * quads;
    constexpr int U = 2;
    for (int q0 = lane; q0 < quads; q0 += 32 * U) {
      float4 wv[U][4];
#pragma unroll
      for (int k = 0; k < U; ++k)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (q0 + 32 * k < quads) wv[k][r] = w[r][q0 + 32 * k];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (q0 + 32 * k >= quads) break;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float4 xv = x[n][q0 + 32 * k];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            acc[r][n] = fma2(make_float2(wv[k][r].x, wv[k][r].y), make_float2(xv.x, xv.y), acc[r][n]);
            acc[r][n] = fma2(make_float2(wv[k][r].z, wv[k][r].w), make_float2(xv.z, xv.w), acc[r][n]);
          }
        }
      }
    }
  } else {
    constexpr int P = 4;  // pairs of columns in 16 bytes
    const int vecs = c.D / 8;
    const uint4* w[4];  // two gate rows, two value rows
#pragma unroll
    for (int r = 0; r < 4; ++r)
      w[r] = static_cast<const uint4*>(c.W) + (long long)(f0 + (r & 1) + (r >> 1) * c.F) * vecs;
    const uint4* x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
      x[n] = static_cast<const uint4*>(c.x) + (long long)min(n0 + n, c.N - 1) * vecs;
    constexpr int U = 2;
    for (int q0 = lane; q0 < vecs; q0 += 32 * U) {
      uint4 wv[U][4];
#pragma unroll
      for (int k = 0; k < U; ++k)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (q0 + 32 * k < vecs) wv[k][r] = w[r][q0 + 32 * k];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (q0 + 32 * k >= vecs) break;
        float2 wp[4][P];
#pragma unroll
        for (int r = 0; r < 4; ++r) unpack(wv[k][r], wp[r]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float2 xp[P];
          unpack(x[n][q0 + 32 * k], xp);
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < P; ++j) acc[r][n] = fma2(wp[r][j], xp[j], acc[r][n]);
        }
      }
    }
  }
  constexpr int V = 4 * NT;
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = acc[i / NT][i % NT].x + acc[i / NT][i % NT].y;
#pragma unroll
  for (int o = 16, left = V / 2; o; o >>= 1, left >>= 1) {
    if (left) {
      const bool upper = lane & o;
#pragma unroll
      for (int i = 0; i < left; ++i) {
        const float give = upper ? v[i] : v[i + left], keep = upper ? v[i + left] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
  // sum i (of V, gates in the lower half) lies in the lanes from i * 32 / V on
  const float g = v[0], u = __shfl_xor_sync(0xffffffffu, g, 16);
  const int i = lane * V / 32, f = f0 + i / NT, n = n0 + i % NT;
  if (lane >= 16 || lane % (32 / V) || n >= c.N) return;
  constexpr bool F32 = sizeof(T) == 4;
  const long long at = (long long)n * c.z_pitch + f, at_h = (long long)n * c.F + f;
  T* const z = static_cast<T*>(c.z);
  if (c.dh) {
    const float2 d = gated_grad<F32>(g, u, (float)static_cast<const T*>(c.dh)[at_h], act);
    const T a = T(d.x), b = T(d.y);
    z[at] = a;
    z[at + c.F] = b;
    if constexpr (!F32) {
      static_cast<T*>(c.z2)[at] = T(rest_of(d.x, a));
      static_cast<T*>(c.z2)[at + c.F] = T(rest_of(d.y, b));
    }
    return;
  }
  if (c.h) static_cast<T*>(c.h)[at_h] = T(gated<F32>(g, u, act));
  if (z) {
    z[at] = T(g);
    z[at + c.F] = T(u);
  }
}

// CTAs of an SM: through L1 as many as the registers can be held to.  (Eight fp32 tokens, 16 x 4096 x 14336:
// two 221 us, three 190, four 261; one bf16 token, 4096 x 8192: six 22.4, five 27.5.)
constexpr int fwd_ctas(int NT, int ring) { return ring ? 1 : (NT == 1 ? 6 : (NT == 2 ? 5 : 3)); }
template <typename T, int NT, int RING>
__global__ void __launch_bounds__(32 * fwd_warps(RING), fwd_ctas(NT, RING))
    rows_fwd_kernel(const FwdArgs p) {
  extern __shared__ __align__(16) float4 x_here[];
  pdl_trigger();
  pdl_wait();
  RowsForward c = p.c;
  if constexpr (RING > 0) {  // the block's tokens (through L1 there is one block)
    const long long t0 = (long long)blockIdx.y * kBlock;
    c.x = static_cast<const T*>(c.x) + t0 * c.D;
    if (c.h) c.h = static_cast<T*>(c.h) + t0 * c.F;
    if (c.z) c.z = static_cast<T*>(c.z) + t0 * c.z_pitch;
    if (c.dh) c.dh = static_cast<const T*>(c.dh) + t0 * c.F;
    c.N = min(c.N - (int)t0, kBlock);
  }
  const int lane = threadIdx.x & 31;
  if (RING) {
    const int quads = c.D / 4;
    const float4* const x = static_cast<const float4*>(c.x);
    for (int i = threadIdx.x; i < c.N * quads; i += 32 * fwd_warps(RING))
      copy_async<16>(smem_u32(x_here + i), x + i);
    copy_commit();
    copy_wait<0>();
    __syncthreads();
  }
  // the groups of a pair side by side in one CTA: they meet W's lines in L1
  const int warp = threadIdx.x >> 5, teams = fwd_warps(RING) / p.groups, team = warp / p.groups;
  if (team >= teams || warp % p.groups * NT >= c.N) return;
  const int n0 = warp % p.groups * NT;
  const uint8_t* const ring =
      reinterpret_cast<const uint8_t*>(x_here) + p.x_bytes + warp * RING * kStepBytes + lane * 16;
  if (RING) {
    for (int pair = team * gridDim.x + blockIdx.x; 2 * pair < c.F; pair += teams * gridDim.x)
      rows_fwd_unit<T, NT, RING>(c, p.act, 2 * pair, n0, lane, x_here, ring);
  } else if (const int pair = blockIdx.x * teams + team; 2 * pair < c.F) {
    rows_fwd_unit<T, NT, RING>(c, p.act, 2 * pair, n0, lane, x_here, ring);
  }
}

// ---------------------------------------------------------------- gradients
constexpr int kGradWarps = 8;
constexpr int kBatch = 8;  // rows whose dz a warp has in shared memory

// CTAs of an SM, by the registers that a lane's four columns of x and dx take per token.  (Two columns and two
// CTAs for sixteen tokens: 56.8 us instead of 47.9 at 2048 x 5632.)
constexpr int grad_ctas(int NT) { return NT > 8 ? 1 : 2; }
// Shared memory of a CTA: two batches of W (and of dW), a batch's dz and the sums of dx of each warp.
constexpr int kSlot = 32 * 16;                   // a warp's bytes of a row
constexpr int kArray = 2 * kBatch * kSlot;
constexpr int grad_smem(int NT, bool add) {
  return kGradWarps * ((add ? 2 : 1) * kArray + kBatch * NT * (int)sizeof(float2) + NT * kSlot);
}

struct GradArgs {
  RowsGradients c;
  int tiles;   // of 32 lanes' columns
  int splits;  // CTAs over the rows
};

// ADD: dW is added to what is there.
template <int NT, bool ADD>
__global__ void __launch_bounds__(32 * kGradWarps, grad_ctas(NT)) rows_grad_kernel(const GradArgs p) {
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_trigger();
  pdl_wait();
  const RowsGradients& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x % p.tiles, split = blockIdx.x / p.tiles;
  const int col = (tile * 32 + lane) * 4;
  const bool mine = col < c.D, dx = c.dx != nullptr, dW = c.dW != nullptr;
  const long long part = (long long)split * kGradWarps + warp, parts = (long long)p.splits * kGradWarps;
  const int first = (int)(c.V * part / parts), end = (int)(c.V * (part + 1) / parts);

  float2 x[NT][2], acc[NT][2] = {};
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mine && n < c.N) v = *reinterpret_cast<const float4*>(c.x + (long long)n * c.D + col);
    x[n][0] = make_float2(v.x, v.y);
    x[n][1] = make_float2(v.z, v.w);
  }
  // a thread's own bytes of each row: it copies them a batch ahead and reads them itself (a lane without
  // columns: the last ones', and stores nothing)
  constexpr int kHalf = kBatch * kSlot;
  const int from = mine ? col : c.D - 4;
  uint8_t* const ring = smem + warp * (ADD ? 2 : 1) * kArray + lane * 16;
  const uint32_t ring_at = smem_u32(ring);
  const float* const W_at = (dx ? c.W : c.x) + from;
  float* const dW_at = c.dW + from;
  const long long step = dx ? c.D : 0;
  auto request = [&](int r, int half) {
    if (r < end) {
      const float* w = W_at + r * step;
      const float* g = dW_at + (long long)r * c.D;
      const bool whole = r + kBatch <= end;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (whole || r + k < end) {
          copy_async<16>(ring_at + half + k * kSlot, w);
          if (ADD) copy_async<16>(ring_at + kArray + half + k * kSlot, g);
        }
        w += step;
        g += c.D;
      }
    }
    copy_commit();
  };
  request(first, 0);
  // dz of a batch: lane's row lane % 8, tokens lane / 8 and every fourth one from there
  constexpr int M = (NT + 3) / 4;
  float v[M];
  auto fetch = [&](int r) {
    r += lane & 7;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int n = (lane >> 3) + 4 * m;
      v[m] = 0.f;
      if (n < c.N && r < end) v[m] = c.dz[(long long)n * c.V + r];
    }
  };
  constexpr int kRings = kGradWarps * (ADD ? 2 : 1) * kArray;
  float2* const dz = reinterpret_cast<float2*>(smem + kRings) + warp * kBatch * NT;
  fetch(first);
  int half = 0;
  for (int r0 = first; r0 < end; r0 += kBatch, half ^= kHalf) {
    __syncwarp();
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int n = (lane >> 3) + 4 * m;
      if (n < NT) dz[(lane & 7) * NT + n] = both(v[m]);
    }
    __syncwarp();
    fetch(r0 + kBatch);
    request(r0 + kBatch, half ^ kHalf);
    copy_wait<1>();
    float* out = dW_at + (long long)r0 * c.D;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (r0 + k >= end) break;
      const uint8_t* const slot = ring + half + k * kSlot;
      const float4 wv = *reinterpret_cast<const float4*>(slot);
      float4 g = make_float4(0.f, 0.f, 0.f, 0.f);
      if (ADD) g = *reinterpret_cast<const float4*>(slot + kArray);
      const float2 w[2] = {make_float2(wv.x, wv.y), make_float2(wv.z, wv.w)};
      float2 d[2] = {make_float2(g.x, g.y), make_float2(g.z, g.w)};
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        const float4 two = *reinterpret_cast<const float4*>(dz + k * NT + n);
        const float2 s0 = make_float2(two.x, two.y), s1 = make_float2(two.z, two.w);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          d[j] = fma2(s0, x[n][j], d[j]);
          acc[n][j] = fma2(s0, w[j], acc[n][j]);
          d[j] = fma2(s1, x[n + 1][j], d[j]);
          acc[n + 1][j] = fma2(s1, w[j], acc[n + 1][j]);
        }
      }
      if (mine && dW) *reinterpret_cast<float4*>(out) = make_float4(d[0].x, d[0].y, d[1].x, d[1].y);
      out += c.D;
    }
  }
  if (!dx) return;

  // [warp][token][column]
  float* const red = reinterpret_cast<float*>(smem + kRings + kGradWarps * kBatch * NT * sizeof(float2));
  constexpr int kRow = 32 * 4;
#pragma unroll
  for (int n = 0; n < NT; ++n)
    *reinterpret_cast<float4*>(red + (warp * NT + n) * kRow + lane * 4) =
        make_float4(acc[n][0].x, acc[n][0].y, acc[n][1].x, acc[n][1].y);
  __syncthreads();
  for (int i = threadIdx.x; i < NT * kRow / 4; i += 32 * kGradWarps) {
    const int n = i / (kRow / 4), q = i % (kRow / 4) * 4, at_col = tile * kRow + q;
    if (n >= c.N || at_col >= c.D) continue;
    float4 s = *reinterpret_cast<const float4*>(red + n * kRow + q);
#pragma unroll
    for (int k = 1; k < kGradWarps; ++k) {
      const float4 b = *reinterpret_cast<const float4*>(red + (k * NT + n) * kRow + q);
      s.x += b.x;
      s.y += b.y;
      s.z += b.z;
      s.w += b.w;
    }
    float* const out = p.splits > 1 ? c.dxp + (long long)split * c.N * c.D : c.dx;
    *reinterpret_cast<float4*>(out + (long long)n * c.D + at_col) = s;
  }
}

template <typename T, int NT, int RING>
poetx_status launch_fwd1(const FwdArgs& a, cudaStream_t s) {
  auto k = rows_fwd_kernel<T, NT, RING>;
  size_t smem = 0;
  if (RING) {
    static PerDevice<cudaError_t> attr;
    POETX_CUDA_TRY(allow_smem(attr, k, (int)(x_room(RING) + ring_bytes(RING))));
    smem = a.x_bytes + ring_bytes(RING);
  }
  const int blocks = ceil_div(a.c.N, kBlock), pairs = a.c.F / 2;
  const int grid = RING ? std::max(1, std::min(pairs, sm_count() / blocks))
                        : ceil_div(pairs, fwd_warps(RING) / a.groups);
  POETX_CUDA_TRY(launch_pdl(k, dim3(grid, blocks), dim3(32 * fwd_warps(RING)), smem, s, a));
  POETX_CUDA_TRY(cudaGetLastError());
  after_launch(s, ST_FFN_GEMM);
  return POETX_OK;
}
template <int NT>
poetx_status launch_fwd(FwdArgs a, cudaStream_t s) {
  const size_t x_bytes = (size_t)std::min(a.c.N, kBlock) * a.c.D * 4;
  // From three rows on x in shared memory is faster (2048 x 5632: two rows 19.2 us there and 15.9 through
  // L1, four 17.1 and 26.3, eight 18.1 and 27.2, sixteen 28.7 and 42.4), with four steps of W on their way, or
  // with two (20, 21 and 34 us) where x leaves no room for four; what does not fit goes through L1.
  if constexpr (NT > 2) {
    if (x_bytes <= x_room(2)) {
      a.x_bytes = (int)x_bytes;
      return x_bytes <= x_room(4) ? launch_fwd1<float, NT, 4>(a, s) : launch_fwd1<float, NT, 2>(a, s);
    }
  }
  return launch_fwd1<float, NT, 0>(a, s);
}

template <int NT, bool ADD>
poetx_status launch_grad1(const GradArgs& a, cudaStream_t s) {
  auto k = rows_grad_kernel<NT, ADD>;
  static PerDevice<cudaError_t> attr;
  POETX_CUDA_TRY(allow_smem(attr, k, grad_smem(NT, ADD)));
  POETX_CUDA_TRY(launch_pdl(k, dim3(a.tiles * a.splits), dim3(32 * kGradWarps), grad_smem(NT, ADD), s, a));
  POETX_CUDA_TRY(cudaGetLastError());
  after_launch(s, ST_FFN_GEMM);
  return POETX_OK;
}
template <int NT>
poetx_status launch_grad(const GradArgs& a, cudaStream_t s) {
  return a.c.dW && a.c.accumulate ? launch_grad1<NT, true>(a, s) : launch_grad1<NT, false>(a, s);
}

int tokens_of(int N) { return N <= 4 ? 4 : (N <= 8 ? 8 : 16); }
int tiles_of(int D) { return ceil_div(D, 32 * 4); }

}  // namespace

// CTAs over W's rows: as many as fill the SMs' places once or twice, whichever leaves fewer of them empty
// (2048 columns are 16 tiles: 9 splits fill 144 of 152 places, 19 all of two rounds), with sixteen rows to a
// warp at least.
int rows_splits(int N, int D, int V) {
  const int tiles = tiles_of(D), places = sm_count() * grad_ctas(tokens_of(N));
  const int one = places / tiles, two = 2 * places / tiles;
  int s = 2 * one * 100 < two * 97 ? two : one;
  const int most = V / (16 * kGradWarps);
  if (s > most) s = most;
  return s < 1 ? 1 : s;
}

// Beyond a block of tokens, with x in shared memory, the multiply-adds are the time (16 TFMA/s of whole
// blocks, a pair of features another 256 columns); on the tensor cores it is two launches, the split of W and
// a tile's K: 11 us + 2 F D / 577,000 + D / 40.  (64 x 1024 x 2816: 27.1 us here and 43.8 there, 90: 38.4
// and 44.2; 128 x 256 x 512: 6.2 and 18.2, 512: 16.0 and 18.4, 700: 21 and 18.3; 100 x 1024 x 64: 4.4 and 36.8;
// 100 x 64 x 2816: 15.1 and 13.4.)  Up to 32 rows are always
// here, also where x goes through L1 (33 x 4096 x 14336 438 us there, 32 here 344).
bool rows_forward_fits(int N, int D, int F) {
  if (N <= kRowsForward) return true;
  const double tokens = (double)align_up((size_t)N, kBlock), rows = 2.0 * F;
  return (size_t)kBlock * D * 4 <= x_room(2) &&
         tokens * rows * (D + 256) / 16e6 < 11 + rows * D / 577e3 + D / 40.0;
}

// One bf16 row is always here (4096 x 14336: 36.9 us, on the tensor cores 39.6; 1024 x 2816: 3.5 and 6.8), two
// to four of blocks whose W is small enough (two: 2048 x 5632 10.4 and 11.6 us, 4096 x 14336 43.5 and 39.5;
// four: 1024 x 4096 5.7 and 7.0, 1600 x 4264 9.9 and 9.5).
bool rows_forward_fits_bf16(int N, int D, int F) {
  const long long weights = 2ll * F * D;
  return N == 1 || (N == 2 && weights <= 3 << 23) || (N <= 4 && weights <= 1 << 23);
}

poetx_status rows_forward(const RowsForward& c, const Act& act, cudaStream_t s) {
  const int nt = c.N == 1 ? 1 : (c.N == 2 ? 2 : (c.N <= 4 ? 4 : kGroup));
  const int groups = ceil_div(std::min(c.N, kBlock), nt);
  const FwdArgs a{c, groups, 0, act};
  if (!c.f32) {
    using H = __nv_bfloat16;
    return nt == 1 ? launch_fwd1<H, 1, 0>(a, s)
                   : (nt == 2 ? launch_fwd1<H, 2, 0>(a, s) : launch_fwd1<H, 4, 0>(a, s));
  }
  switch (nt) {
    case 1: return launch_fwd<1>(a, s);
    case 2: return launch_fwd<2>(a, s);
    case 4: return launch_fwd<4>(a, s);
    default: return launch_fwd<kGroup>(a, s);
  }
}

poetx_status rows_gradients(const RowsGradients& c, cudaStream_t s) {
  const GradArgs a{c, tiles_of(c.D), rows_splits(c.N, c.D, c.V)};
  switch (tokens_of(c.N)) {
    case 4: POETX_TRY(launch_grad<4>(a, s)); break;
    case 8: POETX_TRY(launch_grad<8>(a, s)); break;
    default: POETX_TRY(launch_grad<16>(a, s));
  }
  if (!c.dx || a.splits == 1) return POETX_OK;
  const long long count = (long long)c.N * c.D;
  return sum_partials(true, c.dxp, a.splits, count, count, c.dx, s);
}

}  // namespace poetx
