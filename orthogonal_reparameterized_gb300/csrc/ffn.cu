// The gated feed-forward block: h = a(g) u of a gate g and a value u.
//
//   z = x W^T, W [2F, D]: g = z[:, :F], u = z[:, F:]
//   a(g) = g s, s = 1 / (1 + exp(-t));  SiLU: t = g;  GELU (tanh form): t = 2 sqrt(2 / pi) (g + 0.044715 g^3)
//   a'(g) = s + g s (1 - s) t'(g)
//   backward: dz = [dh u a'(g) | dh a(g)],  dx = dz W,  dW = dz^T x
//
// Forward: one product over W's rows taken in pairs.  A 256 x 256 tile of a 2-CTA pair has 128 gate rows
// of W (the even CTA's half of the B operand) beside the 128 value rows of the same features (the odd
// CTA's), so that a row of the accumulator holds both g and u of its features and the epilogue forms h
// from the fp32 sums; z is stored only where the backward wants it.  Backward: dz elementwise (from the
// kept z, or in the epilogue of the same product run again), then the two products of the linear head's
// gradients (head.cu), for which dz is what that head's is.  fp32 forwards of up to 32 rows (or more of small
// blocks) and gradients of up to 16, and bf16 forwards of one row (four of small blocks), are ffn_rows.cu's;
// bf16 gradients of up to 64 rows ffn_grad.cu's.
//
// The tensor core truncates when it adds into its fp32 accumulator (about 2^-24 of the sum per add of 16
// products, all in one direction), so after every `chunk` of K the partial tile moves into the epilogue's
// registers and is added there with IEEE adds: every 4096 of K in bf16 (256 adds, 1.5e-5, against the
// result's 2^-8); fp32 operands are split into three bf16 pieces, the six pairs of pieces above 2^-24
// multiplied, 256 of K per accumulator.
//
// Forward 8192 x 4096 x 14336 with z: 1.13-1.16 ms (1.66-1.70 PFLOP/s in a run of calls, at the board's power;
// tensor pipe 89 %).  Eight rows of 4096 x 14336: 235 MB of W in 39-40 us (6.0 TB/s).  Backward 4096 x 2048 x
// 8192 from kept z: dz 46 us (335 MB, 7.3 TB/s), products 299 us (1.84 PFLOP/s).
//
// Every mbarrier wait is bounded; on expiry the kernel records POETX_ERR_TIMEOUT, drains its own
// copies, frees its TMEM and returns.
#include <algorithm>

#include "common.cuh"
#include "gated.cuh"
#include "kernels.h"
#include "pieces.cuh"

namespace poetx {

// Site id of this file's bounded waits (file id x 10000 + source line).
constexpr int kSite = 8 * 10000;

namespace {

// ---------------------------------------------------------------- elementwise kernels
// Eight neighbouring elements.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const void* p, long long at) {
    w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, long long at) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    a = q[0];
    b = q[1];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
__device__ __forceinline__ void put8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = pack8(v);
}
__device__ __forceinline__ void put8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
// What the elementwise kernels read and write, in vectors of eight elements: vector i lies in row i / vpr
// (the quotient by a multiplication: fewer than 2^31 vectors), or all in one row (magic 0) where the rows
// follow each other.
struct GluArgs {
  const void *g, *u, *dh;
  void *a, *b;            // forward: h; backward: dg, du (dz's first piece)
  void *a2, *b2, *a3, *b3;  // dz's further pieces
  long long in_pitch, out_pitch;  // of g and u, of dg and du (h and dh: F)
  uint32_t vpr, magic, shift;
  long long vecs;
  Act act;
};
__device__ __forceinline__ uint32_t row_of(const GluArgs& p, uint32_t i) {
  return (uint32_t)((unsigned long long)i * p.magic >> p.shift);
}

constexpr int kGluThreads = 256;
constexpr int kGluUnroll = 4;  // vectors in flight per thread and array
// (fp32 pieces are arithmetic as well: one vector, 512 x 1024 x 2816 in fp32 68.5 -> 66.7 us)
constexpr int bwd_unroll(int pieces) { return pieces == 3 ? 1 : 2; }

template <typename T>
__global__ void __launch_bounds__(kGluThreads) glu_fwd_kernel(const GluArgs p) {
  pdl_trigger();
  pdl_wait();
  constexpr int U = sizeof(T) == 2 ? kGluUnroll : kGluUnroll / 2;
  const long long step = (long long)gridDim.x * kGluThreads;
  for (long long i0 = (long long)blockIdx.x * kGluThreads + threadIdx.x; i0 < p.vecs; i0 += U * step) {
    Eight<T> g[U], u[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const long long i = i0 + k * step;
      if (i < p.vecs) {
        const uint32_t r = row_of(p, (uint32_t)i);
        const long long at = r * p.in_pitch + 8 * (i - (long long)r * p.vpr);
        g[k].load(p.g, at);
        u[k].load(p.u, at);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const long long i = i0 + k * step;
      if (i >= p.vecs) break;
      float x[8], y[8];
      g[k].get(x);
      u[k].get(y);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = gated<sizeof(T) == 4>(x[j], y[j], p.act);
      put8(static_cast<T*>(p.a) + 8 * i, x);
    }
  }
}

// PIECES 0: dg and du of type T.  Otherwise they are dz's 2 or 3 bf16 pieces.
template <typename T, int PIECES>
__global__ void __launch_bounds__(kGluThreads) glu_bwd_kernel(const GluArgs p) {
  pdl_trigger();
  pdl_wait();
  constexpr int U = bwd_unroll(PIECES);
  const long long step = (long long)gridDim.x * kGluThreads;
  for (long long i0 = (long long)blockIdx.x * kGluThreads + threadIdx.x; i0 < p.vecs; i0 += U * step) {
    Eight<T> g[U], u[U], d[U];
    uint32_t row[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const long long i = i0 + k * step;
      if (i < p.vecs) {
        row[k] = row_of(p, (uint32_t)i);
        const long long at = row[k] * p.in_pitch + 8 * (i - (long long)row[k] * p.vpr);
        g[k].load(p.g, at);
        u[k].load(p.u, at);
        d[k].load(p.dh, 8 * i);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const long long i = i0 + k * step;
      if (i >= p.vecs) break;
      float x[8], y[8], w[8];
      g[k].get(x);
      u[k].get(y);
      d[k].get(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 o = gated_grad<sizeof(T) == 4>(x[j], y[j], w[j], p.act);
        x[j] = o.x;
        y[j] = o.y;
      }
      const long long at = row[k] * p.out_pitch + 8 * (i - (long long)row[k] * p.vpr);
      if constexpr (PIECES == 0) {
        put8(static_cast<T*>(p.a) + at, x);
        put8(static_cast<T*>(p.b) + at, y);
      } else if constexpr (PIECES == 2) {
        put8(static_cast<__nv_bfloat16*>(p.a) + at, x);
        put8(static_cast<__nv_bfloat16*>(p.b) + at, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] = rest_of(x[j], __float2bfloat16_rn(x[j]));
          y[j] = rest_of(y[j], __float2bfloat16_rn(y[j]));
        }
        put8(static_cast<__nv_bfloat16*>(p.a2) + at, x);
        put8(static_cast<__nv_bfloat16*>(p.b2) + at, y);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          __nv_bfloat16* const da[3] = {static_cast<__nv_bfloat16*>(p.a) + at + j,
                                        static_cast<__nv_bfloat16*>(p.a2) + at + j,
                                        static_cast<__nv_bfloat16*>(p.a3) + at + j};
          __nv_bfloat16* const db[3] = {static_cast<__nv_bfloat16*>(p.b) + at + j,
                                        static_cast<__nv_bfloat16*>(p.b2) + at + j,
                                        static_cast<__nv_bfloat16*>(p.b3) + at + j};
          store3(make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]), da);
          store3(make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]), db);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- the projections
constexpr int BM = 128;  // rows per CTA (256 per pair)
constexpr int BF = 128;  // features per pair tile: 128 gate and 128 value columns
constexpr int BK = 64;
constexpr int kStages = 5;
constexpr int kEpiWarps = 8;  // two per TMEM lane quarter, each 64 features
constexpr int kEpiWarp0 = 4;  // (whole warpgroups for the split of the registers)
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
// Registers: 168 a thread at the launch, of which the first warpgroup keeps 72 and the epilogue's get 216.
constexpr int kFewRegs = 72, kManyRegs = 216;
static_assert(kFewRegs * 128 + kManyRegs * 32 * kEpiWarps == 168 * kThreads, "registers");
constexpr uint32_t kABytes = BM * BK * 2;
constexpr uint32_t kStageBytes = 2 * kABytes;
constexpr uint32_t kStgBytes = 32 * 128;  // one epilogue warp's box: 32 rows of 128 bytes
constexpr int kBoxes = 2;                 // boxes of a warp in flight
constexpr int kBand = 16;                 // M tiles of a raster band (x's stripes stay in L2)
constexpr int kSmem = kStages * (int)kStageBytes + kEpiWarps * kBoxes * (int)kStgBytes + 1024 + 512;
static_assert(kSmem <= 227 * 1024, "ffn projections: shared memory");
constexpr int kSegs = 6;

struct FfnMaps {
  CUtensorMap a[3], g[3], u[3];  // x, W's gate rows, W's value rows (their pieces)
  CUtensorMap h;       // DZ: dh
  CUtensorMap zg, zu;  // DZ: dz's halves
};
struct FfnGemm {
  int tiles_m, tiles_f, num_tiles, num_kb;
  int chunk;  // K blocks per accumulator hand-over
  int M, F;
  int store_h, store_z;
  Act act;
  int* err;
  unsigned long long limit_ns;
};

__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          int* err, unsigned long long limit_ns, int site) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*abort_flag || !mbar_wait_bounded(bar, parity, err, limit_ns, site)) {
    *abort_flag = 1;
    return false;
  }
  return true;
}

// Tile t: bands of kBand row tiles, those fastest, so that a tile of W's rows serves a whole band.
__device__ __forceinline__ void tile_at(const FfnGemm& p, int t, int* mi, int* fi) {
  const int m0 = t / (kBand * p.tiles_f) * kBand, width = min(kBand, p.tiles_m - m0);
  const int q = t - m0 * p.tiles_f;
  *mi = m0 + q % width;
  *fi = q / width;
}

// Bands of 16 row tiles as in the head's products; five stages of 32 KB leave room for two boxes a warp.
// Warp 0 of each CTA loads its 128 rows of x and its 128 rows of W, one thread of the even CTA's warp 1
// issues the MMAs, warps 4-11 read the accumulators back (warp w: rows 32 (w % 4).. of the CTA's 128,
// features 64 ((w - 4) / 4).. of the tile's 128: their gates and their values).
// DZ: the backward without kept projections.  The epilogue turns the fp32 sums into dz with the warp's box of
// dh, which arrives by TMA in one of the warp's two staging boxes while the products run, so that the
// projections are neither rounded nor stored.
template <int SEGS, bool DZ>
__global__ void __launch_bounds__(kThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ FfnMaps maps, const __grid_constant__ FfnGemm p) {
  constexpr bool F32 = SEGS == kSegs;
  // fp32: the pairs of pieces, small ones first, so that the accumulator is small while they are added
  constexpr int8_t SEG_X[kSegs] = {1, 0, 2, 1, 0, 0}, SEG_W[kSegs] = {1, 2, 0, 0, 1, 0};
  constexpr uint32_t TMEM_COLS = 4 * BF;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* staging = smem + kStages * kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kEpiWarps * kBoxes * kStgBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;  // [2] accumulator written
  uint64_t* tempty = tfull + 2;       // [2] accumulator read by both CTAs' epilogue warps
  uint64_t* dfull = tempty + 2;       // [kEpiWarps] the warp's box of dh has landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dfull + kEpiWarps);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int crank = (int)cluster_ctarank();
  pdl_trigger();
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kEpiWarps);
    }
    for (int w = 0; w < kEpiWarps; ++w) mbar_init(&dfull[w], 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(crank ? &maps.u[0] : &maps.g[0]);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t smem_base = smem_u32(smem);
  pdl_wait();
  const int t0 = (int)blockIdx.x / 2, t_step = (int)gridDim.x / 2;
  auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
    return ring_wait(bar, parity, abort_flag, p.err, p.limit_ns, site);
  };

  if (warp < kEpiWarp0) {
    regs_give<kFewRegs>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------ TMA producer
      Ring<kStages> rg;
      bool ok = true;
      long long issued = 0;
      const uint32_t full0 = mapa_shared(full, 0);  // the even CTA's barriers
      const CUtensorMap* const wm = crank ? maps.u : maps.g;
      for (int t = t0; t < p.num_tiles && ok; t += t_step) {
        int mi, fi;
        tile_at(p, t, &mi, &fi);
        const int row = (2 * mi + crank) * BM, col = fi * BF;
        for (int c0 = 0; c0 < p.num_kb && ok; c0 += p.chunk) {
          const int len = min(p.num_kb - c0, p.chunk);
          int sg = 0, i = 0;  // a chunk's K blocks once per pair of pieces
          for (int j = 0; j < len * SEGS; ++j, rg.next(), ++issued) {
            if (!wait(&empty[rg.s], rg.ph ^ 1, kSite + __LINE__)) {
              ok = false;
              break;
            }
            uint8_t* dst = smem + rg.s * kStageBytes;
            if (crank == 0) mbar_arrive_expect_tx(&full[rg.s], 2 * kStageBytes);
            const uint32_t fb = full0 + rg.s * 8;
            const int k = (c0 + i) * BK;
            tma_load_2d_pair(dst, F32 ? &maps.a[SEG_X[sg]] : maps.a, fb, k, row);
            tma_load_2d_pair(dst + kABytes, F32 ? wm + SEG_W[sg] : wm, fb, k, col);
            if (++i == len) {
              i = 0;
              ++sg;
            }
          }
        }
      }
      // no copy may be in flight when the CTA exits: the MMAs release a stage after reading it
      for (long long j = issued - 1; j >= 0 && j >= issued - kStages; --j)
        mbar_wait_bounded(&empty[j % kStages], (uint32_t)((j / kStages) & 1), p.err, p.limit_ns,
                          kSite + __LINE__);
    } else if (warp == 1 && lane == 0 && crank == 0) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t IDESC = make_idesc(2 * BM, 2 * BF, false, false);
      Ring<kStages> rg;
      Ring<2> acc;
      bool any = false, ok = true;
      for (int t = t0; t < p.num_tiles && ok; t += t_step)
        for (int c0 = 0; c0 < p.num_kb && ok; c0 += p.chunk, acc.next()) {
          if (!wait(&tempty[acc.s], acc.ph ^ 1, kSite + __LINE__)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(acc.s * 2 * BF);
          const int blocks = min(p.num_kb - c0, p.chunk) * SEGS;
          for (int j = 0; j < blocks; ++j, rg.next()) {
            if (!wait(&full[rg.s], rg.ph, kSite + __LINE__)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a_base = smem_base + rg.s * kStageBytes;
            const uint64_t ad = make_sdesc(a_base, 16, 1024), bd = make_sdesc(a_base + kABytes, 16, 1024);
#pragma unroll
            for (int k = 0; k < BK / 16; ++k)
              umma_bf16_pair(d, ad + k * 2, bd + k * 2, IDESC, (j | k) != 0);
            umma_commit_pair(&empty[rg.s]);
          }
          if (!ok) break;
          umma_commit_pair(&tfull[acc.s]);
          any = true;
        }
      if (any) {  // TMEM is freed after the final barrier: wait for the last hand-over's MMAs
        const int last = acc.s ^ 1;
        mbar_wait_bounded(&tfull[last], last ? acc.ph ^ 1 : acc.ph, p.err, p.limit_ns, kSite + __LINE__);
      }
    }
  } else {
    regs_take<kManyRegs>();
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int fbeg = ((warp - kEpiWarp0) >> 2) * (BF / 2);
    uint8_t* stg = staging + (warp - kEpiWarp0) * kBoxes * kStgBytes;
    Ring<2> acc;
    uint64_t* dbar = &dfull[warp - kEpiWarp0];
    uint32_t dph = 0;
    int buf = 0;
    bool ok = true;
    for (int t = t0; t < p.num_tiles && ok; t += t_step) {
      int mi, fi;
      tile_at(p, t, &mi, &fi);
      const int row_w = (2 * mi + crank) * BM + q * 32;  // the warp's first row
      const int f0 = fi * BF + fbeg;
      const bool live = f0 < p.F && row_w < p.M;
      if (DZ && live && lane == 0) {
        bulk_wait_read<0>();  // the boxes of the tile before have been read
        mbar_arrive_expect_tx(dbar, kStgBytes);
        tma_load_2d(stg, &maps.h, dbar, f0, row_w);
      }
      float v[BF];  // 64 gates, then their 64 values
      for (int c0 = 0; c0 < p.num_kb; c0 += p.chunk, acc.next()) {
        const int a = acc.s;
        const bool got = wait(&tfull[a], acc.ph, kSite + __LINE__);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t ta = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * 2 * BF + fbeg);
#pragma unroll
        for (int j = 0; j < BF; j += 32) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(ta + (j < BF / 2 ? j : j + BF / 2), r);
          tmem_ld_wait();
          if (c0 == 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[j + i] = __uint_as_float(r[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 w = add2(make_float2(v[j + i], v[j + i + 1]),
                                    make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])));
              v[j + i] = w.x;
              v[j + i + 1] = w.y;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_tmem(mapa_shared(&tempty[a], 0));
      }
      if (DZ && live) {  // (also where the products were given up: the copy must have landed at the end)
        const bool got = mbar_wait_bounded(dbar, dph, p.err, p.limit_ns, kSite + __LINE__);
        dph ^= 1;
        if (!__all_sync(0xffffffffu, got)) {
          *abort_flag = 1;
          ok = false;
        }
      }
      if (!ok) break;
      if (!live) continue;
      // Stores by TMA: boxes of 32 rows x 128 bytes, 128-byte swizzle; rows and features outside the
      // tensor are clipped.
      auto box = [&](const CUtensorMap* map, int col, auto chunk) {  // chunk(i): 16 bytes i of the row
        uint8_t* at = stg + buf * kStgBytes;
        buf ^= 1;
        if (lane == 0) bulk_wait_read<kBoxes - 1>();  // the buffer's previous box has been read
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(at + lane * 128 + ((i ^ (lane & 7)) << 4)) = chunk(i);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(map, at, col, row_w);
          bulk_commit();
        }
      };
      auto put = [&](const CUtensorMap* map, const float* w) {  // 64 features
        if constexpr (F32) {
#pragma unroll
          for (int j = 0; j < BF / 2; j += 32)
            if (f0 + j < p.F)
              box(map, f0 + j, [&](int i) {
                const float* f = w + j + 4 * i;
                return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                  __float_as_uint(f[3]));
              });
        } else {
          box(map, f0, [&](int i) {
            const float* f = w + 8 * i;
            return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                              pack_bf16x2(f[6], f[7]));
          });
        }
      };
      if constexpr (DZ) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 w = *reinterpret_cast<const uint4*>(stg + lane * 128 + ((i ^ (lane & 7)) << 4));
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float d = __uint_as_float(j & 1 ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
            const float2 o = gated_grad<false>(v[8 * i + j], v[BF / 2 + 8 * i + j], d, p.act);
            v[8 * i + j] = o.x;
            v[BF / 2 + 8 * i + j] = o.y;
          }
        }
        buf = 1;  // (the first box into the buffer that dh is not in)
        put(&maps.zu, v + BF / 2);
        put(&maps.zg, v);
        continue;
      }
      if (p.store_z) {
        put(&maps.zg, v);
        put(&maps.zu, v + BF / 2);
      }
      if (p.store_h) {
#pragma unroll
        for (int i = 0; i < BF / 2; ++i) v[i] = gated<F32>(v[i], v[BF / 2 + i], p.act);
        put(&maps.h, v);
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// ---------------------------------------------------------------- few rows
// At most 128 rows (a token being served, a short step): bound by reading W once, so the roles are
// swapped.  W is the 128-row operand (one CTA per tile of `height` features, chosen so that every SM gets
// the same number of them), the NT (16 to 128) padded tokens are the columns, and nearly all of the shared
// memory is a ring of W tiles in flight.
//
// A box costs its issuing thread some 0.25 us whatever its size, so there are few of them: one box brings
// both halves' rows of several K blocks, and x's come from a thread of their own.  An MMA of 128 rows costs
// about as much for 16 tokens as for 64, so up to 64 features per tile the gate and the value rows are one
// operand (MERGED; the epilogue brings them together through shared memory), above that two accumulators
// side by side.  There neighbouring K blocks go to different accumulators (score_accs, added in fp32 by the
// epilogue), so that an MMA need not wait for the one before; D is at most 16384, at most 1024 adds into
// one (6e-5).
struct FfnScore {
  int tiles, height;  // height: a multiple of 8 (the swizzle's rows)
  int F, rows, stages;
  int kps, num_st;    // K blocks per stage, stages per tile
  int grouped;        // the maps are of groups of 64 columns (else kps is 1)
  __nv_bfloat16 *h, *z;  // [rows][F], [rows][z_pitch] (each nullable)
  const __nv_bfloat16* dh;  // [rows][F]: z and z2 are dz's two pieces (nullable)
  __nv_bfloat16* z2;
  long long z_pitch;
  Act act;
  int* err;
  unsigned long long limit_ns;
};
constexpr int kScoreRows = 128;
constexpr int kScoreMaxD = 16384;
constexpr int kScoreRing = 12;
constexpr int kScoreSmem = 220 * 1024;
// Sets of four epilogue warps, which take turns with the groups of 16 tokens.
constexpr int score_sets(int NT) { return NT >= 64 ? 2 : 1; }
constexpr int score_threads(int NT) { return 32 * (3 + 4 * score_sets(NT)); }
constexpr int kTurnPitch = 17;  // floats of a row of 16 tokens (MERGED)
constexpr int kTurnBytes = 128 * kTurnPitch * 4;  // of one set
int score_room(int NT, bool merged) {  // shared memory of the ring
  return kScoreSmem - 1024 - 512 - (int)kABytes - (merged ? score_sets(NT) * kTurnBytes : 0);
}
int score_stage_bytes(int NT, int height, int kps) { return kps * (2 * height + NT) * BK * 2; }
constexpr int score_accs(int NT, bool merged) {  // (two buffers of them in 512 columns)
  return !merged ? 1 : (NT <= 64 ? 4 : 2);
}
// The barrier of a set of four epilogue warps, with or without a vote.
__device__ __forceinline__ void bar_sync(int id) {
  asm volatile("barrier.sync %0, 128;" ::"r"(id) : "memory");
}
__device__ __forceinline__ int bar_all(int id, bool v) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\tbarrier.red.and.pred q, %1, 128, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(id), "r"((int)v)
      : "memory");
  return r;
}

template <int NT, bool MERGED>
__global__ void __launch_bounds__(score_threads(NT), 1)
    ffn_score_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                     const FfnScore p) {
  constexpr uint32_t IDESC = make_idesc(BM, NT, false, false);
  constexpr int SETS = score_sets(NT), XWARP = 2 + 4 * SETS;
  constexpr int ACCS = score_accs(NT, MERGED), COLS = (MERGED ? 1 : 2) * NT;  // columns of an accumulator
  constexpr uint32_t TMEM_COLS = 2 * ACCS * COLS;
  const uint32_t half = (uint32_t)p.height * BK * 2;  // one K block of gate (value) rows
  const uint32_t x_off = p.kps * 2 * half;
  const uint32_t stage = x_off + p.kps * NT * BK * 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  // (16 KB kept behind the last stage: the MMAs read 128 rows from its last K block's first)
  float* turn = reinterpret_cast<float*>(smem + p.stages * stage + kABytes);  // [128][kTurnPitch]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.stages * stage + kABytes +
                                               (MERGED ? SETS * kTurnBytes : 0));
  uint64_t* empty = full + kScoreRing;
  uint64_t* tfull = empty + kScoreRing;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 2);  // W's thread and x's
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 4 * SETS);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mw);
    tma_prefetch_desc(&mx);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t smem_base = smem_u32(smem);
  pdl_wait();
  auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
    return ring_wait(bar, parity, abort_flag, p.err, p.limit_ns, site);
  };
  int s = 0;
  uint32_t ph = 0;
  auto next = [&]() {
    if (++s == p.stages) {
      s = 0;
      ph ^= 1;
    }
  };
  if ((warp == 0 || warp == XWARP) && lane == 0) {
    const bool is_x = warp == XWARP;
    int issued = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x)
      for (int st = 0; st < p.num_st; ++st, next(), ++issued) {
        if (!wait(&empty[s], ph ^ 1, kSite + __LINE__)) {
          ok = false;
          break;
        }
        uint8_t* at = smem + s * stage;
        mbar_arrive_expect_tx(&full[s], is_x ? stage - x_off : x_off);
        if (is_x) {
          if (p.grouped) tma_load_3d(at + x_off, &mx, &full[s], 0, 0, st * p.kps);
          else tma_load_2d(at + x_off, &mx, &full[s], st * BK, 0);
        } else {
          if (p.grouped) tma_load_4d(at, &mw, &full[s], 0, t * p.height, 0, st * p.kps);
          else tma_load_3d(at, &mw, &full[s], st * BK, t * p.height, 0);
        }
      }
    // every copy has landed (of this thread, and where both went on, the other's)
    for (int j = issued - 1; j >= 0 && j >= issued - p.stages; --j)
      mbar_wait_bounded(&full[j % p.stages], (uint32_t)((j / p.stages) & 1), p.err, p.limit_ns,
                        kSite + __LINE__);
  } else if (warp == 1 && lane == 0) {
    Ring<2> acc;
    bool any = false, ok = true;
    for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x, acc.next()) {
      if (!wait(&tempty[acc.s], acc.ph ^ 1, kSite + __LINE__)) break;
      tc_fence_after();
      const uint32_t d0 = tmem_base + (uint32_t)(acc.s * ACCS * COLS);
      int kb = 0;
      for (int j = 0; j < p.num_st; ++j, next()) {
        if (!wait(&full[s], ph, kSite + __LINE__)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // (rows past the box's are whatever follows in shared memory: not looked at)
        const uint32_t base = smem_base + s * stage;
        for (int i = 0; i < p.kps; ++i, ++kb) {
          const uint32_t d = d0 + (uint32_t)(kb % ACCS * COLS);
          const uint64_t gd = make_sdesc(base + 2 * i * half, 16, 1024);
          const uint64_t ud = make_sdesc(base + (2 * i + 1) * half, 16, 1024);
          const uint64_t xd = make_sdesc(base + x_off + i * NT * BK * 2, 16, 1024);
#pragma unroll
          for (int k = 0; k < BK / 16; ++k) {
            umma_bf16(d, gd + k * 2, xd + k * 2, IDESC, kb >= ACCS || k != 0);
            if (!MERGED) umma_bf16(d + NT, ud + k * 2, xd + k * 2, IDESC, kb >= ACCS || k != 0);
          }
        }
        umma_commit(&empty[s]);
      }
      if (!ok) break;
      umma_commit(&tfull[acc.s]);
      any = true;
    }
    if (any) {
      const int last = acc.s ^ 1;
      mbar_wait_bounded(&tfull[last], last ? acc.ph ^ 1 : acc.ph, p.err, p.limit_ns, kSite + __LINE__);
    }
  } else if (warp >= 2 && warp < XWARP) {
    const int set = (warp - 2) >> 2, q = warp & 3;
    const int mine = q * 32 + lane;  // the thread's lane of the accumulators
    const int used = min(ACCS, p.num_st * p.kps);
    // h, z or dz of a feature and a token
    auto put = [&](long long f, int token, float g, float u, float d) {
      if (p.h) p.h[(long long)token * p.F + f] = __float2bfloat16_rn(gated<false>(g, u, p.act));
      if (!p.z) return;
      const long long at = (long long)token * p.z_pitch + f;
      const float2 o = p.dh ? gated_grad<false>(g, u, d, p.act) : make_float2(g, u);
      const __nv_bfloat16 a = __float2bfloat16_rn(o.x), b = __float2bfloat16_rn(o.y);
      p.z[at] = a;
      p.z[at + p.F] = b;
      if (p.dh) {
        p.z2[at] = __float2bfloat16_rn(rest_of(o.x, a));
        p.z2[at + p.F] = __float2bfloat16_rn(rest_of(o.y, b));
      }
    };
    // the values that a thread makes of 16 tokens, token << 8 | feature: all tokens of its own feature, or
    // (MERGED) eight of features and tokens in turn, features fastest
    constexpr int EACH = MERGED ? 8 : 16;
    int where[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int e = i * 128 + mine;
      if (MERGED) where[i] = e < 16 * p.height ? (e / p.height) << 8 | e % p.height : -1;
      else where[i] = mine < p.height ? i << 8 | mine : -1;
    }
    turn += set * 128 * kTurnPitch;
    Ring<2> acc;
    for (int t = blockIdx.x; t < p.tiles; t += gridDim.x, acc.next()) {
      const uint32_t ta = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc.s * ACCS * COLS);
      const long long f0 = (long long)t * p.height;
      float d[EACH], d_next[EACH];
      auto upstream = [&](int j) {  // dh of the thread's values, a group of tokens ahead of their use
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
          const int token = j + (where[i] >> 8);
          const long long f = f0 + (where[i] & 255);
          d_next[i] = where[i] >= 0 && f < p.F && token < p.rows
                          ? __bfloat162float(p.dh[(long long)token * p.F + f]) : 0.f;
        }
      };
      if (p.dh) upstream(16 * set);
      const bool got = wait(&tfull[acc.s], acc.ph, kSite + __LINE__);
      // (MERGED: all four warps go on or none, for their barrier)
      if (MERGED ? bar_all(1 + set, got) == 0 : !__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
#pragma unroll 1
      for (int j = 16 * set; j < NT && j < p.rows; j += 16 * SETS) {
        float g[16], u[16];
#pragma unroll
        for (int k = 0; k < ACCS; ++k) {
          if (k >= used) break;
          uint32_t r[16], v[16];
          tmem_ld_32x32b_x16(ta + k * COLS + j, r);
          if (!MERGED) tmem_ld_32x32b_x16(ta + k * COLS + NT + j, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            g[i] = k ? g[i] + __uint_as_float(r[i]) : __uint_as_float(r[i]);
            if (!MERGED) u[i] = k ? u[i] + __uint_as_float(v[i]) : __uint_as_float(v[i]);
          }
        }
        if (p.dh) {
#pragma unroll
          for (int i = 0; i < EACH; ++i) d[i] = d_next[i];
          upstream(j + 16 * SETS);
        }
        if (MERGED) {
#pragma unroll
          for (int i = 0; i < 16; ++i) turn[mine * kTurnPitch + i] = g[i];
          bar_sync(1 + set);
        }
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
          const int token = where[i] >> 8, in = where[i] & 255;
          if (where[i] < 0 || f0 + in >= p.F || j + token >= p.rows) continue;
          if (MERGED) {
            const float* at = turn + in * kTurnPitch + token;
            put(f0 + in, j + token, at[0], at[p.height * kTurnPitch], d[i]);
          } else {
            put(f0 + in, j + token, g[i], u[i], d[i]);
          }
        }
        if (MERGED) bar_sync(1 + set);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc.s]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ---------------------------------------------------------------- host side
// Launches an elementwise kernel over N rows of F elements (h, dh: rows of F), at most 2^31 - 1 vectors
// at a time; rows that follow each other in every array count as one.
struct GluCall {
  poetx_dtype dt;
  Act act;
  const void *g, *u, *dh;
  int N;
  long long F, in_pitch, out_pitch;
  void* out[6];  // as GluArgs' a, b, a2, b2, a3, b3
  int pieces;    // 0: outputs of type dt
};
poetx_status run_glu(const GluCall& c, cudaStream_t s) {
  const size_t esz = dtype_size(c.dt);
  const size_t osz = c.pieces ? 2 : esz;
  const bool flat = c.in_pitch == c.F && (!c.dh || c.out_pitch == c.F);
  const long long vpr = c.F / 8, most = 0x7fffffffLL / vpr;
  for (long long r0 = 0; r0 < c.N; r0 += most) {
    const long long rows = c.N - r0 < most ? c.N - r0 : most;
    GluArgs a{};
    const size_t in = (size_t)r0 * c.in_pitch * esz, out = (size_t)r0 * c.out_pitch * osz;
    a.g = static_cast<const uint8_t*>(c.g) + in;
    a.u = static_cast<const uint8_t*>(c.u) + in;
    a.dh = c.dh ? static_cast<const uint8_t*>(c.dh) + (size_t)r0 * c.F * esz : nullptr;
    void** dst[6] = {&a.a, &a.b, &a.a2, &a.b2, &a.a3, &a.b3};
    for (int i = 0; i < 6; ++i) *dst[i] = c.out[i] ? static_cast<uint8_t*>(c.out[i]) + out : nullptr;
    a.in_pitch = c.in_pitch;
    a.out_pitch = c.out_pitch;
    a.vecs = rows * vpr;
    a.vpr = (uint32_t)vpr;
    a.act = c.act;
    if (!flat) {
      // i / vpr for i < 2^31: with 2^l >= vpr and m = ceil(2^(31 + l) / vpr) < 2^32 the quotient is
      // (i m) >> (31 + l), the error m vpr - 2^(31 + l) < 2^l times i staying below 2^(31 + l)
      int l = 0;
      while ((1ll << l) < vpr) ++l;
      a.magic = (uint32_t)(((1ull << (31 + l)) + vpr - 1) / (unsigned long long)vpr);
      a.shift = 31 + l;
    }
    const int U = c.dh ? bwd_unroll(c.pieces) : (c.dt == POETX_BF16 ? kGluUnroll : kGluUnroll / 2);
    const dim3 grid(grid_for((a.vecs + U - 1) / U, kGluThreads)), block(kGluThreads);
    cudaError_t e;
    const bool b16 = c.dt == POETX_BF16;
    if (!c.dh)
      e = b16 ? launch_pdl(glu_fwd_kernel<__nv_bfloat16>, grid, block, 0, s, a)
              : launch_pdl(glu_fwd_kernel<float>, grid, block, 0, s, a);
    else if (c.pieces == 0)
      e = b16 ? launch_pdl(glu_bwd_kernel<__nv_bfloat16, 0>, grid, block, 0, s, a)
              : launch_pdl(glu_bwd_kernel<float, 0>, grid, block, 0, s, a);
    else if (c.pieces == 2)
      e = launch_pdl(glu_bwd_kernel<__nv_bfloat16, 2>, grid, block, 0, s, a);
    else
      e = launch_pdl(glu_bwd_kernel<float, 3>, grid, block, 0, s, a);
    POETX_CUDA_TRY(e);
    POETX_CUDA_TRY(cudaGetLastError());
    after_launch(s, ST_GLU);
  }
  return POETX_OK;
}

template <int NT, bool MERGED>
poetx_status score(const CUtensorMap& mw, const CUtensorMap& mx, FfnScore p, cudaStream_t s) {
  auto k = ffn_score_kernel<NT, MERGED>;
  static PerDevice<cudaError_t> attr;
  POETX_CUDA_TRY(allow_smem(attr, k, kScoreSmem));
  p.stages = score_room(NT, MERGED) / score_stage_bytes(NT, p.height, p.kps);
  if (p.stages > kScoreRing) p.stages = kScoreRing;
  p.err = device_error_word();
  p.limit_ns = kWaitLimitNs;
  const int grid = p.tiles < sm_count() ? p.tiles : sm_count();
  POETX_CUDA_TRY(launch_pdl(k, dim3(grid), dim3(score_threads(NT)), kScoreSmem, s, mw, mx, p));
  POETX_CUDA_TRY(cudaGetLastError());
  after_launch(s, ST_FFN_GEMM);
  return POETX_OK;
}

template <int SEGS, bool DZ>
poetx_status gemm(const FfnMaps& m, FfnGemm& p, cudaStream_t s) {
  auto k = ffn_gemm_kernel<SEGS, DZ>;
  static PerDevice<Clusters> setup;
  const Clusters c = allow_clusters(setup, k, sm_count() / 2 * 2, kThreads, kSmem, 2);
  POETX_CUDA_TRY(c.err);
  p.err = device_error_word();
  p.limit_ns = kWaitLimitNs;
  const int pairs = p.num_tiles < c.resident ? p.num_tiles : c.resident;
  POETX_CUDA_TRY(launch_pdl_cluster(k, dim3(2 * pairs), dim3(kThreads), kSmem, s, 2, m, p));
  POETX_CUDA_TRY(cudaGetLastError());
  after_launch(s, ST_FFN_GEMM);
  return POETX_OK;
}

bool shape_ok(poetx_dtype dt, int N, int D, int F) {
  return (dt == POETX_F32 || dt == POETX_BF16) && N >= 0 && D >= 8 && D % 8 == 0 && D <= (1 << 17) &&
         F >= 8 && F % 8 == 0 && F <= (1 << 21);
}
// The rows' tiles and W's together stay within what a launch counts.
bool tiles_ok(int N, int F) {
  return (long long)ceil_div(N, 2 * BM) * ceil_div(F, BF) <= 0x3fffffffLL;
}

// Bytes between the three pieces of an fp32 array of `count` values.
size_t piece_step(size_t count) { return align_up(count * 2, 1024); }

// What a projection leaves: h and / or z (each nullable), or with dh (bf16) dz in rows of `pitch` elements,
// in two pieces (z2) for few rows.
struct Outputs {
  void *h, *z;
  const void* dh;
  void* z2;
  long long pitch;  // of z
};
bool few_rows(int N, int D) { return N <= kScoreRows && D <= kScoreMaxD; }

// xp, wp: x and W, or their fp32 pieces.
poetx_status project(poetx_dtype dt, Act act, const uint8_t* xp, int N, int D, const uint8_t* wp, int F,
                     const Outputs& o, cudaStream_t s) {
  const bool f32 = dt == POETX_F32;
  const size_t half = (size_t)F * D * 2;  // bytes of W's gate rows in bf16
  auto bf16_map = [&](CUtensorMap* m, const void* p, long long outer, int bi, int bo) {
    return encode_tma_2d(m, p, TMA_BF16, D, outer, D, bi, bo, true);
  };
  if (!f32 && rows_forward_fits_bf16(N, D, F))
    return rows_forward({false, xp, wp, N, D, F, o.h, o.z, o.dh, o.z2, o.pitch}, act, s);
  if (!f32 && few_rows(N, D)) {
    FfnScore p{};
    const int sms = sm_count(), each = ceil_div(F, (long long)sms * BM);
    const int height = ceil_div(F, (long long)sms * each);
    p.height = (int)align_up((size_t)height, 8);
    p.tiles = ceil_div(F, p.height);
    p.F = F;
    p.rows = N;
    p.h = static_cast<__nv_bfloat16*>(o.h);
    p.z = static_cast<__nv_bfloat16*>(o.z);
    p.dh = static_cast<const __nv_bfloat16*>(o.dh);
    p.z2 = static_cast<__nv_bfloat16*>(o.z2);
    p.z_pitch = o.pitch;
    p.act = act;
    const int nt = N <= 16 ? 16 : (N <= 32 ? 32 : (N <= 64 ? 64 : 128));
    // K blocks per stage: as many as leave four stages (three where two blocks go in)
    p.grouped = D % 64 == 0;
    p.kps = 1;
    const bool merged = 2 * p.height <= BM;
    const int blocks = ceil_div(D, BK), room = score_room(nt, merged);
    for (int k = 2; p.grouped && k <= 8 && k < 2 * blocks; k *= 2)
      if ((k == 2 ? 3 : 4) * score_stage_bytes(nt, p.height, k) <= room) p.kps = k;
    p.num_st = ceil_div(blocks, p.kps);
    CUtensorMap mw, mx;
    if (!encode_tma_halves(&mw, wp, D, F, p.height, p.kps) ||
        !(p.grouped ? encode_tma_groups(&mx, xp, D, N, nt, p.kps) : bf16_map(&mx, xp, N, BK, nt)))
      return POETX_ERR_CUDA;
    switch (nt) {
      case 16: return merged ? score<16, true>(mw, mx, p, s) : score<16, false>(mw, mx, p, s);
      case 32: return merged ? score<32, true>(mw, mx, p, s) : score<32, false>(mw, mx, p, s);
      case 64: return merged ? score<64, true>(mw, mx, p, s) : score<64, false>(mw, mx, p, s);
      default: return merged ? score<128, true>(mw, mx, p, s) : score<128, false>(mw, mx, p, s);
    }
  }
  FfnMaps m;
  FfnGemm p{};
  const size_t x_step = piece_step((size_t)N * D), w_step = piece_step((size_t)2 * F * D);
  const int np = f32 ? 3 : 1;
  for (int i = 0; i < 3; ++i) {
    const int k = i < np ? i : 0;
    if (!bf16_map(&m.a[i], xp + k * x_step, N, BK, BM) ||
        !bf16_map(&m.g[i], wp + k * w_step, F, BK, BF) ||
        !bf16_map(&m.u[i], wp + k * w_step + half, F, BK, BF))
      return POETX_ERR_CUDA;
  }
  const TmaElem et = f32 ? TMA_F32 : TMA_BF16;
  const int bi = f32 ? 32 : 64;
  const size_t esz = dtype_size(dt);
  m.h = m.zg = m.zu = m.a[0];
  const void* h = o.dh ? o.dh : o.h;
  if (h && !encode_tma_2d(&m.h, h, et, F, N, F, bi, 32, true)) return POETX_ERR_CUDA;
  if (o.z && (!encode_tma_2d(&m.zg, o.z, et, F, N, o.pitch, bi, 32, true) ||
              !encode_tma_2d(&m.zu, static_cast<uint8_t*>(o.z) + (size_t)F * esz, et, F, N, o.pitch, bi, 32,
                             true)))
    return POETX_ERR_CUDA;
  p.tiles_m = ceil_div(N, 2 * BM);
  p.tiles_f = ceil_div(F, BF);
  p.num_tiles = p.tiles_m * p.tiles_f;
  p.num_kb = ceil_div(D, BK);
  p.chunk = f32 ? 4 : 64;
  p.M = N;
  p.F = F;
  p.store_h = o.h != nullptr;
  p.store_z = o.z != nullptr;
  p.act = act;
  if (f32) return gemm<kSegs, false>(m, p, s);
  return o.dh ? gemm<1, true>(m, p, s) : gemm<1, false>(m, p, s);
}

// The backward's workspace.
//
// dz's pieces: bf16 products take dz rounded to bf16, as a program would that keeps its gradients in bf16.  dx and
// dW are then 1.41 times as far from 64 bits as the rounding of the result alone (0.0023 and 0.0017 at 4096 x 2048 x
// 8192).  A second piece makes that 1.0, and where W is what takes the time it is next to free (up to 128 rows); above,
// it would double the K of dW's product and the rows of dx's (299 us there would be some 600).
struct Plan {
  bool f32, fine;
  bool rows, few;   // so few rows that ffn_rows.cu (fp32) or ffn_grad.cu has the gradients
  bool direct;      // dz from the projections' sums (else from z, kept or written to the workspace)
  int pieces;       // bf16 pieces of dz (0: it is fp32)
  long long pitch;  // of dz: 2 F up to a multiple of 64
  int splits;
  size_t xs, ws, z, dz, z_step, dxp, bytes;
};
Plan plan(poetx_dtype dt, int N, int D, int F, bool have_z, bool dx) {
  Plan o{};
  const size_t n = N > 0 ? N : 1;
  o.f32 = dt == POETX_F32;
  o.fine = !o.f32 && N <= kScoreRows;
  o.rows = o.f32 && N <= kRowsGradients;
  o.few = !o.f32 && N <= kFewGradients;
  o.pieces = o.f32 ? (o.rows ? 0 : 3) : (o.fine ? 2 : 1);
  o.pitch = o.pieces ? (long long)align_up((size_t)2 * F, 64) : 2ll * F;
  o.splits = !dx      ? 1
             : o.rows ? rows_splits((int)n, D, 2 * F)
             : o.few  ? few_splits((int)n, D, 2 * F)
                      : grad_splits(n, D, 2 * F, o.f32);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += align_up(bytes, 1024);
    return a;
  };
  o.xs = o.pieces == 3 ? take(3 * piece_step(n * D)) : 0;
  o.ws = o.pieces == 3 ? take(3 * piece_step((size_t)2 * F * D)) : 0;
  // (128 rows or fewer of a D beyond the few-row kernel's go by z: dz is then in two pieces)
  o.direct = !have_z && (o.f32 ? o.rows : !o.fine || few_rows(N, D));
  o.z = have_z || o.direct ? 0 : take(n * 2 * F * dtype_size(dt));
  o.z_step = align_up(n * o.pitch * (o.pieces ? 2 : 4), 1024);
  o.dz = take((o.pieces ? o.pieces : 1) * o.z_step);
  if (dx && (o.splits > 1 || o.fine))
    o.dxp = take((size_t)o.splits * (o.rows || o.few ? n : align_up(n, 256)) * D * 4);
  o.bytes = at;
  return o;
}

}  // namespace
}  // namespace poetx

using namespace poetx;

namespace {

poetx_status glu_check(poetx_dtype dt, poetx_activation act, const void* g, const void* u, int N, int F,
                       long long pitch) {
  if (N < 0 || !act_ok(act)) return POETX_ERR_ARG;
  if (dt != POETX_F32 && dt != POETX_BF16) return POETX_ERR_DTYPE;
  if (F < 8 || F % 8 || F > (1 << 21) || pitch < F || pitch % 8 || pitch > (1ll << 40))
    return POETX_ERR_SHAPE;
  if (!aligned16(g) || !aligned16(u)) return POETX_ERR_ALIGN;
  return N > 0 && (!g || !u) ? POETX_ERR_ARG : POETX_OK;
}

}  // namespace

extern "C" poetx_status poetx_glu_fwd(poetx_dtype dt, poetx_activation act, const void* g, const void* u,
                                      int N, int F, long long pitch, void* h, cudaStream_t stream) {
  POETX_TRY(glu_check(dt, act, g, u, N, F, pitch));
  if (!aligned16(h)) return POETX_ERR_ALIGN;
  if (N == 0) return POETX_OK;
  if (!h) return POETX_ERR_ARG;
  const GluCall c{dt, act_of(act), g, u, nullptr, N, F, pitch, F, {h}, 0};
  return run_glu(c, stream);
}

extern "C" poetx_status poetx_glu_bwd(poetx_dtype dt, poetx_activation act, const void* g, const void* u,
                                      const void* dh, int N, int F, long long pitch, void* dg, void* du,
                                      long long d_pitch, cudaStream_t stream) {
  POETX_TRY(glu_check(dt, act, g, u, N, F, pitch));
  if (d_pitch < F || d_pitch % 8 || d_pitch > (1ll << 40)) return POETX_ERR_SHAPE;
  if (!aligned16(dh) || !aligned16(dg) || !aligned16(du)) return POETX_ERR_ALIGN;
  if (N == 0) return POETX_OK;
  if (!dh || !dg || !du) return POETX_ERR_ARG;
  const GluCall c{dt, act_of(act), g, u, dh, N, F, pitch, d_pitch, {dg, du}, 0};
  return run_glu(c, stream);
}

extern "C" size_t poetx_ffn_fwd_workspace_bytes(poetx_dtype dt, int N, int D, int F) {
  if (!shape_ok(dt, N, D, F) || dt != POETX_F32) return 0;
  // What the CUDA cores take needs none of W's pieces, and none of x's: but so an fp32 call without a workspace
  // is refused at every N.  (Up to a megabyte W's are asked for from 33 rows on, whichever way the call goes.)
  const size_t x_bytes = 3 * piece_step((size_t)(N > 0 ? N : 1) * D), w_bytes = 3 * piece_step((size_t)2 * F * D);
  const bool rows = rows_forward_fits(N, D, F) && (N <= kRowsForward || w_bytes > (1u << 20));
  return rows ? x_bytes : x_bytes + w_bytes;
}

extern "C" poetx_status poetx_ffn_fwd(poetx_dtype dt, poetx_activation act, const void* x, int N, int D,
                                      const void* W, int F, void* h, void* z, void* ws, size_t ws_bytes,
                                      cudaStream_t stream) {
  if (N < 0 || !act_ok(act)) return POETX_ERR_ARG;
  if (dt != POETX_F32 && dt != POETX_BF16) return POETX_ERR_DTYPE;
  if (!shape_ok(dt, N, D, F) || !tiles_ok(N, F)) return POETX_ERR_SHAPE;
  for (const void* p : {x, W, (const void*)h, (const void*)z, (const void*)ws})
    if (!aligned16(p)) return POETX_ERR_ALIGN;
  if (N == 0) return POETX_OK;
  const size_t need = poetx_ffn_fwd_workspace_bytes(dt, N, D, F);
  if (!x || !W || !h || (need && !ws)) return POETX_ERR_ARG;
  if (ws_bytes < need) return POETX_ERR_WORKSPACE;
  if (h == x || h == W || h == z || (z && (z == x || z == W))) return POETX_ERR_ARG;
  if (!umma_supported()) return POETX_ERR_UNSUPPORTED;
  if (dt == POETX_F32 && rows_forward_fits(N, D, F))
    return rows_forward({true, x, W, N, D, F, h, z, nullptr, nullptr, 2ll * F}, act_of(act), stream);
  const uint8_t *xp = static_cast<const uint8_t*>(x), *wp = static_cast<const uint8_t*>(W);
  if (dt == POETX_F32) {
    uint8_t* w = static_cast<uint8_t*>(ws);
    const size_t x_step = piece_step((size_t)N * D), w_step = piece_step((size_t)2 * F * D);
    POETX_TRY(split_pieces(static_cast<const float*>(x), (long long)N * D, w, x_step,
                           static_cast<const float*>(W), 2ll * F * D, w + 3 * x_step, w_step, stream));
    xp = w;
    wp = w + 3 * x_step;
  }
  return project(dt, act_of(act), xp, N, D, wp, F, Outputs{h, z, nullptr, nullptr, 2ll * F}, stream);
}

extern "C" size_t poetx_ffn_bwd_workspace_bytes(poetx_dtype dt, int N, int D, int F, int have_z,
                                                int want_dx, int want_dW) {
  if (!shape_ok(dt, N, D, F) || (!want_dx && !want_dW)) return 0;
  return plan(dt, N, D, F, have_z != 0, want_dx != 0).bytes;
}

extern "C" poetx_status poetx_ffn_bwd(poetx_dtype dt, poetx_activation act, const void* x, int N, int D,
                                      const void* W, int F, const void* z, const void* dh, void* dx,
                                      void* dW, int accumulate, void* ws, size_t ws_bytes,
                                      cudaStream_t stream) {
  if (N < 0 || !act_ok(act) || (!dx && !dW)) return POETX_ERR_ARG;
  if (dt != POETX_F32 && dt != POETX_BF16) return POETX_ERR_DTYPE;
  if (!shape_ok(dt, N, D, F) || !tiles_ok(N, F)) return POETX_ERR_SHAPE;
  for (const void* p : {x, W, z, dh, (const void*)dx, (const void*)dW, (const void*)ws})
    if (!aligned16(p)) return POETX_ERR_ALIGN;
  const size_t esz = dtype_size(dt);
  if (N == 0) {
    if (dW && !accumulate) POETX_CUDA_TRY(cudaMemsetAsync(dW, 0, (size_t)2 * F * D * esz, stream));
    return POETX_OK;
  }
  if (!x || !W || !dh || !ws) return POETX_ERR_ARG;
  const Plan pl = plan(dt, N, D, F, z != nullptr, dx != nullptr);
  if (ws_bytes < pl.bytes) return POETX_ERR_WORKSPACE;
  if ((dW && (dW == x || dW == W || dW == dx || dx == x)) || dx == W) return POETX_ERR_ARG;
  if (!umma_supported()) return POETX_ERR_UNSUPPORTED;
  uint8_t* w = static_cast<uint8_t*>(ws);
  const uint8_t *xp = static_cast<const uint8_t*>(x), *wp = static_cast<const uint8_t*>(W);
  if (pl.pieces == 3) {
    xp = w + pl.xs;
    wp = w + pl.ws;
    POETX_TRY(split_pieces(static_cast<const float*>(x), (long long)N * D, w + pl.xs,
                           piece_step((size_t)N * D), static_cast<const float*>(W), 2ll * F * D, w + pl.ws,
                           piece_step((size_t)2 * F * D), stream));
  }
  const int pieces = pl.pieces;
  if (pl.direct && pl.f32) {
    POETX_TRY(rows_forward({true, x, W, N, D, F, nullptr, w + pl.dz, dh, nullptr, 2ll * F}, act_of(act),
                           stream));
  } else if (pl.direct) {
    POETX_TRY(project(dt, act_of(act), xp, N, D, wp, F,
                      Outputs{nullptr, w + pl.dz, dh, pl.fine ? w + pl.dz + pl.z_step : nullptr, pl.pitch},
                      stream));
  } else {
    if (!z) {
      z = w + pl.z;
      if (pl.f32 && N <= kRowsForward)
        POETX_TRY(rows_forward({true, x, W, N, D, F, nullptr, w + pl.z, nullptr, nullptr, 2ll * F},
                               act_of(act), stream));
      else
        POETX_TRY(project(dt, act_of(act), xp, N, D, wp, F,
                          Outputs{nullptr, w + pl.z, nullptr, nullptr, 2ll * F}, stream));
    }
    // dz: the gate's half, then the value's, in fp32 or in one to three bf16 pieces
    GluCall c{dt, act_of(act), z, static_cast<const uint8_t*>(z) + (size_t)F * esz, dh, N, F, 2ll * F,
              pl.pitch, {}, pieces == 1 ? 0 : pieces};
    for (int i = 0; i < std::max(pieces, 1); ++i) {
      c.out[2 * i] = w + pl.dz + i * pl.z_step;
      c.out[2 * i + 1] = w + pl.dz + i * pl.z_step + (size_t)F * (pieces ? 2 : 4);
    }
    POETX_TRY(run_glu(c, stream));
  }
  float* const dxp = reinterpret_cast<float*>(w + pl.dxp);
  if (pl.rows)
    return rows_gradients({reinterpret_cast<const float*>(w + pl.dz), static_cast<const float*>(x),
                           static_cast<const float*>(W), N, D, 2 * F,
                           static_cast<float*>(dx), static_cast<float*>(dW), accumulate, dxp},
                          stream);
  if (pl.few)
    return few_gradients({w + pl.dz, w + pl.dz + pl.z_step, pl.pitch, x, W, N, D, 2 * F, dx, dW, accumulate,
                          dxp},
                         stream);
  GradProducts g{};
  g.f32 = pl.f32;
  g.fine = pl.fine;
  g.rows = N;
  g.D = D;
  g.V = 2 * F;
  g.pitch = pl.pitch;
  g.z_cols = 2ll * F;
  for (int i = 0; i < pieces; ++i) g.z[i] = w + pl.dz + i * pl.z_step;
  g.x = xp;
  g.x_step = piece_step((size_t)N * D);
  g.w = wp;
  g.w_step = piece_step((size_t)2 * F * D);
  g.T = 1.f;
  g.dx = dx;
  g.dW = dW;
  g.accumulate = accumulate;
  g.first = g.last = true;
  g.splits = pl.splits;
  g.dxp = dxp;
  return grad_products(g, stream);
}
