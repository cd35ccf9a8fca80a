// The linear head's loss over a large vocabulary without keeping the logits, with its gradients:
// softmax cross entropy (labels) and distillation (a teacher's top logits).
//
//   z = W x / T per row,  lse = ln sum_v exp z_v,  p = exp(z - lse)
//   cross entropy (T = 1)   loss = lse - z_t + zl lse^2,      dz = g ((1 + 2 zl lse) p - onehot_t)
//   distillation            q = softmax over the row's K teacher logits / T,
//                           loss = T^2 sum_k q_k (ln q_k - z_{i_k} + lse),
//                           d(Wx) = g T (p - sum_k q_k onehot_{i_k})
//   dx = dz W,  dW = dz^T x
//
// Both are the same three products with a sparse target, so they share every kernel.  The rows are
// taken in pieces.  Per piece: (1) the logits' product, whose epilogue leaves for each row and each
// group of 128 columns the maximum m and the sum of exp(z - m), and stores exp(z - m) in 16 bits
// (fp16: it lies in [0, 1], so its rounding, 2^-12, stays below the bf16 rounding of dz that
// follows; no fp32 logit is stored); (2) a row kernel that joins the groups into lse, writes the
// loss and turns the row into dz in place (bf16); (3) dx = dz W; (4) dW (+)= dz^T x.  That is
// 6 N V D flops: nothing is computed twice.  The logits of the sparse targets come from fp32 dot
// products of their own, so that a loss or a p - 1 near zero does not see the 16-bit rounding.
//
// The products run on tcgen05 in 2-CTA pairs (256 x 256 tiles, operands by TMA).  The tensor core
// truncates when it adds into its fp32 accumulator, which over a long K drifts by about 2^-24 of
// the sum per step; so after every `chunk` of K the partial tile moves from TMEM into the epilogue's
// registers and is added there with IEEE adds, while the next chunk runs in the other half of TMEM.
//
// fp32 heads run on the same kernels: each fp32 operand is split into three bf16 pieces (8 + 8 + 8
// significant bits) and a product takes the six pairs of pieces whose weight is above 2^-24, the
// small ones first.  Their exp(z - m) is kept in fp32.
//
// Every mbarrier wait is bounded; on expiry the kernel records POETX_ERR_TIMEOUT, drains its own
// copies, frees its TMEM and returns.
#include <cuda_fp16.h>

#include <mutex>

#include "common.cuh"
#include "kernels.h"

namespace poetx {

// Site id of this file's bounded waits (file id x 10000 + source line).
constexpr int kSite = 6 * 10000;

namespace {

constexpr int BM = 128;           // rows per CTA (256 per pair)
constexpr int BN = 256;           // columns per pair tile
constexpr int BK = 64;
constexpr int kStages = 6;
constexpr int kEpiWarps = 8;      // two per TMEM lane quarter, each 128 columns
constexpr int kGemmThreads = 64 + 32 * kEpiWarps;
constexpr int kGroup = 128;       // columns of one (max, sum) group
constexpr uint32_t kABytes = BM * BK * 2;
constexpr uint32_t kBBytes = BN / 2 * BK * 2;
constexpr uint32_t kStageBytes = kABytes + kBBytes;  // 32 KB per CTA
constexpr uint32_t kStgBytes = 32 * 128;             // one epilogue warp's box: 32 rows of 128 bytes
constexpr int kGemmSmem = kStages * kStageBytes + kEpiWarps * kStgBytes + 1024 + 512;
static_assert(kGemmSmem <= 227 * 1024, "head products: shared memory");
constexpr int kMaxSegs = 6;

enum Epi : int {
  EPI_LSE = 0,    // groups' (max, sum) and, where the gradients are wanted, exp(z - max)
  EPI_STORE = 1,  // the product itself
};

struct HeadMaps {
  CUtensorMap a[3], b[3];  // the operands' pieces (one for bf16)
  CUtensorMap c;           // the stored tile
};

struct HeadGemm {
  int tiles_m, tiles_n, splits, num_tiles;
  int n_fast;            // raster: 1: tiles of a row stripe first (A read once), 0: of a column stripe
  int num_kb, kb_split;  // 64-wide K blocks in all, per split
  int chunk;             // K blocks per accumulator hand-over
  int nseg;              // products of operand pieces per K block
  int8_t seg_a[kMaxSegs], seg_b[kMaxSegs];
  int M, N;              // valid rows and columns
  int n_store;           // columns of the stored tensor
  int c_rows;            // EPI_STORE: rows of the stored tensor per split
  // EPI_LSE
  float scale2;          // log2(e) / T
  float2* part;          // [M][groups]
  int groups;
  const int32_t* ucol;   // [M][K] the rows' distinct target columns, ascending (K = 1: any value)
  const uint16_t* gstart;  // [M][groups + 1] first of them in each group; NULL: K = 1
  int K;
  float* tl;             // [M][K] their logits, before 1/T
  int store;             // whether c is stored
  // EPI_STORE: added before the store (nullable)
  const float* add_f32;
  const __nv_bfloat16* add_bf16;
  int* err;
  unsigned long long limit_ns;
};

template <bool MN>
__device__ __forceinline__ uint64_t tile_desc(uint32_t base, int k) {
  return MN ? make_sdesc(base + k * 2048, 8192, 1024) : make_sdesc(base + k * 32, 16, 1024);
}

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

struct Tile {
  int mi, nt, split, kb0, kb1;
};
__device__ __forceinline__ Tile tile_of(const HeadGemm& p, int t) {
  Tile c;
  const int per = p.tiles_m * p.tiles_n;
  c.split = t / per;
  const int r = t - c.split * per;
  c.mi = p.n_fast ? r / p.tiles_n : r % p.tiles_m;
  c.nt = p.n_fast ? r % p.tiles_n : r / p.tiles_m;
  c.kb0 = c.split * p.kb_split;
  c.kb1 = min(p.num_kb, c.kb0 + p.kb_split);
  return c;
}

// C[M, N] = A[M, K] B[N, K]^T over 256 x 256 tiles; A_MN / B_MN: the operand is stored with its M
// or N axis contiguous ([K][M], [K][N]).  Warp 0 of each CTA loads its 128 rows of A and its half
// of B, one thread of the even CTA's warp 1 issues the MMAs, warps 2-9 read the accumulators back
// (warp w: rows 32 (w % 4).. of the CTA's 128, columns 128 ((w - 2) / 4)..).
template <bool A_MN, bool B_MN, int EPI, bool OUT_F32>
__global__ void __launch_bounds__(kGemmThreads, 1)
    head_gemm_kernel(const __grid_constant__ HeadMaps maps, const HeadGemm p) {
  constexpr uint32_t IDESC = make_idesc(2 * BM, BN, A_MN, B_MN);
  constexpr uint32_t TMEM_COLS = 2 * BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* staging = smem + kStages * kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kEpiWarps * kStgBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;  // [2] accumulator written
  uint64_t* tempty = tfull + 2;       // [2] accumulator read by both CTAs' epilogue warps
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
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
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(&maps.b[0]);
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

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ TMA producer
    long long g = 0;
    bool ok = true;
    for (int t = t0; t < p.num_tiles && ok; t += t_step) {
      const Tile c = tile_of(p, t);
      const int m0 = (2 * c.mi + crank) * BM, n0 = c.nt * BN;
      for (int kb = c.kb0; kb < c.kb1 && ok; ++kb)
        for (int sg = 0; sg < p.nseg; ++sg, ++g) {
          const int s = (int)(g % kStages);
          if (*abort_flag || !mbar_wait_bounded(&empty[s], (uint32_t)((g / kStages) & 1) ^ 1, p.err,
                                                p.limit_ns, kSite + __LINE__)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          uint8_t* sa = smem + s * kStageBytes;
          uint8_t* sb = sa + kABytes;
          const CUtensorMap* ma = &maps.a[p.seg_a[sg]];
          const CUtensorMap* mb = &maps.b[p.seg_b[sg]];
          const int k = kb * BK;
          if (crank == 0) mbar_arrive_expect_tx(&full[s], 2 * kStageBytes);
          const uint32_t fb = mapa_shared(&full[s], 0);
          if (!A_MN) {
            tma_load_2d_pair(sa, ma, fb, k, m0);
          } else {
            tma_load_2d_pair(sa, ma, fb, m0, k);
            tma_load_2d_pair(sa + 8192, ma, fb, m0 + 64, k);
          }
          if (!B_MN) {
            tma_load_2d_pair(sb, mb, fb, k, n0 + crank * (BN / 2));
          } else {
            tma_load_2d_pair(sb, mb, fb, n0 + crank * (BN / 2), k);
            tma_load_2d_pair(sb + 8192, mb, fb, n0 + crank * (BN / 2) + 64, k);
          }
        }
    }
    // no copy may be in flight when the CTA exits: the MMAs release a stage after reading it
    for (long long j = g - 1; j >= 0 && j >= g - kStages; --j)
      mbar_wait_bounded(&empty[j % kStages], (uint32_t)((j / kStages) & 1), p.err, p.limit_ns,
                        kSite + __LINE__);
  } else if (warp == 1 && lane == 0 && crank == 0) {
    // ------------------------------------------------------------ MMA issuer
    long long g = 0, it = 0;  // ring position; accumulator hand-overs
    bool ok = true;
    for (int t = t0; t < p.num_tiles && ok; t += t_step) {
      const Tile c = tile_of(p, t);
      for (int kb = c.kb0; kb < c.kb1 && ok; kb += p.chunk, ++it) {
        const int a = (int)(it & 1);
        if (*abort_flag || !mbar_wait_bounded(&tempty[a], (uint32_t)((it >> 1) & 1) ^ 1, p.err,
                                              p.limit_ns, kSite + __LINE__)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(a * BN);
        const int blocks = (min(c.kb1, kb + p.chunk) - kb) * p.nseg;
        for (int j = 0; j < blocks; ++j, ++g) {
          const int s = (int)(g % kStages);
          if (*abort_flag || !mbar_wait_bounded(&full[s], (uint32_t)((g / kStages) & 1), p.err,
                                                p.limit_ns, kSite + __LINE__)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_base = smem_base + s * kStageBytes;
          const uint32_t b_base = a_base + kABytes;
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            umma_bf16_pair(d, tile_desc<A_MN>(a_base, k), tile_desc<B_MN>(b_base, k), IDESC,
                           (j | k) != 0);
          umma_commit_pair(&empty[s]);
        }
        umma_commit_pair(&tfull[a]);
      }
    }
    if (it > 0)  // TMEM is freed after the final barrier: wait for the last MMAs
      mbar_wait_bounded(&tfull[(it - 1) & 1], (uint32_t)(((it - 1) >> 1) & 1), p.err, p.limit_ns,
                        kSite + __LINE__);
  } else if (warp >= 2) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int cbeg = ((warp - 2) >> 2) * kGroup;
    uint8_t* stg = staging + (warp - 2) * kStgBytes;
    long long it = 0;
    bool ok = true;
    for (int t = t0; t < p.num_tiles && ok; t += t_step) {
      const Tile c = tile_of(p, t);
      const int row_w = (2 * c.mi + crank) * BM + q * 32;  // the warp's first row
      const int row = row_w + lane;
      const int col0 = c.nt * BN + cbeg;
      // the row's targets in this group: [u0, u1) of its list (read ahead of the wait)
      int u0 = 0, u1 = 0;
      if (EPI == EPI_LSE && row < p.M && col0 < p.N) {
        if (p.gstart) {
          const uint16_t* gs = p.gstart + (long long)row * (p.groups + 1) + col0 / kGroup;
          u0 = gs[0];
          u1 = gs[1];
        } else {
          const int tc = p.ucol[row];
          u1 = tc >= col0 && tc < min(col0 + kGroup, p.N);
        }
      }
      float v[kGroup];
      for (int kb = c.kb0; kb < c.kb1; kb += p.chunk, ++it) {
        const int a = (int)(it & 1);
        const bool got = !*abort_flag && mbar_wait_bounded(&tfull[a], (uint32_t)((it >> 1) & 1),
                                                           p.err, p.limit_ns, kSite + __LINE__);
        if (!__all_sync(0xffffffffu, got)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t ta = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * BN + cbeg);
#pragma unroll
        for (int j = 0; j < kGroup; j += 32) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(ta + j, r);
          tmem_ld_wait();
          if (kb == c.kb0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[j + i] = __uint_as_float(r[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[j + i] += __uint_as_float(r[i]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(&tempty[a], 0));
      }
      if (!ok) break;
      if (col0 >= p.N || row_w >= p.M) continue;
      if (EPI == EPI_LSE) {
        if (col0 + kGroup > p.N) {
#pragma unroll
          for (int i = 0; i < kGroup; ++i)
            if (col0 + i >= p.N) v[i] = __int_as_float(0xff800000);  // -inf: exp 0
        }
        if (__any_sync(0xffffffffu, u0 < u1)) {  // take the targets out of the group
          uint32_t mask[kGroup / 32] = {};
          const int32_t* uc = p.ucol + (long long)row * p.K;
          for (int u = u0; u < u1; ++u) {
            const int j = uc[u] - col0;
#pragma unroll
            for (int k = 0; k < kGroup / 32; ++k)
              if ((j >> 5) == k) mask[k] |= 1u << (j & 31);
          }
          float* tl = p.tl + (long long)row * p.K;
#pragma unroll
          for (int i = 0; i < kGroup; ++i)
            if (mask[i >> 5] >> (i & 31) & 1u) {
              tl[u0++] = v[i];
              v[i] = __int_as_float(0xff800000);
            }
        }
        float m = v[0];
#pragma unroll
        for (int i = 1; i < kGroup; ++i) m = fmaxf(m, v[i]);
        m *= p.scale2;
        const float off = m == __int_as_float(0xff800000) ? 0.f : m;  // a group of -inf sums to 0
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < kGroup; i += 2) {
          v[i] = ex2(fmaf(v[i], p.scale2, -off));
          v[i + 1] = ex2(fmaf(v[i + 1], p.scale2, -off));
          s0 += v[i];
          s1 += v[i + 1];
        }
        if (row < p.M)
          p.part[(long long)row * p.groups + (col0 / kGroup)] = make_float2(m, s0 + s1);
        if (!p.store) continue;
      } else {
        if (p.add_f32 && row < p.M) {
          const float* src = p.add_f32 + (long long)row * p.N + col0;
#pragma unroll
          for (int i = 0; i < kGroup; i += 4)
            if (col0 + i < p.N) {  // N is a multiple of 8
              const float4 w = *reinterpret_cast<const float4*>(src + i);
              v[i] += w.x;
              v[i + 1] += w.y;
              v[i + 2] += w.z;
              v[i + 3] += w.w;
            }
        }
        if (p.add_bf16 && row < p.M) {
          const __nv_bfloat16* src = p.add_bf16 + (long long)row * p.N + col0;
#pragma unroll
          for (int i = 0; i < kGroup; i += 8)
            if (col0 + i < p.N) {
              const uint4 w = *reinterpret_cast<const uint4*>(src + i);
              const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                v[i + 2 * j] += __uint_as_float(u[j] << 16);
                v[i + 2 * j + 1] += __uint_as_float(u[j] & 0xffff0000u);
              }
            }
        }
      }
      // store by TMA: boxes of 32 rows x 128 bytes, 128-byte swizzle; rows and columns outside
      // the tensor are clipped
      constexpr int PASS = OUT_F32 ? 32 : 64;
      const int orow = EPI == EPI_STORE ? c.split * p.c_rows + row_w : row_w;
#pragma unroll
      for (int j = 0; j < kGroup; j += PASS) {
        if (col0 + j >= p.n_store) break;
        if (lane == 0) bulk_wait_read<0>();  // the previous box has been read
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint4 w;
          if (OUT_F32) {
            w = make_uint4(__float_as_uint(v[j + 4 * i]), __float_as_uint(v[j + 4 * i + 1]),
                           __float_as_uint(v[j + 4 * i + 2]), __float_as_uint(v[j + 4 * i + 3]));
          } else {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float lo = v[j + 8 * i + 2 * k], hi = v[j + 8 * i + 2 * k + 1];
              if (EPI == EPI_LSE) {
                const __half2 h = __floats2half2_rn(lo, hi);
                u[k] = *reinterpret_cast<const uint32_t*>(&h);
              } else {
                u[k] = pack_bf16x2(lo, hi);
              }
            }
            w = make_uint4(u[0], u[1], u[2], u[3]);
          }
          *reinterpret_cast<uint4*>(stg + lane * 128 + ((i ^ (lane & 7)) << 4)) = w;
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&maps.c, stg, col0 + j, orow);
          bulk_commit();
        }
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

// ---------------------------------------------------------------- CUDA-core kernels
constexpr uint16_t kNoSlot = 0xffff;

// A row's K target columns: slot[k] = place of idx[k] among the row's distinct columns in ascending
// order (kNoSlot for an absent entry or one beyond the vocabulary), ucol = those columns, gstart =
// the first of them in each group of 128.  By ranks: K is at most a thousand.
__global__ void __launch_bounds__(256)
    head_targets_kernel(const int32_t* __restrict__ idx, int K, int V, int groups,
                        uint16_t* __restrict__ slot, int32_t* __restrict__ ucol,
                        uint16_t* __restrict__ gstart) {
  extern __shared__ int tsm[];
  int* is = tsm;           // [K] columns
  int* first = is + K;     // [K] whether it is the column's first entry
  int* us = first + K;     // [K] distinct columns, ascending
  __shared__ int nu;
  pdl_trigger();
  pdl_wait();
  const long long row = blockIdx.x;
  const int t = threadIdx.x;
  if (t == 0) nu = 0;
  for (int k = t; k < K; k += 256) is[k] = idx[row * K + k];
  __syncthreads();
  for (int k = t; k < K; k += 256) {
    const int c = is[k];
    bool f = c >= 0 && c < V;
    for (int j = 0; j < k && f; ++j) f = is[j] != c;
    first[k] = f;
    if (f) atomicAdd(&nu, 1);
  }
  __syncthreads();
  for (int k = t; k < K; k += 256) {
    const int c = is[k];
    int r = 0;
    if (c >= 0 && c < V) {
      for (int j = 0; j < K; ++j) r += first[j] && is[j] < c;
      if (first[k]) us[r] = c;
    } else {
      r = kNoSlot;
    }
    slot[row * K + k] = (uint16_t)r;
  }
  __syncthreads();
  const int n = nu;
  uint16_t* gs = gstart + row * (groups + 1);
  for (int u = t; u <= n; u += 256) {  // groups after the previous column's, up to this one's
    const int lo = u ? us[u - 1] / kGroup + 1 : 0, hi = u < n ? us[u] / kGroup : groups;
    for (int g = lo; g <= hi; ++g) gs[g] = (uint16_t)u;
    if (u < n) ucol[row * K + u] = us[u];
  }
}

struct RowArgs {
  int V, groups, K;
  long long pitch;        // columns of a row of e
  const float2* part;     // [rows][groups], log2 units
  const float* tl;        // [rows][K] logits of the distinct targets (before 1/T)
  const int32_t* idx;     // [rows][K] the targets as given
  const int32_t* ucol;    // [rows][K] distinct, ascending
  const uint16_t* slot;   // [rows][K] place of idx in ucol
  const float* tlogit;    // [rows][K] the teacher's logits; NULL: cross entropy (K = 1)
  const float* dloss;     // [rows] upstream gradients (with e)
  float T, zl;
  float* loss;
  float* lse;             // nullable
  void* e;                // exp(z - m) of the rows, turned into dz (nullable: loss only)
  __nv_bfloat16* piece[3];  // fp32 heads: dz in three bf16 pieces
};

constexpr int kRowThreads = 256;
constexpr float kLn2 = 0.69314718055994530942f, kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < kRowThreads / 32; ++w) v += red[w];
  return v;
}
__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < kRowThreads / 32; ++w) v = fmaxf(v, red[w]);
  return v;
}

__device__ __forceinline__ void split3(float v, __nv_bfloat16 (&o)[3]) {
  o[0] = __float2bfloat16_rn(v);
  v -= __bfloat162float(o[0]);
  o[1] = __float2bfloat16_rn(v);
  v -= __bfloat162float(o[1]);
  o[2] = __float2bfloat16_rn(v);
}

// One CTA per row: joins the groups, writes loss and lse and turns e into dz.
template <bool F32>
__global__ void __launch_bounds__(kRowThreads) head_row_kernel(const RowArgs p) {
  extern __shared__ float sm[];
  float* fac = sm;            // [groups] maximum, then factor of each group
  float* z2 = fac + p.groups;  // [K] the distinct targets' logits in log2 units
  float* qs = z2 + p.K;       // [K] their weights q
  float* qk = qs + p.K;       // [K] the entries' weights
  __shared__ float red[kRowThreads / 32];
  pdl_trigger();
  pdl_wait();
  const long long row = blockIdx.x;
  const int t = threadIdx.x;
  const float ninf = __int_as_float(0xff800000);
  const float scale2 = kLog2e / p.T;
  const int32_t* idx = p.idx + row * p.K;
  const uint16_t* slot = p.slot + row * p.K;
  const int32_t* ucol = p.ucol + row * p.K;
  // the distinct targets: nu of them
  float nbad = 0.f, top = -1.f;  // (slots are below 1024: exact in fp32)
  for (int k = t; k < p.K; k += kRowThreads) {
    const int c = idx[k];
    nbad += c >= p.V ? 1.f : 0.f;
    if (c >= 0 && c < p.V) top = fmaxf(top, p.tlogit ? (float)slot[k] : 0.f);
  }
  const bool bad = block_max(nbad, red) > 0.f;  // an index beyond the vocabulary
  const int nu = (int)block_max(top, red) + 1;
  float zm = ninf;
  for (int u = t; u < nu; u += kRowThreads) {
    z2[u] = p.tl[row * p.K + u] * scale2;
    qs[u] = 0.f;
    zm = fmaxf(zm, z2[u]);
  }
  zm = block_max(zm, red);
  // log-sum-exp in log2 units: the groups leave the targets out
  const float2* part = p.part + row * p.groups;
  float m = zm;
  for (int g = t; g < p.groups; g += kRowThreads) {
    fac[g] = part[g].x;
    m = fmaxf(m, fac[g]);
  }
  m = block_max(m, red);
  const float off = m == ninf ? 0.f : m;
  // the largest target on its own (the first of equals), all others with the groups
  float um = 2048.f;
  for (int u = t; u < nu; u += kRowThreads)
    if (z2[u] == zm) um = fminf(um, (float)u);
  const int umax = (int)-block_max(-um, red);
  float s = 0.f;
  for (int g = t; g < p.groups; g += kRowThreads) s += part[g].y * exp2f(fac[g] - off);
  for (int u = t; u < nu; u += kRowThreads)
    if (u != umax) s += exp2f(z2[u] - off);
  const float others = block_sum(s, red);
  const float emax = nu ? exp2f(zm - off) : 0.f;
  const float total = others + emax;
  const float lse2 = off + log2f(total);
  const float lse = lse2 * kLn2;
  const bool sure = emax > others;  // the largest target has more than half
  const float lnp_max = sure ? -log1pf(others / emax) : (zm - lse2) * kLn2;
  float some, loss, weight;  // weight: of p in dz, before the upstream gradient
  float rest = 0.f;          // 1 - q of the largest target
  if (!p.tlogit) {
    some = nu ? 1.f : 0.f;
    loss = p.zl * lse * lse - lnp_max;
    weight = 1.f + 2.f * p.zl * lse;
    if (t == 0) qs[0] = 1.f;
  } else {
    const float* u = p.tlogit + row * p.K;
    const float invT = 1.f / p.T;
    float tm = ninf;
    for (int k = t; k < p.K; k += kRowThreads)
      if (idx[k] >= 0) tm = fmaxf(tm, u[k] * invT);
    tm = block_max(tm, red);
    some = tm == ninf ? 0.f : 1.f;
    float us = 0.f;
    for (int k = t; k < p.K; k += kRowThreads)
      if (idx[k] >= 0 && some > 0.f) us += expf(u[k] * invT - tm);
    us = block_sum(us, red);
    const float lus = logf(us);
    float l = 0.f;
    for (int k = t; k < p.K; k += kRowThreads) {
      float q = 0.f;
      if (slot[k] != kNoSlot && some > 0.f) {
        const float lq = u[k] * invT - tm - lus;
        q = expf(lq);
        if (q > 0.f) l += q * (lq - (slot[k] == umax ? lnp_max : (z2[slot[k]] - lse2) * kLn2));
        if (slot[k] != umax) rest += q;
      }
      qk[k] = q;
    }
    loss = block_sum(l, red) * p.T * p.T;
    rest = block_sum(rest, red);
    weight = 1.f;
    // weights per distinct column, the entries added in their order
    for (int v = t; v < nu; v += kRowThreads) {
      float q = 0.f;
      for (int k = 0; k < p.K; ++k)
        if (slot[k] == v) q += qk[k];
      qs[v] = q;
    }
  }
  if (t == 0) {
    p.loss[row] = bad ? __int_as_float(0x7fc00000) : (some > 0.f ? loss : 0.f);
    if (p.lse) p.lse[row] = lse;
  }
  if (!p.e) return;
  const bool live = some > 0.f && !bad;
  const float gT = live ? p.dloss[row] * p.T : 0.f;
  const float coef = gT * weight;
  for (int g = t; g < p.groups; g += kRowThreads) fac[g] = coef * exp2f(fac[g] - lse2);
  __syncthreads();
  if (!F32) {
    uint4* er = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.e) + row * p.pitch);
    for (long long i = t; i < p.pitch / 8; i += kRowThreads) {
      uint4 o = make_uint4(0u, 0u, 0u, 0u);
      if (live) {
        const uint4 w = er[i];
        const float f = fac[i / (kGroup / 8)];
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
          r[j] = pack_bf16x2(v.x * f, v.y * f);
        }
        o = make_uint4(r[0], r[1], r[2], r[3]);
      }
      er[i] = o;
    }
  } else {
    const float4* er = reinterpret_cast<const float4*>(static_cast<float*>(p.e) + row * p.pitch);
    for (long long i = t; i < p.pitch / 4; i += kRowThreads) {
      __nv_bfloat16 o[4][3];
      const float4 w = live ? er[i] : make_float4(0.f, 0.f, 0.f, 0.f);
      const float f = live ? fac[i / (kGroup / 4)] : 0.f;
      split3(w.x * f, o[0]);
      split3(w.y * f, o[1]);
      split3(w.z * f, o[2]);
      split3(w.w * f, o[3]);
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        __nv_bfloat16* d = p.piece[k] + row * p.pitch + 4 * i;
        *reinterpret_cast<__nv_bfloat162*>(d) = __halves2bfloat162(o[0][k], o[1][k]);
        *reinterpret_cast<__nv_bfloat162*>(d + 2) = __halves2bfloat162(o[2][k], o[3][k]);
      }
    }
  }
  if (!live) return;
  __syncthreads();
  // the targets' own columns: weight p - q, without cancellation where p is near 1
  for (int u = t; u < nu; u += kRowThreads) {
    const float pv = exp2f(z2[u] - lse2);
    float dz;
    if (u == umax && sure)
      dz = gT * ((weight - 1.f) * pv + ((p.tlogit ? rest : 0.f) - others / total));
    else
      dz = coef * pv - gT * qs[u];
    const int c = ucol[u];
    if (!F32) {
      static_cast<__nv_bfloat16*>(p.e)[row * p.pitch + c] = __float2bfloat16_rn(dz);
    } else {
      __nv_bfloat16 o[3];
      split3(dz, o);
#pragma unroll
      for (int j = 0; j < 3; ++j) p.piece[j][row * p.pitch + c] = o[j];
    }
  }
}

// The three bf16 pieces of `count` fp32 values (a multiple of 4).
__global__ void __launch_bounds__(256)
    head_split_kernel(const float4* __restrict__ src, long long quads, __nv_bfloat16* p0,
                      __nv_bfloat16* p1, __nv_bfloat16* p2) {
  pdl_trigger();
  pdl_wait();
  const long long stride = (long long)gridDim.x * blockDim.x;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < quads; i += stride) {
    const float4 w = src[i];
    __nv_bfloat16 o[4][3];
    split3(w.x, o[0]);
    split3(w.y, o[1]);
    split3(w.z, o[2]);
    split3(w.w, o[3]);
    __nv_bfloat16* d[3] = {p0, p1, p2};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      *reinterpret_cast<__nv_bfloat162*>(d[k] + 4 * i) = __halves2bfloat162(o[0][k], o[1][k]);
      *reinterpret_cast<__nv_bfloat162*>(d[k] + 4 * i + 2) = __halves2bfloat162(o[2][k], o[3][k]);
    }
  }
}

// out = sum over S fp32 partials of `stride` elements each, in order (count a multiple of 4).
template <typename T>
__global__ void __launch_bounds__(256)
    head_sum_kernel(const float* __restrict__ part, int S, long long stride, long long quads,
                    T* __restrict__ out) {
  pdl_trigger();
  pdl_wait();
  const long long step = (long long)gridDim.x * blockDim.x;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < quads; i += step) {
    float4 a = *reinterpret_cast<const float4*>(part + 4 * i);
    for (int k = 1; k < S; ++k) {
      const float4 b = *reinterpret_cast<const float4*>(part + k * stride + 4 * i);
      a.x += b.x;
      a.y += b.y;
      a.z += b.z;
      a.w += b.w;
    }
    if (sizeof(T) == 2) {
      *reinterpret_cast<uint2*>(out + 4 * i) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    } else {
      *reinterpret_cast<float4*>(out + 4 * i) = a;
    }
  }
}

// ---------------------------------------------------------------- host side
unsigned grid_for(long long items, int threads) {
  long long b = (items + threads - 1) / threads;
  const long long cap = (long long)sm_count() * 8;
  if (b > cap) b = cap;
  return (unsigned)(b < 1 ? 1 : b);
}

template <bool A_MN, bool B_MN, int EPI, bool OUT_F32>
poetx_status gemm(const HeadMaps& maps, HeadGemm p, cudaStream_t s) {
  auto k = head_gemm_kernel<A_MN, B_MN, EPI, OUT_F32>;
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  static int max_pairs = 0;
  std::call_once(once, [&] {
    attr_err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem);
    if (attr_err != cudaSuccess) return;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sm_count() / 2 * 2);
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = kGemmSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    attr_err = cudaOccupancyMaxActiveClusters(&max_pairs, k, &cfg);
    if (attr_err == cudaSuccess && max_pairs < 1) attr_err = cudaErrorInvalidConfiguration;
  });
  POETX_CUDA_TRY(attr_err);
  const long long tiles = (long long)p.tiles_m * p.tiles_n * p.splits;
  if (tiles > 0x7fffffffLL) return POETX_ERR_SHAPE;
  p.num_tiles = (int)tiles;
  p.err = device_error_word();
  p.limit_ns = kWaitLimitNs;
  const int pairs = (int)(tiles < max_pairs ? tiles : max_pairs);
  POETX_CUDA_TRY(launch_pdl_cluster(k, dim3(2 * pairs), dim3(kGemmThreads), kGemmSmem, s, 2, maps, p));
  POETX_CUDA_TRY(cudaGetLastError());
  after_launch(s, ST_HEAD_GEMM);
  return POETX_OK;
}

// The K splits of dx: enough work units to fill the pairs evenly, against the partials' traffic
// (per unit, a 64-wide K block of a 256 x 256 tile takes about 0.3 us of a pair, and the partials
// move at about 5 TB/s).
int dx_splits(long long rows, int D, int V) {
  const long long tiles = (long long)ceil_div(rows, 2 * BM) * ceil_div(D, BN);
  const int kb = ceil_div(V, BK), pairs = sm_count() / 2;
  int best = 1;
  double best_us = 1e30;
  for (int S = 1; S <= 64 && S <= kb; ++S) {
    const long long waves = (tiles * S + pairs - 1) / pairs;
    double us = (double)waves * (ceil_div(kb, S) * 0.3 + 2.0);
    if (S > 1) us += 3.0 + 8e-6 * (double)S * (double)rows * D / 5.0;
    if (us < best_us) {
      best_us = us;
      best = S;
    }
  }
  // every split non-empty
  return ceil_div(kb, ceil_div(kb, best));
}

constexpr size_t kPieceBytes = (size_t)1 << 30;  // bound of a piece's stored exponentials
constexpr int kMaxTargets = 1024;

struct Plan {
  bool f32, grads;
  long long Vp;      // columns of a stored row
  int groups;
  long long rows;    // rows of a piece
  int pieces;
  int splits;        // K splits of dx
  // workspace offsets
  size_t part, tl, ucol, slot, gstart, e, dz, xs, ws, acc, dxp, bytes;
};

bool plan(poetx_dtype dt, int N, int D, int V, int K, bool dx, bool dW, Plan* o) {
  if (N < 0 || D < 8 || D % 8 || D > (1 << 17) || V < 1 || V > (1 << 22) || K < 1 || K > kMaxTargets)
    return false;
  o->f32 = dt == POETX_F32;
  o->grads = dx || dW;
  o->Vp = (long long)align_up((size_t)V, 64);
  o->groups = ceil_div(V, kGroup);
  const size_t row_bytes = (o->grads ? (size_t)o->Vp * (o->f32 ? 10 : 2) : 0) +
                           (size_t)o->groups * 8 * (o->grads ? 1 : 4);
  long long rows = (long long)(kPieceBytes / row_bytes) / 256 * 256;
  if (rows < 256) rows = 256;
  if (rows > (1 << 18)) rows = 1 << 18;
  const long long n = N > 0 ? N : 1;
  o->pieces = ceil_div(n, rows);
  o->rows = o->pieces == 1 ? n : (long long)align_up((size_t)ceil_div(n, o->pieces), 256);
  o->pieces = ceil_div(n, o->rows);
  o->splits = dx ? dx_splits(o->rows, D, V) : 1;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += align_up(bytes, 1024);
    return a;
  };
  const size_t R = (size_t)o->rows;
  o->part = take(R * o->groups * sizeof(float2));
  o->tl = take(R * K * 4);
  // the sorted target lists of a distillation (a call with K = 1 may be either: both fit)
  o->ucol = take(R * K * 4);
  o->slot = take(R * K * 2);
  o->gstart = take(R * (o->groups + 1) * 2);
  o->e = o->grads ? take(R * o->Vp * (o->f32 ? 4 : 2)) : 0;
  o->dz = o->f32 && o->grads ? take(3 * align_up(R * o->Vp * 2, 1024)) : o->e;
  o->xs = o->f32 ? take(3 * align_up(R * D * 2, 1024)) : 0;
  o->ws = o->f32 ? take(3 * align_up((size_t)V * D * 2, 1024)) : 0;
  o->acc = !o->f32 && dW && o->pieces > 1 ? take((size_t)V * D * 4) : 0;
  o->dxp = o->splits > 1 ? take((size_t)o->splits * align_up(R, 256) * D * 4) : 0;
  o->bytes = at;
  return true;
}

bool bf16_map(CUtensorMap* m, const void* p, long long inner, long long outer, int bi, int bo) {
  return encode_tma_2d(m, p, TMA_BF16, inner, outer, inner, bi, bo, true);
}

void set_segs(HeadGemm* g, bool f32) {
  // small pieces first, so that the accumulator is small while they are added
  static const int8_t a[kMaxSegs] = {1, 0, 2, 1, 0, 0}, b[kMaxSegs] = {1, 2, 0, 0, 1, 0};
  g->nseg = f32 ? kMaxSegs : 1;
  for (int i = 0; i < kMaxSegs; ++i) {
    g->seg_a[i] = f32 ? a[i] : 0;
    g->seg_b[i] = f32 ? b[i] : 0;
  }
  // K of one accumulator: 512 (32 adds of 16 products) in bf16, 64 per piece pair in fp32
  g->chunk = f32 ? 1 : 8;
}

struct HeadCall {
  poetx_dtype dt;
  const void* x;
  int N, D;
  const void* W;
  int V;
  const int32_t* idx;
  const float* tlogit;
  int K;
  float T, zl;
  const float* dloss;
  float* loss;
  float* lse;
  void* dx;
  void* dW;
  int accumulate;
  void* ws;
  size_t ws_bytes;
};

poetx_status run_split(const float* src, long long count, uint8_t* dst, size_t step, cudaStream_t s) {
  POETX_CUDA_TRY(launch_pdl(head_split_kernel, dim3(grid_for(count / 4, 256)), dim3(256), 0, s,
                            reinterpret_cast<const float4*>(src), count / 4,
                            reinterpret_cast<__nv_bfloat16*>(dst),
                            reinterpret_cast<__nv_bfloat16*>(dst + step),
                            reinterpret_cast<__nv_bfloat16*>(dst + 2 * step)));
  POETX_CUDA_TRY(cudaGetLastError());
  after_launch(s, ST_HEAD_ROW);
  return POETX_OK;
}

poetx_status run_head(const HeadCall& c, cudaStream_t s) {
  if (c.N < 0 || c.D < 0 || c.V < 0) return POETX_ERR_ARG;
  if (c.dt != POETX_F32 && c.dt != POETX_BF16) return POETX_ERR_DTYPE;
  Plan pl;
  if (!plan(c.dt, c.N, c.D, c.V, c.K, c.dx, c.dW, &pl)) return POETX_ERR_SHAPE;
  const size_t esz = dtype_size(c.dt);
  if (!(c.T > 0.f) || !(c.zl >= 0.f)) return POETX_ERR_ARG;
  for (const void* q : {c.x, c.W, (const void*)c.idx, (const void*)c.tlogit, (const void*)c.dloss,
                        (const void*)c.loss, (const void*)c.lse, (const void*)c.dx,
                        (const void*)c.dW, (const void*)c.ws})
    if (!aligned16(q)) return POETX_ERR_ALIGN;
  if (c.N == 0) {
    if (c.dW && !c.accumulate)
      POETX_CUDA_TRY(cudaMemsetAsync(c.dW, 0, (size_t)c.V * c.D * esz, s));
    return POETX_OK;
  }
  if (!c.x || !c.W || !c.idx || !c.loss || !c.ws || (pl.grads && !c.dloss)) return POETX_ERR_ARG;
  if (c.ws_bytes < pl.bytes) return POETX_ERR_WORKSPACE;
  if (!umma_supported()) return POETX_ERR_UNSUPPORTED;
  const size_t row_smem = (size_t)pl.groups * 4 + (size_t)c.K * 12;
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [] {
    attr_err = cudaFuncSetAttribute(head_row_kernel<false>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (attr_err == cudaSuccess)
      attr_err = cudaFuncSetAttribute(head_row_kernel<true>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
  });
  POETX_CUDA_TRY(attr_err);

  uint8_t* w = static_cast<uint8_t*>(c.ws);
  const size_t x_step = align_up((size_t)pl.rows * c.D * 2, 1024);
  const size_t w_step = align_up((size_t)c.V * c.D * 2, 1024);
  const size_t z_step = align_up((size_t)pl.rows * pl.Vp * 2, 1024);
  const int np = pl.f32 ? 3 : 1;
  if (pl.f32)
    POETX_TRY(run_split(static_cast<const float*>(c.W), (long long)c.V * c.D, w + pl.ws, w_step, s));
  float2* part = reinterpret_cast<float2*>(w + pl.part);
  float* tl = reinterpret_cast<float*>(w + pl.tl);
  const uint8_t* wp = pl.f32 ? w + pl.ws : static_cast<const uint8_t*>(c.W);

  for (int pc = 0; pc < pl.pieces; ++pc) {
    const long long r0 = pc * pl.rows;
    const int rows = (int)((long long)c.N - r0 < pl.rows ? (long long)c.N - r0 : pl.rows);
    const uint8_t* xr = static_cast<const uint8_t*>(c.x) + (size_t)r0 * c.D * esz;
    const uint8_t* xp = pl.f32 ? w + pl.xs : xr;
    if (pl.f32)
      POETX_TRY(run_split(reinterpret_cast<const float*>(xr), (long long)rows * c.D, w + pl.xs,
                          x_step, s));
    // a teacher's entries: distinct columns in order
    const int32_t* idx = c.idx + r0 * c.K;
    const int32_t* ucol = idx;
    uint16_t* slot = reinterpret_cast<uint16_t*>(w + pl.slot);
    uint16_t* gstart = nullptr;
    if (c.tlogit) {
      int32_t* u = reinterpret_cast<int32_t*>(w + pl.ucol);
      gstart = reinterpret_cast<uint16_t*>(w + pl.gstart);
      POETX_CUDA_TRY(launch_pdl(head_targets_kernel, dim3(rows), dim3(256), (size_t)c.K * 12, s, idx,
                                c.K, c.V, pl.groups, slot, u, gstart));
      POETX_CUDA_TRY(cudaGetLastError());
      after_launch(s, ST_HEAD_ROW);
      ucol = u;
    }
    // the logits' product
    HeadMaps mp;
    HeadGemm g{};
    set_segs(&g, pl.f32);
    for (int i = 0; i < np; ++i)
      if (!bf16_map(&mp.a[i], xp + i * x_step, c.D, rows, 64, 128) ||
          !bf16_map(&mp.b[i], wp + i * w_step, c.D, c.V, 64, 128))
        return POETX_ERR_CUDA;
    g.tiles_m = ceil_div(rows, 2 * BM);
    g.tiles_n = ceil_div(c.V, BN);
    g.splits = 1;
    g.num_kb = g.kb_split = ceil_div(c.D, BK);
    g.M = rows;
    g.N = c.V;
    g.n_store = (int)pl.Vp;  // columns V .. Vp - 1 are stored as zeros
    g.scale2 = kLog2e / c.T;
    g.part = part;
    g.groups = pl.groups;
    g.ucol = ucol;
    g.gstart = gstart;
    g.K = c.K;
    g.tl = tl;
    g.store = pl.grads;
    if (pl.grads && !encode_tma_2d(&mp.c, w + pl.e, pl.f32 ? TMA_F32 : TMA_BF16, pl.Vp, rows, pl.Vp,
                                   pl.f32 ? 32 : 64, 32, true))
      return POETX_ERR_CUDA;
    if (!pl.grads) mp.c = mp.a[0];
    if (pl.f32)
      POETX_TRY((gemm<false, false, EPI_LSE, true>(mp, g, s)));
    else
      POETX_TRY((gemm<false, false, EPI_LSE, false>(mp, g, s)));
    // rows: lse, loss, dz
    RowArgs ra{};
    ra.V = c.V;
    ra.groups = pl.groups;
    ra.K = c.K;
    ra.pitch = pl.Vp;
    ra.part = part;
    ra.tl = tl;
    ra.idx = idx;
    ra.ucol = ucol;
    ra.slot = slot;
    ra.tlogit = c.tlogit ? c.tlogit + r0 * c.K : nullptr;
    ra.dloss = c.dloss ? c.dloss + r0 : nullptr;
    ra.T = c.T;
    ra.zl = c.zl;
    ra.loss = c.loss + r0;
    ra.lse = c.lse ? c.lse + r0 : nullptr;
    ra.e = pl.grads ? w + pl.e : nullptr;
    for (int i = 0; i < 3; ++i)
      ra.piece[i] = reinterpret_cast<__nv_bfloat16*>(w + pl.dz + i * z_step);
    if (pl.f32)
      POETX_CUDA_TRY(launch_pdl(head_row_kernel<true>, dim3(rows), dim3(kRowThreads), row_smem, s, ra));
    else
      POETX_CUDA_TRY(launch_pdl(head_row_kernel<false>, dim3(rows), dim3(kRowThreads), row_smem, s, ra));
    POETX_CUDA_TRY(cudaGetLastError());
    after_launch(s, ST_HEAD_ROW);
    // dx = dz W
    if (c.dx) {
      uint8_t* dxr = static_cast<uint8_t*>(c.dx) + (size_t)r0 * c.D * esz;
      HeadGemm h{};
      set_segs(&h, pl.f32);
      for (int i = 0; i < np; ++i)
        if (!bf16_map(&mp.a[i], w + pl.dz + i * z_step, pl.Vp, rows, 64, 128) ||
            !bf16_map(&mp.b[i], wp + i * w_step, c.D, c.V, 64, 64))
          return POETX_ERR_CUDA;
      h.tiles_m = ceil_div(rows, 2 * BM);
      h.tiles_n = ceil_div(c.D, BN);
      h.splits = pl.splits;
      h.num_kb = ceil_div(c.V, BK);
      h.kb_split = ceil_div(h.num_kb, h.splits);
      h.M = rows;
      h.N = h.n_store = c.D;
      h.c_rows = (int)align_up(rows, 256);
      const bool f32_out = pl.f32 || pl.splits > 1;
      const void* dst = pl.splits > 1 ? w + pl.dxp : dxr;
      const long long drows = pl.splits > 1 ? (long long)pl.splits * h.c_rows : rows;
      if (!encode_tma_2d(&mp.c, dst, f32_out ? TMA_F32 : TMA_BF16, c.D, drows, c.D, f32_out ? 32 : 64,
                         32, true))
        return POETX_ERR_CUDA;
      if (f32_out)
        POETX_TRY((gemm<false, true, EPI_STORE, true>(mp, h, s)));
      else
        POETX_TRY((gemm<false, true, EPI_STORE, false>(mp, h, s)));
      if (pl.splits > 1) {
        const long long quads = (long long)rows * c.D / 4;
        const float* pp = reinterpret_cast<const float*>(w + pl.dxp);
        const long long stride = (long long)h.c_rows * c.D;
        if (pl.f32)
          POETX_CUDA_TRY(launch_pdl(head_sum_kernel<float>, dim3(grid_for(quads, 256)), dim3(256), 0,
                                    s, pp, pl.splits, stride, quads, reinterpret_cast<float*>(dxr)));
        else
          POETX_CUDA_TRY(launch_pdl(head_sum_kernel<__nv_bfloat16>, dim3(grid_for(quads, 256)),
                                    dim3(256), 0, s, pp, pl.splits, stride, quads,
                                    reinterpret_cast<__nv_bfloat16*>(dxr)));
        POETX_CUDA_TRY(cudaGetLastError());
        after_launch(s, ST_HEAD_ROW);
      }
    }
    // dW (+)= dz^T x; between the pieces of a bf16 head the sum stays in fp32
    if (c.dW) {
      HeadGemm h{};
      set_segs(&h, pl.f32);
      for (int i = 0; i < np; ++i)
        if (!bf16_map(&mp.a[i], w + pl.dz + i * z_step, pl.Vp, rows, 64, 64) ||
            !bf16_map(&mp.b[i], xp + i * x_step, c.D, rows, 64, 64))
          return POETX_ERR_CUDA;
      h.tiles_m = ceil_div(c.V, 2 * BM);
      h.tiles_n = ceil_div(c.D, BN);
      h.n_fast = 1;
      h.splits = 1;
      h.num_kb = h.kb_split = ceil_div(rows, BK);
      h.M = c.V;
      h.N = h.n_store = c.D;
      h.c_rows = c.V;
      const bool first = pc == 0, last = pc + 1 == pl.pieces;
      const bool f32_out = pl.f32 || !last;
      void* dst = pl.f32 || last ? c.dW : static_cast<void*>(w + pl.acc);
      if (pl.f32)
        h.add_f32 = !first || c.accumulate ? static_cast<const float*>(c.dW) : nullptr;
      else
        h.add_f32 = !first ? reinterpret_cast<const float*>(w + pl.acc) : nullptr;
      if (!pl.f32 && last && c.accumulate) h.add_bf16 = static_cast<const __nv_bfloat16*>(c.dW);
      if (!encode_tma_2d(&mp.c, dst, f32_out ? TMA_F32 : TMA_BF16, c.D, c.V, c.D, f32_out ? 32 : 64,
                         32, true))
        return POETX_ERR_CUDA;
      if (f32_out)
        POETX_TRY((gemm<true, true, EPI_STORE, true>(mp, h, s)));
      else
        POETX_TRY((gemm<true, true, EPI_STORE, false>(mp, h, s)));
    }
  }
  return POETX_OK;
}

}  // namespace
}  // namespace poetx

using namespace poetx;

extern "C" size_t poetx_head_workspace_bytes(poetx_dtype dt, int N, int D, int V, int K, int want_dx,
                                             int want_dW) {
  Plan pl;
  if (dt != POETX_F32 && dt != POETX_BF16) return 0;
  if (!plan(dt, N, D, V, K, want_dx != 0, want_dW != 0, &pl)) return 0;
  return pl.bytes;
}

extern "C" poetx_status poetx_head_ce(poetx_dtype dt, const void* x, int N, int D, const void* W,
                                      int V, const int32_t* target, float z_loss, const float* dloss,
                                      float* loss, float* lse, void* dx, void* dW, int accumulate,
                                      void* ws, size_t ws_bytes, cudaStream_t stream) {
  const HeadCall c{dt, x,   N,   D,  W,  V,          target, nullptr, 1, 1.f, z_loss,
                   dloss, loss, lse, dx, dW, accumulate, ws,     ws_bytes};
  return run_head(c, stream);
}

extern "C" poetx_status poetx_head_distill(poetx_dtype dt, const void* x, int N, int D, const void* W,
                                           int V, const int32_t* t_index, const float* t_logit, int K,
                                           float temperature, const float* dloss, float* loss,
                                           float* lse, void* dx, void* dW, int accumulate, void* ws,
                                           size_t ws_bytes, cudaStream_t stream) {
  if (N > 0 && !t_logit) return POETX_ERR_ARG;
  const HeadCall c{dt, x,   N,   D,  W,  V,          t_index, t_logit, K, temperature, 0.f,
                   dloss, loss, lse, dx, dW, accumulate, ws,      ws_bytes};
  return run_head(c, stream);
}
