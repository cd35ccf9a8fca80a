// The gradients of the gated feed-forward block (ffn.cu) for few bf16 rows on the tensor cores:
//
//   dx = dz W,  dW = dz^T x,  dz [N][V] in two bf16 pieces, N <= 64
//
// Both are bound by W's way in and dW's way out, so a CTA takes them together, in units of 128 rows of W (and
// dW) by 128 columns: a job is a share of the rows for one block of columns.  W is the operand of 128 rows in
// dx^T = W^T dz^T (its columns; the tokens, first those of one piece and then those of the other, are the
// columns), whose accumulator stays for the whole job; dz^T is it in dW = dz^T x, with the pieces one behind
// the other along K.  The same tile of dz in shared memory serves both: its rows of 64 features are K-major
// as dx's second operand and MN-major as dW's first.  (With the tokens as rows of 256-row tiles, as for many
// tokens, the MMAs read the padding too and shared memory bounds both products: 16 x 4096 x 14336 took
// 100 us.)
//
// Warp 0 loads W and the block's columns of x, warp 10 dz, warp 1 issues the MMAs, and two sets of four
// warps (2 to 9) take turns with the units' accumulators of dW; at a job's end they write its sums of dx,
// which the head's kernel for partial sums adds up.  A job has at most 4096 rows, after which the tensor
// core's truncating adds are 1.5e-5 of the sum.
//
// 16 x 4096 x 14336: 470 MB in 82 us, dz before it and the sum of 9 partial sums included (5.7 TB/s); 64 rows
// 92 us; 64 x 2048 x 5632 25.4 us.
//
// Every mbarrier wait is bounded; on expiry the kernel records POETX_ERR_TIMEOUT, waits for its own copies,
// frees its TMEM and returns.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "pieces.cuh"

namespace poetx {

// Site id of this file's bounded waits (file id x 10000 + source line).
constexpr int kSite = 9 * 10000;

namespace {

constexpr int kUnit = 128;              // rows of W, and its columns
constexpr int kMaxUnits = 32;           // of a job
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (3 + kEpiWarps);
constexpr int kZWarp = 2 + kEpiWarps;
constexpr int kWBytes = kUnit * kUnit * 2;
constexpr int kBoxBytes = 32 * 128;     // a warp's 32 rows of 64 columns of dW
// Units on their way.  (Three: 86.5 us at 16 x 4096 x 14336 instead of 81, 22.6 at 9 x 2048 x 5632 instead
// of 23.3.)
constexpr int kStages = 2;
constexpr int z_bytes(int NT) { return 4 * NT * 128; }  // two pieces of two groups of 64 features
constexpr int x_bytes(int NT) { return 2 * NT * 128; }  // two groups of 64 columns
constexpr int fixed_bytes(int NT) { return 1024 + 512 + kEpiWarps * 2 * kBoxBytes + 2 * x_bytes(NT); }
constexpr int smem_of(int NT) { return fixed_bytes(NT) + kStages * (kWBytes + z_bytes(NT)); }
static_assert(smem_of(64) <= 227 * 1024, "few rows' gradients: shared memory");

struct Args {
  int blocks, splits, units;  // blocks of columns, jobs of a block, units of rows in all
  int N, D, V;
  int dx, dW;
  const __nv_bfloat16* old;  // dW's contents, added (nullable)
  const __nv_bfloat16 *z, *x;  // dz's first piece, [N][pitch], and x (for results that are NaN)
  long long pitch;
  float* dxp;                // [splits][N][D]
  int* err;
  unsigned long long limit_ns;
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
    few_grad_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mz,
                    const __grid_constant__ CUtensorMap mz2, const __grid_constant__ CUtensorMap mx,
                    const __grid_constant__ CUtensorMap mg, const Args p) {
  constexpr int STAGE = kWBytes + z_bytes(NT);
  constexpr uint32_t IDESC_X = make_idesc(kUnit, 2 * NT, true, false);
  constexpr uint32_t IDESC_W = make_idesc(kUnit, kUnit, true, true);
  constexpr uint32_t TMEM_COLS = 512, DX = 2 * kUnit;  // dW's two accumulators, then dx's two
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* const xs = smem + kStages * STAGE;
  uint8_t* const staging = xs + 2 * x_bytes(NT);
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kEpiWarps * 2 * kBoxBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;  // [2] dW's accumulator written, read
  uint64_t* tempty = tfull + 2;
  uint64_t* dfull = tempty + 2;      // [2] dx's
  uint64_t* dempty = dfull + 2;
  uint64_t* xfull = dempty + 2;      // [2] the block's x there, no longer needed
  uint64_t* xempty = xfull + 2;
  uint64_t* done = xempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 2);  // W's thread and dz's
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kEpiWarps / 2);
      mbar_init(&dfull[a], 1);
      mbar_init(&dempty[a], kEpiWarps);
      mbar_init(&xfull[a], 1);
      mbar_init(&xempty[a], 1);
    }
    mbar_init(done, 1);
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
  const int jobs = p.blocks * p.splits;
  auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag || !mbar_wait_bounded(bar, parity, p.err, p.limit_ns, site)) {
      *abort_flag = 1;
      return false;
    }
    return true;
  };
  // a job's block of columns and units
  auto job_at = [&](int job, int* col, int* u0, int* u1) {
    const int split = job / p.blocks;
    *col = (job - split * p.blocks) * kUnit;
    *u0 = (int)((long long)p.units * split / p.splits);
    *u1 = (int)((long long)p.units * (split + 1) / p.splits);
  };

  if ((warp == 0 || warp == kZWarp) && lane == 0) {
    // ------------------------------------------------------------ TMA producers
    const bool is_z = warp == kZWarp;
    Ring<kStages> rg;
    Ring<2> xr;
    int issued = 0, x_issued = 0;
    bool ok = true;
    for (int job = blockIdx.x; job < jobs && ok; job += gridDim.x) {
      int col, u0, u1;
      job_at(job, &col, &u0, &u1);
      if (!is_z && p.dW) {
        if (!(ok = wait(&xempty[xr.s], xr.ph ^ 1, kSite + __LINE__))) break;
        uint8_t* const at = xs + xr.s * x_bytes(NT);
        mbar_arrive_expect_tx(&xfull[xr.s], x_bytes(NT));
        tma_load_2d(at, &mx, &xfull[xr.s], col, 0);
        tma_load_2d(at + NT * 128, &mx, &xfull[xr.s], col + 64, 0);
        xr.next();
        ++x_issued;
      }
      for (int u = u0; u < u1; ++u, rg.next(), ++issued) {
        if (!(ok = wait(&empty[rg.s], rg.ph ^ 1, kSite + __LINE__))) break;
        uint8_t* const at = smem + rg.s * STAGE;
        uint64_t* const bar = &full[rg.s];
        if (is_z) {
          mbar_arrive_expect_tx(bar, z_bytes(NT));
#pragma unroll
          for (int j = 0; j < 2; ++j) {  // a group of 64 features: its second piece's tokens, its first's
            uint8_t* const z = at + kWBytes + j * 2 * NT * 128;
            tma_load_2d(z, &mz2, bar, u * kUnit + 64 * j, 0);
            tma_load_2d(z + NT * 128, &mz, bar, u * kUnit + 64 * j, 0);
          }
        } else if (p.dx) {
          mbar_arrive_expect_tx(bar, kWBytes);
          tma_load_2d(at, &mw, bar, col, u * kUnit);
          tma_load_2d(at + kWBytes / 2, &mw, bar, col + 64, u * kUnit);
        } else {
          mbar_arrive(bar);
        }
      }
    }
    // every copy has landed (of this thread, and where both went on, the other's)
    for (int j = issued - 1; j >= 0 && j >= issued - kStages; --j)
      mbar_wait_bounded(&full[j % kStages], (uint32_t)((j / kStages) & 1), p.err, p.limit_ns,
                        kSite + __LINE__);
    for (int j = x_issued - 1; j >= 0 && j >= x_issued - 2; --j)
      mbar_wait_bounded(&xfull[j & 1], (uint32_t)((j >> 1) & 1), p.err, p.limit_ns, kSite + __LINE__);
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------------ MMA issuer
    Ring<kStages> rg;
    Ring<2> acc, jr;
    bool ok = true;
    for (int job = blockIdx.x; job < jobs && ok; job += gridDim.x, jr.next()) {
      int col, u0, u1;
      job_at(job, &col, &u0, &u1);
      if (p.dW && !(ok = wait(&xfull[jr.s], jr.ph, kSite + __LINE__))) break;
      if (p.dx && !(ok = wait(&dempty[jr.s], jr.ph ^ 1, kSite + __LINE__))) break;
      tc_fence_after();
      const uint32_t dx = tmem_base + DX + (uint32_t)(jr.s * 2 * NT);
      const uint64_t xd = make_sdesc(smem_u32(xs) + jr.s * x_bytes(NT), NT * 128, 1024);
      for (int u = u0; u < u1; ++u, rg.next()) {
        if (!(ok = wait(&full[rg.s], rg.ph, kSite + __LINE__))) break;
        tc_fence_after();
        const uint32_t at = smem_base + rg.s * STAGE;
        if (p.dx) {
          const uint64_t wd = make_sdesc(at, kWBytes / 2, 1024);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint64_t zd = make_sdesc(at + kWBytes + j * 2 * NT * 128, 16, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k)  // (the address counts 16 bytes)
              umma_bf16(dx, wd + (4 * j + k) * 128, zd + 2 * k, IDESC_X, u != u0 || (j | k) != 0);
          }
        }
        if (p.dW) {
          if (!(ok = wait(&tempty[acc.s], acc.ph ^ 1, kSite + __LINE__))) break;
          tc_fence_after();
          const uint64_t zd = make_sdesc(at + kWBytes, 2 * NT * 128, 1024);
          const uint32_t d = tmem_base + (uint32_t)(acc.s * kUnit);
#pragma unroll
          for (int k = 0; k < 2 * NT / 16; ++k)
            umma_bf16(d, zd + k * 128, xd + k % (NT / 16) * 128, IDESC_W, k != 0);
          umma_commit(&tfull[acc.s]);
          acc.next();
        }
        umma_commit(&empty[rg.s]);
      }
      if (!ok) break;
      if (p.dx) umma_commit(&dfull[jr.s]);
      if (p.dW) umma_commit(&xempty[jr.s]);
    }
    // TMEM is freed after the final barrier: wait for the last MMAs
    umma_commit(done);
    mbar_wait_bounded(done, 0, p.err, p.limit_ns, kSite + __LINE__);
  } else if (warp >= 2 && warp < kZWarp) {
    // ------------------------------------------------------------ epilogue
    const int set = (warp - 2) >> 2, q = warp & 3;
    const uint32_t lanes = tmem_base + ((uint32_t)(q * 32) << 16);
    uint8_t* const stg = staging + (warp - 2) * 2 * kBoxBytes;
    Ring<2> jr;
    uint32_t ph = 0;
    int unit = 0;  // units so far
    bool ok = true;
    for (int job = blockIdx.x; job < jobs && ok; job += gridDim.x, jr.next()) {
      int col, u0, u1;
      job_at(job, &col, &u0, &u1);
      for (int u = u0; u < u1 && p.dW; ++u, ++unit) {
        if ((unit & 1) != set) continue;
        const bool got = wait(&tfull[set], ph, kSite + __LINE__);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        ph ^= 1;
        tc_fence_after();
        uint32_t r[4][32];
#pragma unroll
        for (int j = 0; j < 4; ++j) tmem_ld_32x32b_x32(lanes + (uint32_t)(set * kUnit + 32 * j), r[j]);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[set]);
        const int row_w = u * kUnit + q * 32, row = row_w + lane;
        if (row_w >= p.V) continue;
        if (lane == 0) bulk_wait_read<0>();  // the unit before has been read
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) {  // eight columns each
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r[i / 4][i % 4 * 8 + j]);
          if (p.old && row < p.V && col + 8 * i < p.D) {
            const uint4 w = *reinterpret_cast<const uint4*>(p.old + (long long)row * p.D + col + 8 * i);
            const uint32_t o[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[2 * j] += __uint_as_float(o[j] << 16);
              v[2 * j + 1] += __uint_as_float(o[j] & 0xffff0000u);
            }
          }
          const uint4 w = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                     pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
          *reinterpret_cast<uint4*>(stg + i / 8 * kBoxBytes + lane * 128 + (((i % 8) ^ (lane & 7)) << 4)) = w;
        }
        fence_async_shared();
        __syncwarp();
        if (staged_not_finite(stg, kBoxBytes, lane)) {
          first_piece_again(stg, kBoxBytes, lane, row < p.V, p.z + row, p.pitch, p.x, p.N, p.D, col, 1.f,
                            p.old ? p.old + (long long)row * p.D : nullptr);
          fence_async_shared();
          __syncwarp();
        }
        if (lane == 0) {
          tma_store_2d(&mg, stg, col, row_w);
          if (col + 64 < p.D) tma_store_2d(&mg, stg + kBoxBytes, col + 64, row_w);
          bulk_commit();
        }
      }
      if (!ok) break;
      if (p.dx) {
        const bool got = wait(&dfull[jr.s], jr.ph, kSite + __LINE__);
        if (!__all_sync(0xffffffffu, got)) break;
        tc_fence_after();
        const int c = col + q * 32 + lane;
        float* const out = p.dxp + (long long)(job / p.blocks) * p.N * p.D + c;
#pragma unroll 1
        for (int n = 16 * set; n < NT; n += 32) {
          uint32_t lo[16], hi[16];
          const uint32_t ta = lanes + DX + (uint32_t)(jr.s * 2 * NT + n);
          tmem_ld_32x32b_x16(ta, lo);
          tmem_ld_32x32b_x16(ta + NT, hi);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (n + i < p.N && c < p.D)
              out[(long long)(n + i) * p.D] = with_rest(__uint_as_float(hi[i]), __uint_as_float(lo[i]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&dempty[jr.s]);
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

template <int NT>
poetx_status launch(const CUtensorMap (&m)[5], const Args& a, cudaStream_t s) {
  auto k = few_grad_kernel<NT>;
  static PerDevice<cudaError_t> attr;
  POETX_CUDA_TRY(allow_smem(attr, k, smem_of(NT)));
  const int grid = (int)std::min<long long>((long long)a.blocks * a.splits, sm_count());
  POETX_CUDA_TRY(launch_pdl(k, dim3(grid), dim3(kThreads), smem_of(NT), s, m[0], m[1], m[2], m[3], m[4], a));
  POETX_CUDA_TRY(cudaGetLastError());
  after_launch(s, ST_FFN_GEMM);
  return POETX_OK;
}

int tokens_of(int N) { return N <= 16 ? 16 : (N <= 32 ? 32 : 64); }

}  // namespace

// Jobs of a block of columns: the number with the shortest longest CTA (a unit takes some 1.4 us of an SM at
// HBM's rate, a job 1 us besides), the partial sums' traffic added.
int few_splits(int N, int D, int V) {
  const int blocks = ceil_div(D, kUnit), units = ceil_div(V, kUnit), sms = sm_count();
  const int least = ceil_div(units, kMaxUnits);
  int best = least;
  double best_us = 1e30;
  for (int s = least; s <= units && s < least + 64; ++s) {
    const int each = ceil_div((long long)blocks * s, sms);
    const double us = each * (1.4 * ceil_div(units, s) + 1.0) + 8.0 * s * N * D / 5e6;
    if (us < best_us) {
      best_us = us;
      best = s;
    }
  }
  return best;
}

poetx_status few_gradients(const FewGradients& c, cudaStream_t s) {
  const int nt = tokens_of(c.N);
  CUtensorMap m[5];
  auto map = [&](int i, const void* ptr, long long inner, long long outer, long long pitch, int rows) {
    return encode_tma_2d(&m[i], ptr, TMA_BF16, inner, outer, pitch, 64, rows, true);
  };
  // (dz's columns behind V hold whatever was there: the map ends before them)
  if (!map(0, c.W, c.D, c.V, c.D, kUnit) || !map(1, c.dz, c.V, c.N, c.pitch, nt) ||
      !map(2, c.dz2, c.V, c.N, c.pitch, nt) || !map(3, c.x, c.D, c.N, c.D, nt) ||
      !map(4, c.dW ? c.dW : c.W, c.D, c.V, c.D, 32))
    return POETX_ERR_CUDA;
  Args a{};
  a.blocks = ceil_div(c.D, kUnit);
  a.splits = few_splits(c.N, c.D, c.V);
  a.units = ceil_div(c.V, kUnit);
  a.N = c.N;
  a.D = c.D;
  a.V = c.V;
  a.dx = c.dx != nullptr;
  a.dW = c.dW != nullptr;
  a.old = c.accumulate ? static_cast<const __nv_bfloat16*>(c.dW) : nullptr;
  a.z = static_cast<const __nv_bfloat16*>(c.dz);
  a.x = static_cast<const __nv_bfloat16*>(c.x);
  a.pitch = c.pitch;
  a.dxp = c.dxp;
  a.err = device_error_word();
  a.limit_ns = kWaitLimitNs;
  POETX_TRY((nt == 16 ? launch<16>(m, a, s) : (nt == 32 ? launch<32>(m, a, s) : launch<64>(m, a, s))));
  if (!c.dx) return POETX_OK;
  const long long count = (long long)c.N * c.D;
  return sum_partials(false, c.dxp, a.splits, count, count, c.dx, s);
}

}  // namespace poetx
