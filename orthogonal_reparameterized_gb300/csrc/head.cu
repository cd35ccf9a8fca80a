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
// (pack_exp: 11 significant bits down to 43 nats below m, so that its rounding, 2^-11, stays below the
// bf16 rounding of dz that follows; no fp32 logit is stored); (2) a row kernel that joins the groups into
// lse, writes the loss and turns the row into dz in place (bf16); (3) dx = dz W and dW (+)= dz^T x.  That
// is 6 N V D flops: nothing is computed twice.  The logits of the sparse targets leave the first product in
// fp32, and the groups' sums leave the targets out: with O the sum of all other exponentials and e
// the target's, -ln p = log1p(O / e) and p - 1 = -O / (O + e) keep their relative accuracy where p is
// near 1 (lse - z_t and p - 1 would cancel).
//
// The products run on tcgen05 in 2-CTA pairs (256 x 256 tiles, operands by TMA).  The tensor core
// truncates when it adds into its fp32 accumulator, which over a long K drifts by about 2^-24 of
// the sum per step; so after every `chunk` of K the partial tile moves from TMEM into the epilogue's
// registers and is added there with IEEE adds, while the next chunk runs in the other half of TMEM
// (K = 512 per chunk against 1024: 4 % of the products' time, which runs at the power limit).
//
// fp32 heads run on the same kernels: each fp32 operand is split into three bf16 pieces (8 + 8 + 8
// significant bits) and a product takes the six pairs of pieces whose weight is above 2^-24, the
// small ones first.  Their exp(z - m) is kept in fp32.
//
// Every mbarrier wait is bounded; on expiry the kernel records POETX_ERR_TIMEOUT, drains its own
// copies, frees its TMEM and returns.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "pieces.cuh"

namespace poetx {

// Site id of this file's bounded waits (file id x 10000 + source line).
constexpr int kSite = 6 * 10000;

namespace {

constexpr int BM = 128;           // rows per CTA (256 per pair)
constexpr int BN = 256;           // columns per pair tile
constexpr int BK = 64;
constexpr int kStages = 5;  // (6: 3 % slower at 8192 x 128256 x 4096; 4: dx and dW 4 % slower)
constexpr int kEpiWarps = 8;      // two per TMEM lane quarter, each 128 columns
constexpr int kBWarp = 2;         // the gradients' second producer
constexpr int kEpiWarp0 = 4;      // (whole warpgroups for the split of the registers)
constexpr int kGemmThreads = 32 * (kEpiWarp0 + kEpiWarps);
// Registers: 168 a thread at the launch, of which the first warpgroup keeps 72 and the epilogues' get 216.
constexpr int kFewRegs = 72, kManyRegs = 216;
static_assert(kFewRegs * 128 + kManyRegs * 32 * kEpiWarps == 168 * kGemmThreads, "registers");
constexpr int kGroup = 128;       // columns of one (max, sum) group
constexpr uint32_t kABytes = BM * BK * 2;
constexpr uint32_t kBBytes = BN / 2 * BK * 2;
constexpr uint32_t kStageBytes = kABytes + kBBytes;  // 32 KB per CTA
constexpr uint32_t kStgBytes = 32 * 128;             // one epilogue warp's box: 32 rows of 128 bytes
// Tiles of a raster band: the operand stripes of a band (32 MB at K = 4096) stay in L2 while the other
// operand streams past.  Bands of 4, 8, 16 and 32 at 8192 x 128256 x 4096 with gradients: 17.7, 17.1,
// 16.9 and 17.3 ms.
constexpr int kBand = 16;
constexpr int gemm_smem(int segs) {  // (SEGS == 2: two boxes a warp)
  return kStages * (int)kStageBytes + (segs == 2 ? 2 : 1) * kEpiWarps * (int)kStgBytes + 1024 + 512;
}
static_assert(gemm_smem(2) <= 227 * 1024, "head products: shared memory");
constexpr int kMaxSegs = 6;

struct HeadMaps {
  CUtensorMap a[3], b[3];  // the operands' pieces (one for bf16)
  CUtensorMap c;           // the stored tensor
};

// One product C[M, N] = A[M, K] B[N, K]^T over 256 x 256 tiles and K splits.
struct Product {
  int tiles_m, tiles_n, num_tiles;  // num_tiles: with the splits (the split varies slowest)
  int n_fast;            // raster: bands of kBand M tiles (1: N tiles), M (N) fastest in a band
  int num_kb, kb_split;  // 64-wide K blocks in all, per split
  int a_mn;              // A stored with its M axis contiguous ([K][M])
  int b_groups;          // B's map (MN-major) is one of 64-column groups: one box instead of two
  int M, N;              // valid rows and columns
  int n_store;           // columns of the stored tensor
  int c_rows;            // its rows per split
  int c_f32;             // stored in fp32, else 16 bits
  const float* add_f32;  // added before the store (nullable), as is
  const __nv_bfloat16* add_bf16;
};

struct HeadGemm {
  Product prod[2];       // the tiles of the first, then those of the second (none: num_tiles 0)
  int num_tiles;
  int chunk;             // K blocks per accumulator hand-over
  int8_t seg_a[kMaxSegs], seg_b[kMaxSegs];  // fp32: the operand pieces multiplied, in order
  // logits' product
  float scale2;          // log2(e) / T
  float2* part;          // [M][groups]
  int groups;
  const int32_t* ucol;   // [M][K] the rows' distinct target columns, ascending (K = 1: any value)
  const uint16_t* gstart;  // [M][groups + 1] first of them in each group; NULL: K = 1
  int K;
  float* tl;             // [M][K] their logits, before 1/T
  int store;             // whether exp(z - m) is stored
  const float* dloss;    // with store: [M] upstream gradients (lists: of the rows with one, else 0), whose
  float* unit;           //   largest magnitude goes to unit (head_unit), read back as
  const float* out_scale;  // gradients' products: factor of the sums (nullable: 1), times T
  float T;
  const __nv_bfloat16 *z, *x;  // dz in two pieces: the first, [rows][z_pitch], and x [rows][N]
  long long z_pitch;
  int rows;
  int* err;
  unsigned long long limit_ns;
};

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// exp(z - m) as it is stored, a number of [0, 1]: 6 bits of exponent and 10 of mantissa.  These are bits 28
// to 13 of the fp32 number 2^-64 times as large, whose upper ones are 0, rounded to nearest: 11 significant
// bits down to 2^-62 (43 nats below the group's maximum), fewer down to 2^-72.  (An fp16 would lose bits
// below 2^-14, 10 nats, and be 0 from 17 nats on: the gradients of rare entries in a head that has
// learned; 2^15 times as large in fp16 it would be exact to 20 nats.)  The factor 2^64 returns with the row
// kernel's factor of the group.  Four instructions per pair where fp16 takes one: nothing on wide heads
// (4096 x 32000 x 2048 with gradients 967 and 966 us), 3 % at 1000 x 16000 x 1024 (112.6 and 115.7 us), 6 %
// at 300 x 32000 x 512 (89 and 95 us), where the epilogues are a larger part.
constexpr float kExpStore = 0x1p-64f, kExpLoad = 0x1p64f;
__device__ __forceinline__ uint32_t pack_exp(float a, float b) {
  const float2 w = mul2(make_float2(a, b), both(kExpStore));
  return __byte_perm(8u * __float_as_uint(w.x) + 0x8000u, 8u * __float_as_uint(w.y) + 0x8000u, 0x7632);
}
__device__ __forceinline__ float2 unpack_exp(uint32_t u) {  // times 2^-64
  return make_float2(__uint_as_float((u << 13) & 0x1fffe000u), __uint_as_float((u >> 3) & 0x1fffe000u));
}

// K-major tile: rows of 128 bytes (64 along K), 8-row groups 1024 bytes apart, the k-th K = 16 slice
// 32 bytes further; MN-major tile: boxes of 64 K rows x 64 side by side (8 KB), the slice 16 rows
// (2048 bytes) further.
template <bool MN>
__device__ __forceinline__ uint64_t tile_desc(uint32_t base) {
  return MN ? make_sdesc(base, 8192, 1024) : make_sdesc(base, 16, 1024);
}

struct Tile {
  int which;  // product
  int mi, nt, split, kb0, kb1;
};
__device__ __forceinline__ Tile tile_of(const HeadGemm& p, int t) {
  Tile c;
  c.which = t >= p.prod[0].num_tiles;
  if (c.which) t -= p.prod[0].num_tiles;
  const Product& d = p.prod[c.which];
  const int per = d.tiles_m * d.tiles_n;
  c.split = t / per;
  const int r = t - c.split * per;
  const int fast = d.n_fast ? d.tiles_n : d.tiles_m, slow = d.n_fast ? d.tiles_m : d.tiles_n;
  const int f0 = r / (kBand * slow) * kBand;  // the band's first tile of the fast axis
  const int width = min(kBand, fast - f0), q = r - f0 * slow;
  const int f = f0 + q % width, o = q / width;
  c.mi = d.n_fast ? o : f;
  c.nt = d.n_fast ? f : o;
  c.kb0 = c.split * d.kb_split;
  c.kb1 = min(d.num_kb, c.kb0 + d.kb_split);
  return c;
}

// Bounded wait that looks at the abort flag only where the barrier is not ready.
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          const HeadGemm& p, int site) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*abort_flag || !mbar_wait_bounded(bar, parity, p.err, p.limit_ns, site)) {
    *abort_flag = 1;
    return false;
  }
  return true;
}

// The unit of dz: the largest |dloss| of the piece.  dz is kept over unit * T, so that with equal
// upstream gradients (a mean) the bf16 rounding sees p - q alone and not a constant's mantissa too;
// the sums get the factor back in fp32.  At most 2^100, so that with kExpLoad or T nothing overflows; 1
// where there is no finite positive maximum.
__device__ __forceinline__ float head_unit(float top) {
  return top > 0.f && isfinite(top) ? fminf(top, 0x1p100f) : 1.f;
}
// A row's share in that maximum: nothing where it has no gradient (target outside [0, V): ignored or bad),
// whatever its dloss holds.
__device__ __forceinline__ float unit_share(float dloss, int target, int V) {
  return (unsigned)target < (unsigned)V ? fabsf(dloss) : 0.f;
}

// LSE: the logits' product with its softmax epilogue (one product, both operands K-major).
// Otherwise the gradients' products, dx and dW in one launch, so that the second's tiles fill the
// first's last wave.  Warps 0 and 2 of each CTA load its 128 rows of A and its half of B, one thread
// of the even CTA's warp 1 issues the MMAs, warps 4-11 read the accumulators back (warp w: rows
// 32 (w % 4).. of the CTA's 128, columns 128 ((w - 4) / 4)..).
//
// Bound by the tensor pipe, and in a run of calls by the board's power.  4096 x 32000 x 2048: logits
// 307-335 us (1.6-1.75 PFLOP/s, tensor pipe 79 % active), dx and dW 592-615 us (1.75-1.81, 86 %);
// 8192 x 128256 x 4096: 5.0-5.3 ms and 9.6-10.2 ms at 1.4-1.55 GHz.
template <bool LSE, int SEGS>
__global__ void __launch_bounds__(kGemmThreads, 1)
    head_gemm_kernel(const __grid_constant__ HeadMaps maps0, const __grid_constant__ HeadMaps maps1,
                     const __grid_constant__ HeadGemm p) {
  constexpr bool F32 = SEGS == kMaxSegs;
  // SEGS == 2: gradients of at most 128 rows with dz in two pieces.  dx's tile holds the first piece's
  // rows in the even CTA and the second's in the odd one, which would multiply padding otherwise (their
  // sums are added with those of the splits); dW's K axis runs over the second piece, then the first.
  constexpr bool FINE = SEGS == 2;
  // (Its dW's tiles have at most four K blocks and little but an epilogue: both of a warp's boxes are
  // staged at once.)
  constexpr int BOXES = FINE ? 2 : 1, STAGES = kStages;
  constexpr uint32_t STG = BOXES * kStgBytes;
  constexpr uint32_t B_OFF = kABytes, STAGE = kStageBytes;
  constexpr int STEPS = F32 ? SEGS : 1;  // stages per K block
  constexpr uint32_t TMEM_COLS = 2 * BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* staging = smem + STAGES * STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kEpiWarps * STG);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;  // [2] accumulator written
  uint64_t* tempty = tfull + 2;       // [2] accumulator read by both CTAs' epilogue warps
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int crank = (int)cluster_ctarank();
  pdl_trigger();
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kEpiWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps0.a[0]);
    tma_prefetch_desc(&maps0.b[0]);
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
  // With target lists the kernel before this one made them, and started it after everything earlier
  // was complete: only the epilogue, which reads the lists and writes, waits for it (and the warp that
  // makes dz's unit from what that kernel left of dloss).
  if (!LSE || !p.gstart || warp >= kEpiWarp0 || (warp == 1 && blockIdx.x == 1)) pdl_wait();
  const int t0 = (int)blockIdx.x / 2, t_step = (int)gridDim.x / 2;

  if (warp < kEpiWarp0) {
    regs_give<kFewRegs>();
    if ((warp == 0 || (!LSE && warp == kBWarp)) && lane == 0) {
      // ------------------------------------------------------------ TMA producers
      // gradients: warp 0 loads A, warp 2 B (each up to two boxes); logits: warp 0 both (two warps
      // measured 3 % slower there, one 6 % slower for the gradients)
      const bool is_b = !LSE && warp == kBWarp;
      Ring<STAGES> rg;
      bool ok = true;
      long long issued = 0;
      const uint32_t full0 = mapa_shared(full, 0);  // the even CTA's barriers
      uint8_t* const dst0 = smem + (is_b ? B_OFF : 0);
      for (int t = t0; t < p.num_tiles && ok; t += t_step) {
        const Tile c = tile_of(p, t);
        const HeadMaps& maps = c.which ? maps1 : maps0;
        const CUtensorMap* const set = is_b ? maps.b : maps.a;
        const int8_t* const seg = is_b ? p.seg_b : p.seg_a;
        // the operand's first row of M (N), and how it is loaded: K-major; MN-major as one box of two
        // 64-column groups (dz: always) or as two boxes
        const bool a_mn = !LSE && p.prod[c.which].a_mn;
        const int r0 = is_b ? c.nt * BN + crank * (BN / 2)
                            : (FINE && !a_mn ? 0 : (2 * c.mi + crank) * BM);
        const int half = FINE && a_mn ? p.prod[c.which].num_kb / 2 : 0;
        const int how = LSE ? 0 : (is_b ? (p.prod[c.which].b_groups ? 1 : 2) : a_mn);
        const bool expect = !is_b && crank == 0;
        for (int c0 = c.kb0; c0 < c.kb1 && ok; c0 += p.chunk) {
          const int len = min(c.kb1 - c0, p.chunk);
          int sg = 0, i = 0;  // a chunk's K blocks once per pair of pieces
          for (int j = 0; j < len * STEPS; ++j, rg.next(), ++issued) {
            if (!ring_wait(&empty[rg.s], rg.ph ^ 1, abort_flag, p, kSite + __LINE__)) {
              ok = false;
              break;
            }
            uint8_t* dst = dst0 + rg.s * STAGE;
            const int at = sg;
            const CUtensorMap* m = F32 ? &set[seg[at]] : set;
            int k = (c0 + i) * BK;
            if (FINE) {
              if (!is_b) m = set + (a_mn ? c0 + i < half : crank);
              if (c0 + i >= half) k -= half * BK;
            }
            if (++i == len) {
              i = 0;
              ++sg;
            }
            if (expect) mbar_arrive_expect_tx(&full[rg.s], 2 * STAGE);
            const uint32_t fb = full0 + rg.s * 8;
            if (how == 0) {
              tma_load_2d_pair(dst, m, fb, k, r0);
              if (LSE)
                tma_load_2d_pair(dst + B_OFF, &maps.b[F32 ? p.seg_b[at] : 0], fb, k,
                                 c.nt * BN + crank * (BN / 2));
            } else if (how == 1) {
              tma_load_3d_pair(dst, m, fb, 0, k, r0 / 64);
            } else {
              tma_load_2d_pair(dst, m, fb, r0, k);
              tma_load_2d_pair(dst + 8192, m, fb, r0 + 64, k);
            }
          }
        }
      }
      // no copy may be in flight when the CTA exits: the MMAs release a stage after reading it
      for (long long j = issued - 1; j >= 0 && j >= issued - STAGES; --j)
        mbar_wait_bounded(&empty[j % STAGES], (uint32_t)((j / STAGES) & 1), p.err, p.limit_ns,
                          kSite + __LINE__);
    } else if (warp == 1 && lane == 0 && crank == 0) {
      // ------------------------------------------------------------ MMA issuer
      Ring<STAGES> rg;
      Ring<2> acc;
      bool any = false;
      // one tile; the operands' orders are compile-time constants (as run-time values they cost the
      // issuing thread 15 % of the products' time)
      auto tile = [&](const Tile& c, auto a_mn_t) -> bool {
        constexpr bool A_MN = decltype(a_mn_t)::value, B_MN = !LSE;
        constexpr uint32_t IDESC = make_idesc(2 * BM, BN, A_MN, B_MN);
        for (int kb = c.kb0; kb < c.kb1; kb += p.chunk, acc.next()) {
          if (!ring_wait(&tempty[acc.s], acc.ph ^ 1, abort_flag, p, kSite + __LINE__)) return false;
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(acc.s * BN);
          const int blocks = (min(c.kb1, kb + p.chunk) - kb) * STEPS;
          for (int j = 0; j < blocks; ++j, rg.next()) {
            if (!ring_wait(&full[rg.s], rg.ph, abort_flag, p, kSite + __LINE__)) return false;
            tc_fence_after();
            const uint32_t a_base = smem_base + rg.s * STAGE;
            const uint64_t bd = tile_desc<B_MN>(a_base + B_OFF);
            const uint64_t ad = tile_desc<A_MN>(a_base);
#pragma unroll
            for (int k = 0; k < BK / 16; ++k)  // (the address counts 16 bytes in the low bits)
              umma_bf16_pair(d, ad + k * (A_MN ? 128 : 2), bd + k * (B_MN ? 128 : 2), IDESC,
                             (j | k) != 0);
            umma_commit_pair(&empty[rg.s]);
          }
          umma_commit_pair(&tfull[acc.s]);
          any = true;
        }
        return true;
      };
      for (int t = t0; t < p.num_tiles; t += t_step) {
        const Tile c = tile_of(p, t);
        if (!(!LSE && p.prod[c.which].a_mn ? tile(c, std::true_type{}) : tile(c, std::false_type{})))
          break;
      }
      if (any) {  // TMEM is freed after the final barrier: wait for the last hand-over's MMAs
        const int last = acc.s ^ 1;
        mbar_wait_bounded(&tfull[last], last ? acc.ph ^ 1 : acc.ph, p.err, p.limit_ns,
                          kSite + __LINE__);
      }
    } else if (LSE && warp == 1 && blockIdx.x == 1 && p.store) {
      // ------------------------------------------------------------ an idle warp: the unit of dz
      float top = 0.f;
      const int M = p.prod[0].M, V = p.prod[0].N, quads = M / 4;
      const float4* d4 = reinterpret_cast<const float4*>(p.dloss);
      const int4* t4 = reinterpret_cast<const int4*>(p.ucol);
#pragma unroll 4
      for (int r = lane; r < quads; r += 32) {
        const float4 w = d4[r];
        const int4 t = p.gstart ? make_int4(0, 0, 0, 0) : t4[r];
        top = fmaxf(fmaxf(top, fmaxf(unit_share(w.x, t.x, V), unit_share(w.y, t.y, V))),
                    fmaxf(unit_share(w.z, t.z, V), unit_share(w.w, t.w, V)));
      }
      if (lane < M - 4 * quads) {
        const int r = 4 * quads + lane;
        top = fmaxf(top, unit_share(p.dloss[r], p.gstart ? 0 : p.ucol[r], V));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (lane == 0) *p.unit = head_unit(top);
    }
  } else {
    regs_take<kManyRegs>();
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int cbeg = ((warp - kEpiWarp0) >> 2) * kGroup;
    uint8_t* stg = staging + (warp - kEpiWarp0) * STG;
    const float out_scale = LSE ? 1.f : (p.out_scale ? *p.out_scale * p.T : p.T);
    Ring<2> acc;
    bool ok = true;
    for (int t = t0; t < p.num_tiles && ok; t += t_step) {
      const Tile c = tile_of(p, t);
      const Product& d = p.prod[LSE ? 0 : c.which];
      const int row_w = (2 * c.mi + crank) * BM + q * 32;  // the warp's first row
      const int row = row_w + lane;
      const int col0 = c.nt * BN + cbeg;
      // the row's targets in this group: [u0, u1) of its list (read ahead of the wait)
      int u0 = 0, u1 = 0;
      if (LSE && row < d.M && col0 < d.N) {
        if (p.gstart) {
          const uint16_t* gs = p.gstart + (long long)row * (p.groups + 1) + col0 / kGroup;
          u0 = gs[0];
          u1 = gs[1];
        } else {
          const int tc = p.ucol[row];
          u1 = tc >= col0 && tc < min(col0 + kGroup, d.N);
        }
      }
      float v[kGroup];
      for (int kb = c.kb0; kb < c.kb1; kb += p.chunk, acc.next()) {
        const int a = acc.s;
        const bool got = ring_wait(&tfull[a], acc.ph, abort_flag, p, kSite + __LINE__);
        if (!__all_sync(0xffffffffu, got)) {
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
      if (!ok) break;
      if (col0 >= d.N || (FINE && !d.a_mn ? q * 32 : row_w) >= d.M) continue;
      if (LSE) {
        if (col0 + kGroup > d.N) {
#pragma unroll
          for (int i = 0; i < kGroup; ++i)
            if (col0 + i >= d.N) v[i] = __int_as_float(0xff800000);  // -inf: exp 0
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
        m = __fmul_ru(m, p.scale2);  // rounded up: no stored exponential is above 1
        const float off = m == __int_as_float(0xff800000) ? 0.f : m;  // a group of -inf sums to 0
        float2 sum = both(0.f);
#pragma unroll
        for (int i = 0; i < kGroup; i += 2) {
          const float2 z = fma2(make_float2(v[i], v[i + 1]), both(p.scale2), both(-off));
          v[i] = ex2(z.x);
          v[i + 1] = ex2(z.y);
          sum = add2(sum, make_float2(v[i], v[i + 1]));
        }
        if (row < d.M)
          p.part[(long long)row * p.groups + (col0 / kGroup)] = make_float2(m, sum.x + sum.y);
        if (!p.store) continue;
      } else {
#pragma unroll
        for (int i = 0; i < kGroup; i += 2) {
          const float2 w = mul2(make_float2(v[i], v[i + 1]), both(out_scale));
          v[i] = w.x;
          v[i + 1] = w.y;
        }
        if (d.add_f32 && row < d.M) {
          const float* src = d.add_f32 + (long long)row * d.N + col0;
#pragma unroll
          for (int i = 0; i < kGroup; i += 4)
            if (col0 + i < d.N) {  // N is a multiple of 8
              const float4 w = *reinterpret_cast<const float4*>(src + i);
              v[i] += w.x;
              v[i + 1] += w.y;
              v[i + 2] += w.z;
              v[i + 3] += w.w;
            }
        }
        if (!F32 && d.add_bf16 && row < d.M) {
          const __nv_bfloat16* src = d.add_bf16 + (long long)row * d.N + col0;
#pragma unroll
          for (int i = 0; i < kGroup; i += 8)
            if (col0 + i < d.N) {
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
      const int orow = LSE ? row_w : c.split * d.c_rows + row_w;
      const CUtensorMap* mc = &(c.which ? maps1 : maps0).c;
      auto fill = [&](uint8_t* at, auto chunk) {  // chunk(i): 16 bytes i of the lane's row
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(at + lane * 128 + ((i ^ (lane & 7)) << 4)) = chunk(i);
      };
      auto box = [&](int j, auto chunk) {
        if (lane == 0) bulk_wait_read<0>();  // the previous box has been read
        __syncwarp();
        fill(stg, chunk);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(mc, stg, col0 + j, orow);
          bulk_commit();
        }
      };
      if (F32 || (!LSE && d.c_f32)) {
#pragma unroll
        for (int j = 0; j < kGroup; j += 32) {
          if (col0 + j >= d.n_store) break;
          box(j, [&](int i) {
            const float* f = v + j + 4 * i;
            return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                              __float_as_uint(f[3]));
          });
        }
      } else {
        auto half = [&](int j) {  // 64 columns from j
          return [&v, j](int i) {
            const float* f = v + j + 8 * i;
            auto two = [](float lo, float hi) {
              return LSE ? pack_exp(lo, hi) : pack_bf16x2(lo, hi);
            };
            return make_uint4(two(f[0], f[1]), two(f[2], f[3]), two(f[4], f[5]), two(f[6], f[7]));
          };
        };
        if (FINE) {
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
          fill(stg, half(0));
          fill(stg + (BOXES - 1) * kStgBytes, half(64));
          fence_async_shared();
          __syncwarp();
          auto send = [&]() {
            if (lane != 0) return;
            tma_store_2d(mc, stg, col0, orow);
            if (col0 + 64 < d.n_store) tma_store_2d(mc, stg + (BOXES - 1) * kStgBytes, col0 + 64, orow);
            bulk_commit();
          };
          // (looked at behind the store, where it costs 1 % and not 3, unless the store overwrites what is added)
          bool bad = d.add_bf16 && staged_not_finite(stg, kStgBytes, lane);
          if (!bad) {
            send();
            bad = !d.add_bf16 && staged_not_finite(stg, kStgBytes, lane);
            if (bad && lane == 0) bulk_wait_all();
          }
          if (bad) {
            __syncwarp();
            first_piece_again(stg, kStgBytes, lane, row < d.M, p.z + row, p.z_pitch, p.x, p.rows, d.N, col0,
                              out_scale, d.add_bf16 ? d.add_bf16 + (long long)row * d.N : nullptr);
            fence_async_shared();
            __syncwarp();
            send();
          }
        } else {
#pragma unroll
          for (int j = 0; j < kGroup; j += 64) {
            if (col0 + j >= d.n_store) break;
            box(j, half(j));
          }
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

// ---------------------------------------------------------------- few rows
// The logits' product for at most 128 rows (a next token's score, a few sequences' ends, a short
// step): bound by reading W once, so the roles are swapped.  W is the 128-row operand (one CTA, tiles
// of `height` vocabulary rows, chosen so that every SM gets the same number of them), the NT (16 to
// 128) padded tokens are the columns, and nearly all of the shared memory is a ring of W tiles in
// flight.  A warp of the epilogue holds 32 vocabulary rows: it takes the targets out, turns its
// 32 x NT logits over through shared memory and leaves one (max, sum) per token and, where the
// gradients are wanted, the 32 values exp(z - max) of each token in 16 bits.  1 x 32000 x 2048: 131 MB
// in 22 us among other calls (26.6 us from a cold start); 3 x 100003 x 3000 with the store: 600 MB in
// 115 us (5.2 TB/s).
struct HeadScore {
  int tiles, height;       // height: a multiple of 8 (the swizzle's rows)
  int V, rows, stages;
  int kps;                 // K blocks per stage: 1 (two-dimensional maps), or the groups of the maps
  int num_st, chunk;       // stages per tile, per accumulator hand-over
  float scale2;
  float2* part;            // [rows][4 tiles]
  const int32_t* ucol;     // [rows][K] the rows' distinct target columns
  const uint16_t* gstart;  // [rows][tiles + 1] first of them in each tile; NULL: K = 1
  int K;
  float* tl;               // [rows][K]
  uint16_t* e;             // [rows][pitch] exp(z - max); NULL: the loss alone
  long long pitch;
  const float* dloss;      // with e: [rows], whose largest magnitude goes to unit (as in HeadGemm)
  float* unit;
  int* err;
  unsigned long long limit_ns;
};
constexpr int kScoreRows = 128;       // rows at most
constexpr int kScoreThreads = 64 + 128;
constexpr int kScoreRing = 12;        // stages at most
constexpr int kScoreSmem = 220 * 1024;
constexpr int score_turn_bytes(int NT) { return 4 * 32 * (NT + 1) * 4; }
int score_stage_bytes(int NT, int height, int kps) { return kps * (height + NT) * BK * 2; }

template <int NT>
__global__ void __launch_bounds__(kScoreThreads, 1)
    head_score_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mx,
                      const HeadScore p) {
  constexpr uint32_t IDESC = make_idesc(BM, NT, false, false);
  constexpr uint32_t TMEM_COLS = 2 * NT;
  const uint32_t a_kb = (uint32_t)p.height * BK * 2, x_off = p.kps * a_kb;  // one K block; the tokens
  const uint32_t stage = x_off + p.kps * NT * BK * 2;
  constexpr int TOK = (NT + 31) / 32;  // tokens a lane looks after
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  float* turn = reinterpret_cast<float*>(smem + p.stages * stage);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.stages * stage +
                                               (score_turn_bytes(NT) + 15) / 16 * 16);
  uint64_t* empty = full + kScoreRing;
  uint64_t* tfull = empty + kScoreRing;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mW);
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
  if (!p.gstart || warp >= 2) pdl_wait();  // (as in the products: the copies need not wait for the lists)
  auto wait = [&](uint64_t* bar, uint32_t parity, int site) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag || !mbar_wait_bounded(bar, parity, p.err, p.limit_ns, site)) {
      *abort_flag = 1;
      return false;
    }
    return true;
  };
  int s = 0;
  uint32_t ph = 0;
  auto next = [&]() {
    if (++s == p.stages) {
      s = 0;
      ph ^= 1;
    }
  };
  if (warp == 0 && lane == 0) {
    int issued = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x)
      for (int kb = 0; kb < p.num_st * p.kps; kb += p.kps, next(), ++issued) {
        if (!wait(&empty[s], ph ^ 1, kSite + __LINE__)) {
          ok = false;
          break;
        }
        uint8_t* sa = smem + s * stage;
        mbar_arrive_expect_tx(&full[s], stage);
        if (p.kps > 1) {
          tma_load_3d(sa, &mW, &full[s], 0, t * p.height, kb);
          tma_load_3d(sa + x_off, &mx, &full[s], 0, 0, kb);
        } else {
          tma_load_2d(sa, &mW, &full[s], kb * BK, t * p.height);
          tma_load_2d(sa + x_off, &mx, &full[s], kb * BK, 0);
        }
      }
    for (int j = issued - 1; j >= 0 && j >= issued - p.stages; --j)  // every copy has landed
      mbar_wait_bounded(&full[j % p.stages], (uint32_t)((j / p.stages) & 1), p.err, p.limit_ns,
                        kSite + __LINE__);
  } else if (warp == 1 && lane == 0) {
    Ring<2> acc;
    bool any = false, ok = true;
    for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x)
      for (int st0 = 0; st0 < p.num_st && ok; st0 += p.chunk, acc.next()) {
        if (!wait(&tempty[acc.s], acc.ph ^ 1, kSite + __LINE__)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(acc.s * NT);
        const int len = min(p.num_st - st0, p.chunk);
        for (int j = 0; j < len; ++j, next()) {
          if (!wait(&full[s], ph, kSite + __LINE__)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // (rows past `height` of the 128 are whatever follows in shared memory: not looked at)
          const uint32_t a_base = smem_base + s * stage;
          for (int i = 0; i < p.kps; ++i) {
            const uint64_t ad = tile_desc<false>(a_base + i * a_kb);
            const uint64_t bd = tile_desc<false>(a_base + x_off + i * NT * BK * 2);
#pragma unroll
            for (int k = 0; k < BK / 16; ++k)
              umma_bf16(d, ad + k * 2, bd + k * 2, IDESC, (j | i | k) != 0);
          }
          umma_commit(&empty[s]);
        }
        umma_commit(&tfull[acc.s]);
        any = true;
      }
    if (any) {
      const int last = acc.s ^ 1;
      mbar_wait_bounded(&tfull[last], last ? acc.ph ^ 1 : acc.ph, p.err, p.limit_ns,
                        kSite + __LINE__);
    }
  } else if (warp >= 2) {
    const int q = warp & 3;
    float* tw = turn + q * 32 * (NT + 1);
    const float ninf = __int_as_float(0xff800000);
    if (p.e && blockIdx.x == 0 && warp == 2) {
      float top = 0.f;
      for (int r = lane; r < p.rows; r += 32)
        top = fmaxf(top, unit_share(p.dloss[r], p.gstart ? 0 : p.ucol[r], p.V));
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (lane == 0) *p.unit = head_unit(top);
    }
    Ring<2> acc;
    bool ok = true;
    for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
      const int v0 = t * p.height, mine = q * 32 + lane;  // the lane's vocabulary row in the tile
      const int vrow = mine < p.height && v0 + mine < p.V ? v0 + mine : -1;
      // targets of the lane's tokens in this tile (read ahead of the wait)
      int u0[TOK], u1[TOK];
#pragma unroll
      for (int j = 0; j < TOK; ++j) {
        const int c = lane + 32 * j;
        u0[j] = u1[j] = 0;
        if (c < p.rows) {
          if (p.gstart) {
            const uint16_t* gs = p.gstart + (long long)c * (p.tiles + 1) + t;
            u0[j] = gs[0];
            u1[j] = gs[1];
          } else {
            const int tc = p.ucol[c];
            u1[j] = tc >= v0 && tc < min(v0 + p.height, p.V);
          }
        }
      }
      float v[NT];
      for (int st0 = 0; st0 < p.num_st; st0 += p.chunk, acc.next()) {
        const bool got = wait(&tfull[acc.s], acc.ph, kSite + __LINE__);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t ta = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc.s * NT);
#pragma unroll
        for (int j = 0; j < NT; j += 16) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(ta + j, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            v[j + i] = st0 == 0 ? __uint_as_float(r[i]) : v[j + i] + __uint_as_float(r[i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc.s]);
      }
      if (!ok) break;
#pragma unroll
      for (int c = 0; c < NT; ++c) tw[lane * (NT + 1) + c] = vrow >= 0 ? v[c] : ninf;
#pragma unroll
      for (int j = 0; j < TOK; ++j) {  // the targets leave through their vocabulary row's lane
        uint32_t hit = __ballot_sync(0xffffffffu, u0[j] < u1[j]);
        while (hit) {
          const int i = __ffs(hit) - 1, c = 32 * j + i;
          hit &= hit - 1;
          const int b = __shfl_sync(0xffffffffu, u0[j], i), e = __shfl_sync(0xffffffffu, u1[j], i);
          for (int u = b; u < e; ++u)
            if (p.ucol[(long long)c * p.K + u] == vrow) {
              p.tl[(long long)c * p.K + u] = tw[lane * (NT + 1) + c];
              tw[lane * (NT + 1) + c] = ninf;
            }
        }
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < TOK; ++j) {
        const int c = lane + 32 * j;
        if (c < p.rows) {
          float m = ninf;
#pragma unroll
          for (int r = 0; r < 32; ++r) m = fmaxf(m, tw[r * (NT + 1) + c]);
          m = __fmul_ru(m, p.scale2);
          const float off = m == ninf ? 0.f : m;
          float sum = 0.f;
          uint16_t* er = p.e + c * p.pitch + v0 + q * 32;  // (v0 is a multiple of 8: 16-byte stores)
#pragma unroll
          for (int r = 0; r < 32; r += 8) {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = ex2(fmaf(tw[(r + 2 * i) * (NT + 1) + c], p.scale2, -off));
              const float b = ex2(fmaf(tw[(r + 2 * i + 1) * (NT + 1) + c], p.scale2, -off));
              sum += a + b;
              u[i] = pack_exp(a, b);
            }
            if (p.e && q * 32 + r < p.height && v0 + q * 32 + r < p.pitch)
              *reinterpret_cast<uint4*>(er + r) = make_uint4(u[0], u[1], u[2], u[3]);
          }
          p.part[(long long)c * (4 * p.tiles) + 4 * t + q] = make_float2(m, sum);
          if (p.e && q == 0 && t == p.tiles - 1)  // the rest of the row's padding
            for (long long k = (long long)p.tiles * p.height; k < p.pitch; k += 8)
              *reinterpret_cast<uint4*>(p.e + c * p.pitch + k) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      __syncwarp();
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

// ---------------------------------------------------------------- CUDA-core kernels
constexpr uint16_t kNoSlot = 0xffff;
constexpr int kMaxTargets = 1024;

// A row's K target columns: slot[k] = place of idx[k] among the row's distinct columns in ascending
// order (kNoSlot for an absent entry or one beyond the vocabulary), ucol = those columns, gstart =
// the first of them in each group of `width` columns; up = its dloss, or 0 where the row has no gradient (no
// entry, only ones of weight 0, or one beyond the vocabulary).  A sort by ranks (K is at most a thousand; each
// thread compares its entry with all others, four per read), then a scan of the changes of column.  The
// logits' product needs the lists in its epilogue only, and starts beside this kernel: the trigger comes
// after the wait, so that what precedes this kernel is complete when the next one's copies begin.
constexpr int kListThreads = 256;
__global__ void __launch_bounds__(kListThreads)
    head_targets_kernel(const int32_t* __restrict__ idx, int K, int V, int groups, int width,
                        uint16_t* __restrict__ slot, int32_t* __restrict__ ucol,
                        uint16_t* __restrict__ gstart, const float* __restrict__ tlogit, float invT,
                        const float* __restrict__ dloss, float* __restrict__ up) {
  extern __shared__ __align__(16) int tsm[];
  const int K4 = (K + 3) / 4 * 4;
  int* is = tsm;         // [K4] columns, none: the largest integer
  int* ss = is + K4;     // [K4] sorted, then the distinct ones
  int* sl = ss + K4;     // [K4] slot of each sorted place
  __shared__ int warp_sum[kListThreads / 32];
  constexpr int NONE = 0x7fffffff;
  pdl_wait();
  pdl_trigger();
  const long long row = blockIdx.x;
  const int t = threadIdx.x;
  int weighs = 0, beyond = 0;
  for (int k = t; k < K4; k += kListThreads) {
    const int c = k < K ? idx[row * K + k] : -1;
    is[k] = c >= 0 && c < V ? c : NONE;
    ss[k] = NONE;
    beyond |= c >= V;
    if (dloss && c >= 0) weighs |= tlogit[row * K + k] * invT != __int_as_float(0xff800000);
  }
  weighs = __syncthreads_or(weighs);
  constexpr int EACH = kMaxTargets / kListThreads;  // entries of a thread
  int pos[EACH];
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int k = t + e * kListThreads;
    pos[e] = -1;
    if (k < K && is[k] != NONE) {
      const int c = is[k];
      int r = 0;  // smaller ones, and equal ones before it
      for (int j = 0; j < K4; j += 4) {
        const int4 w = *reinterpret_cast<const int4*>(is + j);
        r += (w.x < c || (w.x == c && j < k)) + (w.y < c || (w.y == c && j + 1 < k)) +
             (w.z < c || (w.z == c && j + 2 < k)) + (w.w < c || (w.w == c && j + 3 < k));
      }
      pos[e] = r;
      ss[r] = c;
    }
  }
  beyond = __syncthreads_or(beyond);
  if (dloss && t == 0) up[row] = weighs && !beyond ? dloss[row] : 0.f;
  // slot of place p: the changes of column up to it, less one; a thread takes neighbouring places
  const int per = (K4 + kListThreads - 1) / kListThreads;
  int own[EACH], n = 0;
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int p = t * per + e;
    own[e] = 0;
    if (e < per && p < K4 && ss[p] != NONE) own[e] = p == 0 || ss[p] != ss[p - 1];
    n += own[e];
  }
  int scan = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, scan, o);
    if ((t & 31) >= o) scan += v;
  }
  if ((t & 31) == 31) warp_sum[t >> 5] = scan;
  __syncthreads();
  int total = 0, before = scan - n;
#pragma unroll
  for (int w = 0; w < kListThreads / 32; ++w) {
    if (w < (t >> 5)) before += warp_sum[w];
    total += warp_sum[w];
  }
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int p = t * per + e;
    if (e < per && p < K4) {
      before += own[e];
      sl[p] = before - 1;
      own[e] = own[e] ? ss[p] : NONE;  // the column, where it begins here
    } else {
      own[e] = NONE;
    }
  }
  __syncthreads();  // ss has been read
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    if (own[e] != NONE) {
      const int u = sl[t * per + e];
      ss[u] = own[e];
      ucol[row * K + u] = own[e];
    }
    const int k = t + e * kListThreads;
    if (k < K) slot[row * K + k] = pos[e] < 0 ? kNoSlot : (uint16_t)sl[pos[e]];
  }
  __syncthreads();
  uint16_t* gs = gstart + row * (groups + 1);
  for (int g = t; g <= groups; g += kListThreads) {  // the distinct columns below the group's first
    const long long c = (long long)g * width;
    int lo = 0, hi = total;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (ss[mid] < c) lo = mid + 1;
      else hi = mid;
    }
    gs[g] = (uint16_t)lo;
  }
}

struct RowArgs {
  int V, groups, K;
  long long pitch;        // columns of a row of e
  int height;             // groups: 0: of 128 columns; else of 32 in each tile of `height` columns
  const float2* part;     // [rows][groups], log2 units
  const float* tl;        // [rows][K] logits of the distinct targets (before 1/T)
  const int32_t* idx;     // [rows][K] the targets as given
  const int32_t* ucol;    // [rows][K] distinct, ascending
  const uint16_t* slot;   // [rows][K] place of idx in ucol
  const float* tlogit;    // [rows][K] the teacher's logits; NULL: cross entropy (K = 1)
  const float* dloss;     // [rows] upstream gradients (with e)
  const float* unit;      // dz is kept over *unit * T
  float T, zl;
  float* loss;
  float* lse;             // nullable
  void* e;                // exp(z - m) of the rows, turned into dz (nullable: loss only)
  __nv_bfloat16* piece[3];  // fp32 heads: dz in three bf16 pieces; bf16 ones: [1] its second (nullable)
  int slice;  // 16-byte vectors of e per CTA (of a row's grid.y)
};

constexpr int kRowThreads = 256;
constexpr float kLn2 = 0.69314718055994530942f, kLog2e = 1.44269504088896340736f;

// Two sums (maxima) over the CTA, with one pair of barriers.
template <bool MAX>
__device__ __forceinline__ void block_reduce2(float& a, float& b, float2* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, a, o), y = __shfl_xor_sync(0xffffffffu, b, o);
    a = MAX ? fmaxf(a, x) : a + x;
    b = MAX ? fmaxf(b, y) : b + y;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 w[kRowThreads / 32];
#pragma unroll
  for (int i = 0; i < kRowThreads / 32; ++i) w[i] = red[i];
  a = w[0].x;
  b = w[0].y;
#pragma unroll
  for (int i = 1; i < kRowThreads / 32; ++i) {
    a = MAX ? fmaxf(a, w[i].x) : a + w[i].x;
    b = MAX ? fmaxf(b, w[i].y) : b + w[i].y;
  }
}

// One CTA per row: joins the groups, writes loss and lse and turns e into dz.  Bound by HBM: a row of
// e read and written (4096 x 32000: 524 MB in 85 us, 6.2 TB/s; 8192 x 128256: 0.64 ms, 6.6 TB/s).
// Where there are few rows, several CTAs share one: each joins the groups again and turns its columns.
// (Five CTAs per SM: 48 registers; four, with 63, cost 1 % of a call of 2047 rows.)
template <bool F32>
__global__ void __launch_bounds__(kRowThreads, 5) head_row_kernel(const RowArgs p) {
  extern __shared__ __align__(16) float sm[];
  const int K8 = (p.K + 7) / 8 * 8;
  uint16_t* ks = reinterpret_cast<uint16_t*>(sm);  // [K8] slots of the entries (distillation)
  float* fac = sm + K8 / 2;   // [groups] factor of each group (with e)
  float* z2 = fac + (p.e ? p.groups : 0);  // [K] the distinct targets' logits in log2 units
  float* qs = z2 + p.K;       // [K] their weights q
  float* qk = qs + p.K;       // [K] the entries' weights
  __shared__ float2 red[kRowThreads / 32];
  pdl_trigger();
  pdl_wait();
  const long long row = blockIdx.x;
  const int t = threadIdx.x;
  const float ninf = __int_as_float(0xff800000);
  const float scale2 = kLog2e / p.T;
  const int32_t* idx = p.idx + row * p.K;
  const uint16_t* slot = p.slot + row * p.K;
  const int32_t* ucol = p.ucol + row * p.K;
  const float* u = p.tlogit ? p.tlogit + row * p.K : nullptr;
  const float invT = 1.f / p.T;
  const float2* part = p.part + row * p.groups;
  float m = ninf;
  for (int g = t; g < p.groups; g += kRowThreads) m = fmaxf(m, part[g].x);
  // the distinct targets: nu of them
  bool bad;  // an index beyond the vocabulary
  int nu;
  if (!u) {
    const int c = idx[0];
    bad = c >= p.V;
    nu = c >= 0 && c < p.V;
  } else {
    float nbad = 0.f, top = -1.f;  // (slots are below 1024: exact in fp32)
    for (int k = t; k < K8; k += kRowThreads) {
      const int c = k < p.K ? idx[k] : -1;
      ks[k] = k < p.K ? slot[k] : kNoSlot;
      if (c >= p.V) nbad = 1.f;
      if (c >= 0 && c < p.V) top = fmaxf(top, (float)ks[k]);
    }
    block_reduce2<true>(nbad, top, red);
    bad = nbad > 0.f;
    nu = (int)top + 1;
  }
  float zm = ninf;
  for (int v = t; v < nu; v += kRowThreads) {
    z2[v] = p.tl[row * p.K + v] * scale2;
    qs[v] = 1.f;
    zm = fmaxf(zm, z2[v]);
  }
  // log-sum-exp in log2 units: the groups leave the targets out
  block_reduce2<true>(zm, m, red);
  m = fmaxf(m, zm);
  const float off = m == ninf ? 0.f : m;
  // the largest target on its own (the first of equals), all others with the groups
  int umax = 0;
  float tm = ninf;  // the teacher's largest logit
  if (u) {
    float first = -2048.f;
    for (int v = t; v < nu; v += kRowThreads)
      if (z2[v] == zm) first = fmaxf(first, -(float)v);
    for (int k = t; k < p.K; k += kRowThreads)
      if (idx[k] >= 0) {  // (a NaN makes it +inf, and with that the sum below NaN)
        const float a = u[k] * invT;
        tm = a != a ? -ninf : fmaxf(tm, a);
      }
    block_reduce2<true>(first, tm, red);
    umax = (int)-first;
  }
  float others = 0.f, us = 0.f;
  for (int g = t; g < p.groups; g += kRowThreads) {
    const float2 w = part[g];
    others += w.y * exp2f(w.x - off);
  }
  for (int v = t; v < nu; v += kRowThreads)
    if (v != umax) others += exp2f(z2[v] - off);
  if (u && tm != ninf)
    for (int k = t; k < p.K; k += kRowThreads)
      if (idx[k] >= 0) us += expf(u[k] * invT - tm);
  block_reduce2<false>(others, us, red);
  // (a label's logit itself, not the maximum, which drops a NaN; among a teacher's entries a NaN is none
  // that equals the maximum, and is in `others`)
  const float emax = nu ? exp2f((u ? zm : z2[0]) - off) : 0.f;
  const float total = others + emax;
  const float lse2 = off + log2f(total);
  const float lse = lse2 * kLn2;
  const bool sure = emax > others;  // the largest target has more than half
  const float lnp_max = sure ? -log1pf(others / emax) : (zm - lse2) * kLn2;
  float some, loss, weight;  // weight: of p in dz, before the upstream gradient
  float rest = 0.f;          // 1 - q of the largest target
  if (!u) {
    some = nu ? 1.f : 0.f;
    loss = p.zl * lse * lse - lnp_max;
    weight = 1.f + 2.f * p.zl * lse;
  } else {
    some = tm == ninf ? 0.f : 1.f;
    const float lus = logf(us);
    float l = 0.f;
    for (int k = t; k < p.K; k += kRowThreads) {
      float q = 0.f;
      if (ks[k] != kNoSlot && some > 0.f) {
        const float lq = u[k] * invT - tm - lus;
        q = expf(lq);
        if (!(q == 0.f)) l += q * (lq - (ks[k] == umax ? lnp_max : (z2[ks[k]] - lse2) * kLn2));
        if (ks[k] != umax) rest += q;
      }
      qk[k] = q;
    }
    block_reduce2<false>(l, rest, red);
    loss = l * p.T * p.T;
    weight = 1.f;
    // weights per distinct column, the entries added in their order
    for (int v = t; v < nu && p.e; v += kRowThreads) {
      float q = 0.f;
      for (int k = 0; k < K8; k += 8) {
        const uint4 w = *reinterpret_cast<const uint4*>(ks + k);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if ((x[j] & 0xffffu) == (uint32_t)v) q += qk[k + 2 * j];
          if ((x[j] >> 16) == (uint32_t)v) q += qk[k + 2 * j + 1];
        }
      }
      qs[v] = q;
    }
  }
  if (t == 0 && blockIdx.y == 0) {
    p.loss[row] = bad ? __int_as_float(0x7fc00000) : (some > 0.f ? loss : 0.f);
    if (p.lse) p.lse[row] = lse;
  }
  if (!p.e) return;
  const bool live = some > 0.f && !bad;
  const float gT = live ? p.dloss[row] / *p.unit : 0.f;
  const float coef = gT * weight;
  const float gcoef = F32 ? coef : coef * kExpLoad;
  for (int g = t; g < p.groups; g += kRowThreads) fac[g] = gcoef * exp2f(part[g].x - lse2);
  __syncthreads();
  // the CTA's vectors [lo, n) of the row
  constexpr int VEC = F32 ? 4 : 8;
  const int lo = (int)blockIdx.y * p.slice, n = min(lo + p.slice, (int)(p.pitch / VEC));
  if (!F32) {
    uint4* er = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.e) + row * p.pitch);
    uint4* second = p.piece[1] ? reinterpret_cast<uint4*>(p.piece[1] + row * p.pitch) : nullptr;
    constexpr int U = 4;  // loads in flight per thread
    for (int i0 = lo + t; i0 < n; i0 += U * kRowThreads) {
      uint4 w[U];
      if (live)
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (i0 + k * kRowThreads < n) w[k] = er[i0 + k * kRowThreads];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k * kRowThreads;
        if (i >= n) break;
        uint4 o = make_uint4(0u, 0u, 0u, 0u), o2 = o;
        if (live) {
          int g = i / (kGroup / 8);
          if (p.height) {  // (columns past the last tile hold zeros)
            const uint32_t tile = 8u * i / p.height;
            g = min((int)(4 * tile + (8u * i - tile * p.height) / 32), p.groups - 1);
          }
          const float f = fac[g];
          const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 h = unpack_exp(u[j]);
            v[2 * j] = h.x * f;
            v[2 * j + 1] = h.y * f;
          }
          o = pack8(v);
          if (second) {
            const uint32_t r[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[2 * j] -= __uint_as_float(r[j] << 16);
              v[2 * j + 1] -= __uint_as_float(r[j] & 0xffff0000u);
            }
            o2 = pack8(v);
          }
        }
        if (second) second[i] = o2;
        er[i] = o;
      }
    }
  } else {
    const float4* er = reinterpret_cast<const float4*>(static_cast<float*>(p.e) + row * p.pitch);
    constexpr int U = 4;
    for (int i0 = lo + t; i0 < n; i0 += U * kRowThreads) {
      float4 w[U];
#pragma unroll
      for (int k = 0; k < U; ++k)
        w[k] = live && i0 + k * kRowThreads < n ? er[i0 + k * kRowThreads]
                                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k * kRowThreads;
        if (i >= n) break;
        const float f = live ? fac[i / (kGroup / 4)] : 0.f;
        __nv_bfloat16* d[3];
#pragma unroll
        for (int j = 0; j < 3; ++j) d[j] = p.piece[j] + row * p.pitch + 4 * i;
        store3(make_float4(w[k].x * f, w[k].y * f, w[k].z * f, w[k].w * f), d);
      }
    }
  }
  if (!live) return;
  __syncthreads();
  // the targets' own columns: weight p - q, without cancellation where p is near 1
  for (int u = t; u < nu; u += kRowThreads) {
    const int c = ucol[u];
    if (c / VEC < lo || c / VEC >= n) continue;
    const float pv = exp2f(z2[u] - lse2);
    float dz;
    if (u == umax && sure)
      dz = gT * ((weight - 1.f) * pv + (rest - others / total));
    else
      dz = coef * pv - gT * qs[u];
    if (!F32) {
      const __nv_bfloat16 hi = __float2bfloat16_rn(dz);
      static_cast<__nv_bfloat16*>(p.e)[row * p.pitch + c] = hi;
      if (p.piece[1])
        p.piece[1][row * p.pitch + c] = __float2bfloat16_rn(dz - __bfloat162float(hi));
    } else {
      __nv_bfloat16 o[3];
      split3(dz, o);
#pragma unroll
      for (int j = 0; j < 3; ++j) p.piece[j][row * p.pitch + c] = o[j];
    }
  }
}

// The three bf16 pieces of two fp32 arrays.  Bound by HBM: 4 bytes in, 6 out (8000 x 1024 and 512 x 1024:
// 87 MB in 16 us).
__global__ void __launch_bounds__(256) head_split_kernel(const SplitArray a, const SplitArray b) {
  pdl_trigger();
  pdl_wait();
  split_arrays(a, b, (long long)blockIdx.x * blockDim.x + threadIdx.x, (long long)gridDim.x * blockDim.x);
}

// out = sum over S fp32 partials of `stride` elements each, in order (count a multiple of 4).  PAIRS: every
// second one is of dz's second piece and the one before it of its first (with_rest).  The
// partials were written just before and are read from L2 (1021 x 1600: 10 us).  Few rows have many partials
// each: sixteen are in flight per thread (16 rows of 4096 x 14336, the whole backward: 134 -> 120 us).
template <typename T, bool PAIRS>
__global__ void __launch_bounds__(256)
    head_sum_kernel(const float* __restrict__ part, int S, long long stride, long long quads,
                    T* __restrict__ out) {
  pdl_trigger();
  pdl_wait();
  const long long step = (long long)gridDim.x * blockDim.x;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < quads; i += step) {
    float4 a = *reinterpret_cast<const float4*>(part + 4 * i);
    auto add = [&](auto n) {  // n partials in flight, added in order
      constexpr int U = decltype(n)::value;
      for (int k0 = 1; k0 < S; k0 += U) {
        float4 b[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (k0 + k < S) b[k] = *reinterpret_cast<const float4*>(part + (k0 + k) * stride + 4 * i);
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (k0 + k < S) {
            a.x += b[k].x;
            a.y += b[k].y;
            a.z += b[k].z;
            a.w += b[k].w;
          }
      }
    };
    if (S <= 5) add(std::integral_constant<int, 4>{});
    else add(std::integral_constant<int, 16>{});
    if (PAIRS && isnan((a.x + a.y) + (a.z + a.w))) {  // (also where infinities of both signs are beside each other)
      float v[4] = {};
#pragma unroll 1
      for (int k = 0; k < S; k += 2)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[j] += with_rest(part[k * stride + 4 * i + j], part[(k + 1) * stride + 4 * i + j]);
      a = make_float4(v[0], v[1], v[2], v[3]);
    }
    if (sizeof(T) == 2) {
      *reinterpret_cast<uint2*>(out + 4 * i) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    } else {
      *reinterpret_cast<float4*>(out + 4 * i) = a;
    }
  }
}

// ---------------------------------------------------------------- host side
template <int NT>
poetx_status score(const CUtensorMap& mW, const CUtensorMap& mx, HeadScore p, cudaStream_t s) {
  auto k = head_score_kernel<NT>;
  static PerDevice<cudaError_t> attr;
  POETX_CUDA_TRY(allow_smem(attr, k, kScoreSmem));
  // (16 KB kept behind the last stage: the MMAs read 128 rows from its last K block's first)
  p.stages = (kScoreSmem - 1024 - 512 - score_turn_bytes(NT) - (int)kABytes) /
             score_stage_bytes(NT, p.height, p.kps);
  if (p.stages > kScoreRing) p.stages = kScoreRing;
  p.err = device_error_word();
  p.limit_ns = kWaitLimitNs;
  const int grid = p.tiles < sm_count() ? p.tiles : sm_count();
  POETX_CUDA_TRY(launch_pdl(k, dim3(grid), dim3(kScoreThreads), kScoreSmem, s, mW, mx, p));
  POETX_CUDA_TRY(cudaGetLastError());
  after_launch(s, ST_HEAD_GEMM);
  return POETX_OK;
}

template <bool LSE, int SEGS>
poetx_status gemm(const HeadMaps& m0, const HeadMaps& m1, HeadGemm& p, cudaStream_t s) {
  // (one CTA per SM)
  static PerDevice<Clusters> setup;
  const Clusters c = allow_clusters(setup, head_gemm_kernel<LSE, SEGS>, sm_count() / 2 * 2, kGemmThreads,
                                    gemm_smem(SEGS), 2);
  POETX_CUDA_TRY(c.err);
  long long tiles = 0;
  for (const Product& d : p.prod) {
    if ((long long)d.tiles_m * d.tiles_n > 0x3fffffffLL) return POETX_ERR_SHAPE;
    tiles += d.num_tiles;
  }
  if (tiles > 0x7fffffffLL) return POETX_ERR_SHAPE;
  p.num_tiles = (int)tiles;
  p.err = device_error_word();
  p.limit_ns = kWaitLimitNs;
  const int pairs = (int)(tiles < c.resident ? tiles : c.resident);
  POETX_CUDA_TRY(launch_pdl_cluster(head_gemm_kernel<LSE, SEGS>, dim3(2 * pairs),
                                    dim3(kGemmThreads),
                                    gemm_smem(SEGS), s, 2, m0, m1, p));
  POETX_CUDA_TRY(cudaGetLastError());
  after_launch(s, ST_HEAD_GEMM);
  return POETX_OK;
}

// The K splits of dx, which runs alone or in one launch with dW on pairs that take every P-th tile:
// the split with the shortest longest pair, with the partials' traffic (at about 5 TB/s) against it.
// A 64-wide K block of a 256 x 256 tile takes about 0.3 us of a pair, a tile 0.6 us besides.  One
// split for both uses (the sum of the two times decides), so that dx has the same bits in both.
int dx_splits(long long rows, int D, int V, int nseg) {
  const long long t1 = (long long)ceil_div(rows, 2 * BM) * ceil_div(D, BN);
  const long long t2 = (long long)ceil_div(V, 2 * BM) * ceil_div(D, BN);
  const int kb1 = ceil_div(V, BK), kb2 = ceil_div(rows, BK), pairs = sm_count() / 2;
  int best = 1;
  double best_us = 1e30;
  for (int S = 1; S <= 64 && S <= kb1; ++S) {
    const long long n1 = t1 * S, all = n1 + t2;
    const double us1 = 0.6 + 0.3 * nseg * ceil_div(kb1, S), us2 = 0.6 + 0.3 * nseg * kb2;
    double alone = 0, both = 0;
    // pair i has n1 / P (+ 1 where i < n1 % P) tiles of dx, likewise of all: three kinds of pairs
    for (const long long i : {0LL, n1 % pairs, all % pairs}) {
      const long long a = n1 / pairs + (i < n1 % pairs), c = all / pairs + (i < all % pairs);
      if (a * us1 > alone) alone = a * us1;
      if (a * us1 + (c - a) * us2 > both) both = a * us1 + (c - a) * us2;
    }
    double us = alone + both;
    if (S > 1) us += 2 * (3.0 + 8e-6 * (double)S * (double)rows * D / 5.0);
    if (us < best_us) {
      best_us = us;
      best = S;
    }
  }
  // every split non-empty
  return ceil_div(kb1, ceil_div(kb1, best));
}

// Bound of a piece's stored exponentials, where there is more than one piece: each piece but the
// first reads and writes dW's fp32 sums (8 V D bytes against 6 rows V D flops: at 2 GB per piece of a
// 128-thousand vocabulary about a tenth of the piece's time).
constexpr size_t kPieceBytes = (size_t)9 << 28;  // 2.25 GiB
// Rows up to which dz is kept in two bf16 pieces: over few rows the gradients hang on a few large
// p - q, whose rounding is not averaged (over many rows one piece stays below 1.45 times).  Error of dx
// and dW against their own output's rounding, 1 to 128 rows: 1.15-1.54 times it with one piece, 1.0
// with two.  The second piece costs little: dx's tile has the room for it, and of a dW of so
// few rows its stores are the most (whole call, one piece and two: 98 and 101 us at 33 x 32000 x 2048,
// 117 and 129 us at 128, 550 and 560 us at 33 x 128256 x 4096, 629 and 683 us at 128).
constexpr int kFineRows = kScoreRows;
constexpr int kMaxFactors = 32768;  // groups of a row with gradients (4194304 columns of 128)
constexpr long long kMaxRows = 1 << 16;  // of a piece (one warp looks through its upstream gradients)

struct Plan {
  bool f32, grads;
  bool fine;         // bf16, few rows: dz in two pieces
  long long Vp;      // columns of a stored row
  int groups;
  long long rows;    // rows of a piece
  int pieces;
  int splits;        // K splits of dx
  int sums;          // partial sums of dx (the splits, times dz's pieces)
  int height, tiles;  // few rows: vocabulary rows of a tile and tiles (else 0)
  // workspace offsets
  size_t unit, part, tl, ucol, slot, gstart, up, e, dz, dz2, xs, ws, acc, dxp, bytes;
};

bool plan(poetx_dtype dt, int N, int D, int V, int K, bool dx, bool dW, Plan* o) {
  if (N < 0 || D < 8 || D % 8 || D > (1 << 17) || V < 1 || V > (1 << 22) || K < 1 || K > kMaxTargets)
    return false;
  o->f32 = dt == POETX_F32;
  o->grads = dx || dW;
  o->fine = !o->f32 && o->grads && N <= kFineRows;
  o->Vp = (long long)align_up((size_t)V, 64);
  o->groups = ceil_div(V, kGroup);
  o->height = o->tiles = 0;
  if (!o->f32 && N <= kScoreRows) {
    // every SM the same number of tiles, of at most 128 rows; no lower than 16
    const int sms = sm_count(), each = ceil_div(V, (long long)sms * BM);
    int height = ceil_div(V, (long long)sms * each);
    height = (int)align_up(height < 16 ? 16 : (size_t)height, 8);
    const int tiles = ceil_div(V, height);
    // (with gradients the row kernel keeps a factor per group in shared memory: V up to a million)
    if (!o->grads || 4 * tiles <= kMaxFactors) {
      o->height = height;
      o->tiles = tiles;
      o->groups = 4 * tiles;
    }
  }
  const size_t row_bytes = (o->grads ? (size_t)o->Vp * (o->f32 ? 10 : 2) : 0) +
                           (size_t)o->groups * 8 * (o->grads ? 1 : 4);
  const long long n = N > 0 ? N : 1;
  // one piece where that takes no more memory than a piece and dW's fp32 sums would
  const size_t whole = kPieceBytes + (!o->f32 && dW ? (size_t)V * D * 4 : 0);
  long long rows = n;
  if ((unsigned long long)n > whole / row_bytes) {
    rows = (long long)(kPieceBytes / row_bytes) / 256 * 256;
    if (rows < 256) rows = 256;
  }
  if (rows > kMaxRows) rows = kMaxRows;
  o->pieces = ceil_div(n, rows);
  o->rows = o->pieces == 1 ? n : (long long)align_up((size_t)ceil_div(n, o->pieces), 256);
  o->pieces = ceil_div(n, o->rows);
  o->splits = dx ? dx_splits(o->rows, D, V, o->f32 ? kMaxSegs : 1) : 1;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += align_up(bytes, 1024);
    return a;
  };
  const size_t R = (size_t)o->rows;
  o->unit = take(4);
  o->part = take(R * o->groups * sizeof(float2));
  o->tl = take(R * K * 4);
  // the sorted target lists of a distillation (a call with K = 1 may be either: both fit)
  o->ucol = take(R * K * 4);
  o->slot = take(R * K * 2);
  o->gstart = take(R * ((o->tiles ? o->tiles : o->groups) + 1) * 2);
  o->up = o->grads ? take(R * 4) : 0;
  o->e = o->grads ? take(R * o->Vp * (o->f32 ? 4 : 2)) : 0;
  o->dz = o->f32 && o->grads ? take(3 * align_up(R * o->Vp * 2, 1024)) : o->e;
  o->dz2 = o->fine ? take(R * o->Vp * 2) : 0;
  o->xs = o->f32 ? take(3 * align_up(R * D * 2, 1024)) : 0;
  o->ws = o->f32 ? take(3 * align_up((size_t)V * D * 2, 1024)) : 0;
  o->acc = !o->f32 && dW && o->pieces > 1 ? take((size_t)V * D * 4) : 0;
  o->sums = o->fine && dx ? 2 * o->splits : o->splits;
  o->dxp = o->sums > 1 ? take((size_t)o->splits * align_up(R, 256) * D * 4) : 0;
  o->bytes = at;
  return true;
}

bool bf16_map(CUtensorMap* m, const void* p, long long inner, long long outer, int bi, int bo) {
  return encode_tma_2d(m, p, TMA_BF16, inner, outer, inner, bi, bo, true);
}

// An MN-major operand [K][MN]: 64 rows of K and 128 of MN per load, as one box of two 64-column groups
// where MN is a multiple of 64, else as two boxes.
bool mn_map(CUtensorMap* m, const void* p, long long inner, long long outer) {
  return inner % 64 == 0 ? encode_tma_groups(m, p, inner, outer, 64, 2)
                         : bf16_map(m, p, inner, outer, 64, 64);
}

// Operand pieces and the K of one accumulator.  fp32: small pieces first, so that the accumulator is
// small while they are added (a chunk runs pair by pair of pieces: the adds at full size are those of
// the last pair); 256 of K (16 adds of 16 products at full size; 64: a fifth slower).  bf16: 1024 for
// the logits (64 adds: losses to 7e-7 at K = 2048), or 256 for few rows, whose products are not what
// their time goes into (one row's loss: 1.3e-6 with 1024, 2e-7 with 256); 4096 for the gradients, which
// are rounded to bf16 (256 adds: 1.5e-5).
void set_segs(HeadGemm* g, bool f32, bool lse, int rows) {
  static const int8_t a[kMaxSegs] = {1, 0, 2, 1, 0, 0}, b[kMaxSegs] = {1, 2, 0, 0, 1, 0};
  for (int i = 0; i < kMaxSegs; ++i) {
    g->seg_a[i] = a[i];
    g->seg_b[i] = b[i];
  }
  g->chunk = f32 ? 4 : (lse ? (rows <= 512 ? 4 : 16) : 64);
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

}  // namespace

// The products behind dz (see kernels.h); between the pieces of a bf16 head dW's sum stays in fp32.
poetx_status grad_products(const GradProducts& c, cudaStream_t s) {
  const int np = c.f32 ? 3 : 1, rows = c.rows;
  const int sums = c.fine ? 2 * c.splits : c.splits;  // partial sums of dx
  HeadMaps mp, mw;
  HeadGemm h{};
  const int nz = c.f32 ? 3 : (c.fine ? 2 : 1);  // dz's pieces
  set_segs(&h, c.f32, false, rows);
  h.out_scale = c.unit;
  h.T = c.T;
  if (c.fine) {
    h.z = reinterpret_cast<const __nv_bfloat16*>(c.z[0]);
    h.x = reinterpret_cast<const __nv_bfloat16*>(c.x);
    h.z_pitch = c.pitch;
    h.rows = rows;
  }
  int used = 0;
  const int c_rows = (int)align_up((size_t)rows, 256);
  if (c.dx) {
    Product& d = h.prod[used++];
    for (int i = 0; i < nz; ++i)
      if (!encode_tma_2d(&mp.a[i], c.z[i], TMA_BF16, c.z_cols, rows, c.pitch, 64, 128, true))
        return POETX_ERR_CUDA;
    for (int i = 0; i < np; ++i)
      if (!mn_map(&mp.b[i], c.w + i * c.w_step, c.D, c.V)) return POETX_ERR_CUDA;
    d.b_groups = c.D % 64 == 0;
    d.tiles_m = ceil_div(rows, 2 * BM);
    d.tiles_n = ceil_div(c.D, BN);
    d.num_tiles = d.tiles_m * d.tiles_n * c.splits;
    d.num_kb = ceil_div(c.V, BK);
    d.kb_split = ceil_div(d.num_kb, c.splits);
    d.M = rows;
    d.N = d.n_store = c.D;
    d.c_rows = c_rows;
    d.c_f32 = c.f32 || sums > 1;
    const void* dst = sums > 1 ? static_cast<const void*>(c.dxp) : c.dx;
    const long long drows = sums > 1 ? (long long)c.splits * c_rows : rows;
    if (!encode_tma_2d(&mp.c, dst, d.c_f32 ? TMA_F32 : TMA_BF16, c.D, drows, c.D, d.c_f32 ? 32 : 64, 32,
                       true))
      return POETX_ERR_CUDA;
  }
  if (c.dW) {
    Product& d = h.prod[used];
    HeadMaps& m = used++ ? mw : mp;
    for (int i = 0; i < nz; ++i)
      if (!mn_map(&m.a[i], c.z[i], c.pitch, rows)) return POETX_ERR_CUDA;
    for (int i = 0; i < np; ++i)
      if (!mn_map(&m.b[i], c.x + i * c.x_step, c.D, rows)) return POETX_ERR_CUDA;
    d.b_groups = c.D % 64 == 0;
    d.tiles_m = ceil_div(c.V, 2 * BM);
    d.tiles_n = ceil_div(c.D, BN);
    d.num_tiles = d.tiles_m * d.tiles_n;
    d.n_fast = !c.fine;  // (few rows: down the vocabulary 1-3 % faster)
    d.num_kb = d.kb_split = ceil_div(rows, BK) * (c.fine ? 2 : 1);
    d.a_mn = 1;
    d.M = d.c_rows = c.V;
    d.N = d.n_store = c.D;
    d.c_f32 = c.f32 || !c.last;
    void* dst = c.f32 || c.last ? c.dW : static_cast<void*>(c.acc);
    if (c.f32)
      d.add_f32 = !c.first || c.accumulate ? static_cast<const float*>(c.dW) : nullptr;
    else
      d.add_f32 = !c.first ? c.acc : nullptr;
    if (!c.f32 && c.last && c.accumulate) d.add_bf16 = static_cast<const __nv_bfloat16*>(c.dW);
    if (!encode_tma_2d(&m.c, dst, d.c_f32 ? TMA_F32 : TMA_BF16, c.D, c.V, c.D, d.c_f32 ? 32 : 64, 32,
                       true))
      return POETX_ERR_CUDA;
  }
  const HeadMaps& second = used > 1 ? mw : mp;
  if (c.f32)
    POETX_TRY((gemm<false, kMaxSegs>(mp, second, h, s)));
  else if (c.fine)
    POETX_TRY((gemm<false, 2>(mp, second, h, s)));
  else
    POETX_TRY((gemm<false, 1>(mp, second, h, s)));
  if (c.dx && sums > 1)
    POETX_TRY(sum_partials(c.f32, c.dxp, sums, (long long)(c.fine ? BM : c_rows) * c.D,
                           (long long)rows * c.D, c.dx, s, c.fine));
  return POETX_OK;
}

poetx_status sum_partials(bool f32, const float* part, int S, long long stride, long long count, void* out,
                          cudaStream_t s, bool pairs) {
  const dim3 grid(grid_for(count / 4, 256)), block(256);
  __nv_bfloat16* const out16 = static_cast<__nv_bfloat16*>(out);
  if (f32)
    POETX_CUDA_TRY(launch_pdl(head_sum_kernel<float, false>, grid, block, 0, s, part, S, stride, count / 4,
                              static_cast<float*>(out)));
  else if (pairs)
    POETX_CUDA_TRY(launch_pdl(head_sum_kernel<__nv_bfloat16, true>, grid, block, 0, s, part, S, stride,
                              count / 4, out16));
  else
    POETX_CUDA_TRY(launch_pdl(head_sum_kernel<__nv_bfloat16, false>, grid, block, 0, s, part, S, stride,
                              count / 4, out16));
  POETX_CUDA_TRY(cudaGetLastError());
  after_launch(s, ST_HEAD_ROW);
  return POETX_OK;
}

int grad_splits(long long rows, int D, int V, bool f32) {
  return dx_splits(rows, D, V, f32 ? kMaxSegs : 1);
}

poetx_status split_pieces(const float* a, long long na, uint8_t* da, size_t a_step, const float* b,
                          long long nb, uint8_t* db, size_t b_step, cudaStream_t s) {
  const SplitArray xa = split_of(a, na, da, a_step), wa = split_of(b, nb, db, b_step);
  POETX_CUDA_TRY(launch_pdl(head_split_kernel, dim3(grid_for((xa.quads + wa.quads) / 4 + 1, 256)),
                            dim3(256), 0, s, xa, wa));
  POETX_CUDA_TRY(cudaGetLastError());
  after_launch(s, ST_HEAD_ROW);
  return POETX_OK;
}

namespace {

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
  const size_t row_smem = align_up((size_t)c.K, 8) * 2 + (pl.grads ? (size_t)pl.groups * 4 : 0) +
                          (size_t)c.K * 12;
  static PerDevice<cudaError_t> attr[2];
  POETX_CUDA_TRY(pl.f32 ? allow_smem(attr[1], head_row_kernel<true>, 160 * 1024)
                        : allow_smem(attr[0], head_row_kernel<false>, 160 * 1024));

  uint8_t* w = static_cast<uint8_t*>(c.ws);
  const size_t x_step = align_up((size_t)pl.rows * c.D * 2, 1024);
  const size_t w_step = align_up((size_t)c.V * c.D * 2, 1024);
  const size_t z_step = align_up((size_t)pl.rows * pl.Vp * 2, 1024);
  const int np = pl.f32 ? 3 : 1;
  float2* part = reinterpret_cast<float2*>(w + pl.part);
  float* tl = reinterpret_cast<float*>(w + pl.tl);
  float* unit = reinterpret_cast<float*>(w + pl.unit);
  const uint8_t* wp = pl.f32 ? w + pl.ws : static_cast<const uint8_t*>(c.W);

  for (int pc = 0; pc < pl.pieces; ++pc) {
    const long long r0 = pc * pl.rows;
    const int rows = (int)((long long)c.N - r0 < pl.rows ? (long long)c.N - r0 : pl.rows);
    const uint8_t* xr = static_cast<const uint8_t*>(c.x) + (size_t)r0 * c.D * esz;
    const uint8_t* xp = pl.f32 ? w + pl.xs : xr;
    if (pl.f32) {  // the pieces of these rows, and with the first ones of W
      POETX_TRY(split_pieces(reinterpret_cast<const float*>(xr), (long long)rows * c.D, w + pl.xs, x_step,
                             static_cast<const float*>(c.W), pc ? 0 : (long long)c.V * c.D, w + pl.ws,
                             w_step, s));
    }
    // a teacher's entries: distinct columns in order
    const int32_t* idx = c.idx + r0 * c.K;
    const int32_t* ucol = idx;
    uint16_t* slot = reinterpret_cast<uint16_t*>(w + pl.slot);
    uint16_t* gstart = nullptr;
    const float* unit_of = c.dloss ? c.dloss + r0 : nullptr;
    if (c.tlogit) {
      float* up = reinterpret_cast<float*>(w + pl.up);
      int32_t* u = reinterpret_cast<int32_t*>(w + pl.ucol);
      gstart = reinterpret_cast<uint16_t*>(w + pl.gstart);
      POETX_CUDA_TRY(launch_pdl(head_targets_kernel, dim3(rows), dim3(kListThreads),
                                align_up((size_t)c.K, 4) * 12, s, idx,
                                c.K, c.V, pl.tiles ? pl.tiles : pl.groups,
                                pl.tiles ? pl.height : kGroup, slot, u, gstart, c.tlogit + r0 * c.K,
                                1.f / c.T, pl.grads ? unit_of : (const float*)nullptr, up));
      POETX_CUDA_TRY(cudaGetLastError());
      after_launch(s, ST_HEAD_ROW);
      ucol = u;
      unit_of = up;
    }
    // the logits' product
    HeadMaps mp;
    if (pl.tiles) {
      const int nt = rows <= 16 ? 16 : (rows <= 32 ? 32 : (rows <= 64 ? 64 : 128));
      HeadScore h{};
      h.tiles = pl.tiles;
      h.height = pl.height;
      h.V = c.V;
      h.rows = rows;
      // One box per stage and operand over several K blocks where D is a multiple of 64 (one thread
      // issues all copies, and 14 KB boxes come in at some 50 GB/s per SM, four together at 70)
      h.kps = c.D % 64 ? 1 : (nt <= 32 ? 4 : 2);
      h.num_st = ceil_div(ceil_div(c.D, BK), h.kps);
      h.chunk = 4 / h.kps;  // 256 of K per accumulator
      h.scale2 = kLog2e / c.T;
      h.part = part;
      h.ucol = ucol;
      h.gstart = gstart;
      h.K = c.K;
      h.tl = tl;
      h.e = pl.grads ? reinterpret_cast<uint16_t*>(w + pl.e) : nullptr;
      h.pitch = pl.Vp;
      h.dloss = unit_of;
      h.unit = unit;
      const bool maps = h.kps > 1 ? encode_tma_groups(&mp.a[0], wp, c.D, c.V, pl.height, h.kps) &&
                                        encode_tma_groups(&mp.b[0], xp, c.D, rows, nt, h.kps)
                                  : bf16_map(&mp.a[0], wp, c.D, c.V, 64, pl.height) &&
                                        bf16_map(&mp.b[0], xp, c.D, rows, 64, nt);
      if (!maps) return POETX_ERR_CUDA;
      switch (nt) {
        case 16: POETX_TRY(score<16>(mp.a[0], mp.b[0], h, s)); break;
        case 32: POETX_TRY(score<32>(mp.a[0], mp.b[0], h, s)); break;
        case 64: POETX_TRY(score<64>(mp.a[0], mp.b[0], h, s)); break;
        default: POETX_TRY(score<128>(mp.a[0], mp.b[0], h, s)); break;
      }
    } else {
      HeadGemm g{};
      set_segs(&g, pl.f32, true, rows);
      for (int i = 0; i < np; ++i)
        if (!bf16_map(&mp.a[i], xp + i * x_step, c.D, rows, 64, 128) ||
            !bf16_map(&mp.b[i], wp + i * w_step, c.D, c.V, 64, 128))
          return POETX_ERR_CUDA;
      Product& lg = g.prod[0];
      lg.tiles_m = ceil_div(rows, 2 * BM);
      lg.tiles_n = ceil_div(c.V, BN);
      lg.num_tiles = lg.tiles_m * lg.tiles_n;
      lg.num_kb = lg.kb_split = ceil_div(c.D, BK);
      lg.M = rows;
      lg.N = c.V;
      lg.n_store = (int)pl.Vp;  // columns V .. Vp - 1 are stored as zeros
      g.scale2 = kLog2e / c.T;
      g.part = part;
      g.groups = pl.groups;
      g.ucol = ucol;
      g.gstart = gstart;
      g.K = c.K;
      g.tl = tl;
      g.store = pl.grads;
      g.dloss = unit_of;
      g.unit = unit;
      if (pl.grads && !encode_tma_2d(&mp.c, w + pl.e, pl.f32 ? TMA_F32 : TMA_BF16, pl.Vp, rows, pl.Vp,
                                     pl.f32 ? 32 : 64, 32, true))
        return POETX_ERR_CUDA;
      if (!pl.grads) mp.c = mp.a[0];
      if (pl.f32)
        POETX_TRY((gemm<true, kMaxSegs>(mp, mp, g, s)));
      else
        POETX_TRY((gemm<true, 1>(mp, mp, g, s)));
    }
    // rows: lse, loss, dz
    RowArgs ra{};
    ra.V = c.V;
    ra.groups = pl.groups;
    ra.K = c.K;
    ra.pitch = pl.Vp;
    ra.height = pl.height;
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
    ra.unit = unit;
    ra.e = pl.grads ? w + pl.e : nullptr;
    if (pl.f32)
      for (int i = 0; i < 3; ++i)
        ra.piece[i] = reinterpret_cast<__nv_bfloat16*>(w + pl.dz + i * z_step);
    else if (pl.fine)
      ra.piece[1] = reinterpret_cast<__nv_bfloat16*>(w + pl.dz2);
    // a row's CTAs: up to four per SM in all, with at least 1024 vectors of columns (16 bytes) each
    // (64 x 60416: 19 -> 13 us)
    const int vecs = (int)(pl.Vp * (pl.f32 ? 4 : 2) / 16), room = 4 * sm_count() / rows;
    int ctas = ceil_div(vecs, 1024);
    if (ctas > room) ctas = room;
    if (ctas < 1 || !pl.grads) ctas = 1;
    ra.slice = ceil_div(vecs, ctas);
    const dim3 row_grid(rows, ctas);
    if (pl.f32)
      POETX_CUDA_TRY(launch_pdl(head_row_kernel<true>, row_grid, dim3(kRowThreads), row_smem, s, ra));
    else
      POETX_CUDA_TRY(launch_pdl(head_row_kernel<false>, row_grid, dim3(kRowThreads), row_smem, s, ra));
    POETX_CUDA_TRY(cudaGetLastError());
    after_launch(s, ST_HEAD_ROW);
    if (!pl.grads) continue;
    // dx = dz W and dW (+)= dz^T x
    GradProducts gp{};
    gp.f32 = pl.f32;
    gp.fine = pl.fine;
    gp.rows = rows;
    gp.D = c.D;
    gp.V = c.V;
    gp.pitch = gp.z_cols = pl.Vp;
    for (int i = 0; i < 3; ++i) gp.z[i] = pl.fine && i ? w + pl.dz2 : w + pl.dz + i * z_step;
    gp.x = xp;
    gp.x_step = x_step;
    gp.w = wp;
    gp.w_step = w_step;
    gp.unit = unit;
    gp.T = c.T;
    gp.dx = c.dx ? static_cast<uint8_t*>(c.dx) + (size_t)r0 * c.D * esz : nullptr;
    gp.dW = c.dW;
    gp.accumulate = c.accumulate;
    gp.first = pc == 0;
    gp.last = pc + 1 == pl.pieces;
    gp.acc = reinterpret_cast<float*>(w + pl.acc);
    gp.splits = pl.splits;
    gp.dxp = reinterpret_cast<float*>(w + pl.dxp);
    POETX_TRY(grad_products(gp, s));
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
