// Dense product with a fused epilogue:
//   out[m, n] = act(s_a[m] s_w[n] sum_k a[m, k] w[n, k] + bias[n]) + residual[m, n]
// with a [M, K] and w [N, K] both bf16 (fp32 accumulators) or both signed
// 8-bit (exact int32 accumulators and the scales s_a, s_w). The method's
// sources name no dense product; it is the projection, the shared dense FFN
// and the product with the vocabulary beside the routed experts.
//
// tcgen05 tiles of 128 rows of one operand by BT rows of the other, K in
// 128-byte steps through a TMA ring (128-byte swizzle, K-major; columns past
// K and rows past M or N arrive as zeros, so no size needs padding), two
// accumulator slots in tensor memory so that a tile's epilogue overlaps the
// next tile's products. Which operand takes the 128 rows:
//   features - the 128 rows are rows of w, the BT rows are tokens (BT 16..128).
//     A warp's lanes then hold neighbouring features of one token, so results
//     leave in coalesced rows of any alignment, and few tokens waste little:
//     decode and verify batches, and outputs whose rows are not 16-byte aligned.
//   tokens   - the 128 rows are tokens, a thread holds 16 neighbouring features
//     of its token: large batches. Results leave through shared memory, 32 rows
//     of 128 bytes per warp and TMA store, and the residual comes the same way a
//     step ahead: written straight from the lanes, every 16 bytes of a warp's
//     store lie in another row, and the epilogue took twice the products' time.
//   pairs    - tokens, with two CTAs on one tile of 256 x 256: each loads 128
//     rows of either operand, half of what it would load alone, since the loads
//     from L2 bound the lone CTA (48 KB a step against 32 KB).
// Few tiles (small batches against narrow weights) leave SMs idle: clusters of
// S CTAs then split K, every CTA sends its accumulators to the CTA that owns
// the feature slice through distributed shared memory, and the owner adds them
// in CTA order - one launch, no workspace, the same bits on every run.
// The tensor cores' fp32 accumulation drops low bits at every step (2e-6 of the
// result at K = 2048), so for fp32 results of bf16 operands a slot holds four
// steps only, and the epilogue's threads add the slots' values with rounding.
#include <cuda_bf16.h>

#include "dense.cuh"
#include "tc05.cuh"

namespace qmoe {
namespace {

constexpr int LN_ROWS = 128;                     // rows of the A operand per CTA (MMA M)
constexpr int LN_KB = 128;                       // bytes of K per pipeline step
constexpr int LN_A_BYTES = LN_ROWS * LN_KB;      // 16 KB
constexpr int LN_W_TMA = 0, LN_W_MMA = 1, LN_W_EPI = 2;
constexpr int LN_MAX_STAGES = 10;
constexpr int LN_MAX_SPLIT = 8;
constexpr int LN_MAX_K = 65536;                  // keeps |int32 sums| below 2^31
constexpr int LN_MAX_MN = 1 << 30;               // tile ends stay below 2^31
constexpr long long LN_MAX_LD = 1LL << 37;       // elements: below the tensor maps' 2^40 bytes
constexpr int LN_SMEM = 224 * 1024;              // ring and staging
constexpr int LN_BOX = 4096;                     // staging: 32 rows of 128 bytes
constexpr int LN_GROUP = 8;                      // A tiles that share B tiles in L2
constexpr int LN_SEG = 4;                        // steps per accumulator slot of fp32 results

enum { LN_FEATURES, LN_TOKENS, LN_PAIRS };

struct LnBars {
  uint64_t full[LN_MAX_STAGES], empty[LN_MAX_STAGES];
  uint64_t acc_full[2], acc_empty[2], fin;
  uint64_t res_full[16];
  uint32_t tmem_base;
  int abort;
};

struct LnArgs {
  CUtensorMap tm_a, tm_b;        // the 128-row operand and the BT-row operand
  CUtensorMap tm_out, tm_res;    // tokens, pairs: 32 rows of 128 bytes
  const float *s_a, *s_w;        // per token, per feature (8-bit operands), or null
  const float *bias;             // [N] or null
  const void *res;               // [M, N] like out, or null
  void *out;
  long long ldo, ldr;            // elements
  int M, N;                      // tokens, features
  int tiles_a, tiles_b;          // tiles along the 128-row operand and along the other
  int ksteps;                    // 128-byte steps of K
  int kelems;                    // elements per step
  int act, out_f32, split;
  int32_t *status;
};

// Epilogue warps: four per 32-lane quarter of the widest tiles, else two.
__host__ __device__ constexpr int ln_epi_warps(int mode, int BT) { return mode == LN_PAIRS && BT == 256 ? 16 : 8; }
__host__ __device__ constexpr int ln_threads(int mode, int BT) { return 32 * (LN_W_EPI + ln_epi_warps(mode, BT)); }
// Staging boxes: 16 in all, so one or two per warp.
__host__ __device__ constexpr int ln_boxes(int mode) { return mode == LN_FEATURES ? 0 : 16; }
// What the CTAs that split K send one another: a tile's accumulators.
__host__ __device__ constexpr int ln_xch_bytes(int mode, int BT) { return mode == LN_FEATURES && BT <= 64 ? BT * LN_ROWS * 4 : 0; }
// Rows of the B operand that one CTA loads.
__host__ __device__ constexpr int ln_b_rows(int mode, int BT) { return mode == LN_PAIRS ? BT / 2 : BT; }
__host__ __device__ constexpr int ln_stage_bytes(int mode, int BT) { return LN_A_BYTES + ln_b_rows(mode, BT) * LN_KB; }
__host__ __device__ constexpr int ln_stages(int mode, int BT) {
  return (LN_SMEM - ln_boxes(mode) * LN_BOX - ln_xch_bytes(mode, BT)) / ln_stage_bytes(mode, BT) < LN_MAX_STAGES
             ? (LN_SMEM - ln_boxes(mode) * LN_BOX - ln_xch_bytes(mode, BT)) / ln_stage_bytes(mode, BT)
             : LN_MAX_STAGES;
}
constexpr int ln_smem_bytes(int mode, int BT) {
  return 1024 + ln_stages(mode, BT) * ln_stage_bytes(mode, BT) + ln_boxes(mode) * LN_BOX + ln_xch_bytes(mode, BT) +
         (int)sizeof(LnBars);
}
// TMEM columns of the two accumulator slots: a power of two of at least 32
__host__ __device__ constexpr int ln_tmem_cols(int BT) { return 2 * BT < 32 ? 32 : 2 * BT; }

__device__ __forceinline__ bool ln_aborted(LnBars *b) { return *reinterpret_cast<volatile int *>(&b->abort) != 0; }

// Bounded wait; a wait that runs out aborts the CTA's roles and sets the status.
__device__ __noinline__ bool ln_wait_slow(uint64_t *bar, uint32_t parity, LnBars *b, int32_t *status) {
  const long long deadline = clock64() + WAIT_BUDGET_CYCLES;
  while (!mbar_try_wait(bar, parity)) {
    if (ln_aborted(b)) return false;
    if (clock64() > deadline) {
      *reinterpret_cast<volatile int *>(&b->abort) = 1;
      set_status(status, DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool ln_wait(uint64_t *bar, uint32_t parity, LnBars *b, int32_t *status) {
  if (mbar_try_wait(bar, parity)) return true;
  return ln_wait_slow(bar, parity, b, status);
}
__device__ __forceinline__ bool ln_wait_warp(uint64_t *bar, uint32_t parity, LnBars *b, int32_t *status) {
  return __all_sync(0xffffffffu, ln_wait(bar, parity, b, status));
}

// Tile index -> (A tile, B tile): groups of LN_GROUP A tiles run through all B
// tiles together, so the tiles in flight share operand rows in L2.
__device__ __forceinline__ void ln_tile(const LnArgs &a, int i, int &ta, int &tb) {
  const int per = LN_GROUP * a.tiles_b, g = i / per, r = i - g * per;
  const int h = min(LN_GROUP, a.tiles_a - g * LN_GROUP);
  ta = g * LN_GROUP + r % h;
  tb = r / h;
}

// This CTA's share of the K steps (the whole range without a split).
__device__ __forceinline__ void ln_krange(const LnArgs &a, int rank, int &k0, int &k1) {
  k0 = (int)((long long)a.ksteps * rank / a.split);
  k1 = (int)((long long)a.ksteps * (rank + 1) / a.split);
}

// silu by the hardware exponential and quotient: relative error below 1e-6
// around the origin, where the values are. gelu = v erfc(-v / sqrt 2) / 2 with
// the Chebyshev fit of erfc in Numerical Recipes (W. H. Press et al., "erfcc",
// relative error below 1.2e-7 of its own), which keeps the negative tail's
// relative precision; CUDA's erfcf costs three times the instructions, and the
// epilogue of 4096 x 4096 values with it took longer than the products.
__device__ __forceinline__ float ln_gelu(float v) {
  const float x = -0.70710678118654752f * v, z = fabsf(x);
  const float t = __fdividef(1.0f, __fmaf_rn(0.5f, z, 1.0f));
  float p = 0.17087277f;
  p = __fmaf_rn(p, t, -0.82215223f);
  p = __fmaf_rn(p, t, 1.48851587f);
  p = __fmaf_rn(p, t, -1.13520398f);
  p = __fmaf_rn(p, t, 0.27886807f);
  p = __fmaf_rn(p, t, -0.18628806f);
  p = __fmaf_rn(p, t, 0.09678418f);
  p = __fmaf_rn(p, t, 0.37409196f);
  p = __fmaf_rn(p, t, 1.00002368f);
  p = __fmaf_rn(p, t, -1.26551223f);
  const float e = t * __expf(__fmaf_rn(-z, z, p));   // erfc(|x|)
  return 0.5f * v * (x >= 0.0f ? e : 2.0f - e);
}
__device__ __forceinline__ float ln_relu(float v) { return v > 0.0f ? v : (v == v ? 0.0f : v); }
__device__ __forceinline__ float ln_silu(float v) { return __fdividef(v, 1.0f + __expf(-v)); }

template <int W>
__device__ __forceinline__ void ln_act_all(float (&v)[W], int act) {
  if (act == QMOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = ln_silu(v[i]);
  } else if (act == QMOE_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = ln_relu(v[i]);
  } else if (act == QMOE_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = ln_gelu(v[i]);
  }
}

// Brings a 32-byte sector into L1.
__device__ __forceinline__ void touch(const float *p) {
  asm volatile("{ .reg .f32 t; ld.global.nc.f32 t, [%0]; }" ::"l"(p));
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <bool I8>
__device__ __forceinline__ float ln_acc(float bits, float sa, float sw) {
  if (I8) return __fmul_rn(__fmul_rn(__int2float_rn(__float_as_int(bits)), sa), sw);
  return bits;
}

__device__ __forceinline__ float ln_load(const void *p, long long i, int f32) {
  return f32 ? static_cast<const float *>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void ln_store(void *p, long long i, int f32, float v) {
  if (f32) static_cast<float *>(p)[i] = v;
  else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// Epilogue of a tile whose 128 rows are features: lane = feature, 16 columns = tokens.
template <bool I8>
__device__ __forceinline__ void ln_out_features(const LnArgs &a, float (&v)[16], int n, int m0) {
  if (n >= a.N || m0 >= a.M) return;
  const float sw = I8 ? __ldg(a.s_w + n) : 1.0f, bias = a.bias ? __ldg(a.bias + n) : 0.0f;
  const int mn = min(16, a.M - m0);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = ln_acc<I8>(v[i], I8 ? __ldg(a.s_a + min(m0 + i, a.M - 1)) : 1.0f, sw) + bias;
  ln_act_all(v, a.act);
  if (a.res) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += ln_load(a.res, (long long)min(m0 + i, a.M - 1) * a.ldr + n, a.out_f32);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < mn) ln_store(a.out, (long long)(m0 + i) * a.ldo + n, a.out_f32, v[i]);
}

// Epilogue of 16 neighbouring features (from n0) of the lane's token, into its
// row of a staging box (16-byte chunks from `chunk` on, each at chunk ^ (row % 8),
// the 128-byte swizzle), where the residual already lies.
template <bool I8>
__device__ __forceinline__ void ln_stage_tokens(const LnArgs &a, float (&v)[16], int n0, float sa, uint8_t *row, int chunk) {
  const int swz = threadIdx.x & 7;
  if (n0 + 16 <= a.N) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 sw = I8 ? __ldg(reinterpret_cast<const float4 *>(a.s_w + n0) + j) : make_float4(1.f, 1.f, 1.f, 1.f);
      const float4 bb = a.bias ? __ldg(reinterpret_cast<const float4 *>(a.bias + n0) + j) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[4 * j] = ln_acc<I8>(v[4 * j], sa, sw.x) + bb.x;
      v[4 * j + 1] = ln_acc<I8>(v[4 * j + 1], sa, sw.y) + bb.y;
      v[4 * j + 2] = ln_acc<I8>(v[4 * j + 2], sa, sw.z) + bb.z;
      v[4 * j + 3] = ln_acc<I8>(v[4 * j + 3], sa, sw.w) + bb.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int n = min(n0 + j, a.N - 1);   // (what lies past N is not stored)
      v[j] = ln_acc<I8>(v[j], sa, I8 ? __ldg(a.s_w + n) : 1.0f) + (a.bias ? __ldg(a.bias + n) : 0.0f);
    }
  }
  ln_act_all(v, a.act);
  if (a.out_f32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float4 *p = reinterpret_cast<float4 *>(row + (((chunk + j) ^ swz) << 4));
      float4 x = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      if (a.res) {
        const float4 r = *p;
        x.x += r.x;
        x.y += r.y;
        x.z += r.z;
        x.w += r.w;
      }
      *p = x;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint4 *p = reinterpret_cast<uint4 *>(row + (((chunk + j) ^ swz) << 4));
      uint32_t rw[4] = {0, 0, 0, 0}, ow[4];
      if (a.res) {
        const uint4 r = *p;
        rw[0] = r.x;
        rw[1] = r.y;
        rw[2] = r.z;
        rw[3] = r.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo = v[8 * j + 2 * i], hi = v[8 * j + 2 * i + 1];
        if (a.res) {
          lo += __uint_as_float(rw[i] << 16);
          hi += __uint_as_float(rw[i] & 0xffff0000u);
        }
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        ow[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
      *p = make_uint4(ow[0], ow[1], ow[2], ow[3]);
    }
  }
}

// SEG: a slot holds LN_SEG steps, and the epilogue's threads add the slots.
template <int MODE, int BT, bool I8, bool SEG>
__global__ void __launch_bounds__(ln_threads(MODE, BT), 1) linear_kernel(const __grid_constant__ LnArgs a) {
  extern __shared__ uint8_t ln_smem[];
  constexpr bool FEATURES = MODE == LN_FEATURES, PAIRS = MODE == LN_PAIRS;
  constexpr int STAGES = ln_stages(MODE, BT), STAGE = ln_stage_bytes(MODE, BT), BROWS = ln_b_rows(MODE, BT);
  constexpr int CTAS = PAIRS ? 2 : 1;                       // CTAs on one tile
  constexpr int N_EPI = ln_epi_warps(MODE, BT), THREADS = ln_threads(MODE, BT);
  constexpr int EPI_COLS = BT < 32 ? BT : BT / (N_EPI / 4);  // columns of an epilogue warp
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(ln_smem) + 1023) & ~(uintptr_t)1023);
  uint8_t *boxes = sm + STAGES * STAGE;
  float *xch = reinterpret_cast<float *>(boxes + ln_boxes(MODE) * LN_BOX);
  LnBars *b = reinterpret_cast<LnBars *>(reinterpret_cast<uint8_t *>(xch) + ln_xch_bytes(MODE, BT));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIRS || a.split > 1 ? (int)dense::cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&b->full[i], 1);
      mbar_init(&b->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b->acc_full[i], 1);
      mbar_init(&b->acc_empty[i], CTAS * N_EPI);
    }
    for (int i = 0; i < 16; ++i) mbar_init(&b->res_full[i], 1);
    mbar_init(&b->fin, 1);
    b->abort = 0;
    fence_mbar_init();
  }
  if (warp == LN_W_MMA) {
    if (PAIRS) {
      dense::tmem_alloc_pair(&b->tmem_base, ln_tmem_cols(BT));
    } else {
      tc05::tmem_alloc(&b->tmem_base, ln_tmem_cols(BT));
      tc05::tmem_relinquish();
    }
  }
  if (threadIdx.x == 32 * LN_W_TMA) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a.tm_a)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a.tm_b)) : "memory");
  }
  tc05::fence_before_sync();
  __syncthreads();
  if (PAIRS) dense::cluster_sync();   // the other CTA's barriers are ready
  else if (a.split > 1) dense::cluster_arrive();   // (waited for before the CTAs exchange sums)
  tc05::fence_after_sync();
  pdl_wait();   // (so far nothing but this kernel's own memory)
  pdl_launch_dependents();
  const uint32_t tmem = b->tmem_base;
  const int ntiles = a.tiles_a * a.tiles_b;
  const int per = PAIRS ? 2 : a.split;   // CTAs that share a tile
  const int first = blockIdx.x / per, step = gridDim.x / per;
  int k0 = 0, k1 = a.ksteps;
  if (!PAIRS) ln_krange(a, rank, k0, k1);
  const int segs = SEG ? (k1 - k0 + LN_SEG - 1) / LN_SEG : 1;   // accumulator slots of a tile
  const int a_row = LN_ROWS * (PAIRS ? 2 : 1);                   // A rows per tile

  if (warp == LN_W_TMA) {
    if (lane == 0) {
      uint32_t g = 0;
      bool ok = true;
      for (int i = first; i < ntiles && ok; i += step) {
        int ta, tb;
        ln_tile(a, i, ta, tb);
        for (int s = k0; s < k1; ++s, ++g) {
          const int st = g % STAGES;
          if (!ln_wait(&b->empty[st], ((g / STAGES) & 1) ^ 1, b, a.status)) {
            ok = false;
            break;
          }
          uint8_t *to = sm + st * STAGE;
          if (PAIRS) {
            // both CTAs' loads complete on the first CTA's barrier
            const uint32_t bar = dense::peer_addr(&b->full[st], 0);
            if (rank == 0) mbar_arrive_expect_tx(&b->full[st], 2 * STAGE);
            dense::tma_load_2d_pair(to, &a.tm_a, s * a.kelems, ta * a_row + rank * LN_ROWS, bar);
            dense::tma_load_2d_pair(to + LN_A_BYTES, &a.tm_b, s * a.kelems, tb * BT + rank * BROWS, bar);
          } else {
            mbar_arrive_expect_tx(&b->full[st], STAGE);
            dense::tma_load_2d(to, &a.tm_a, s * a.kelems, ta * a_row, &b->full[st]);
            dense::tma_load_2d(to + LN_A_BYTES, &a.tm_b, s * a.kelems, tb * BT, &b->full[st]);
          }
        }
      }
      // no copy may still be writing shared memory when a CTA exits
      if (rank == 0 || !PAIRS) {
        const uint32_t u0 = g > (uint32_t)STAGES ? g - STAGES : 0;
        for (uint32_t u = u0; u < g; ++u)
          if (!mbar_wait(&b->full[u % STAGES], (u / STAGES) & 1, clock64() + WAIT_BUDGET_CYCLES))
            set_status(a.status, DEV_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (warp == LN_W_MMA) {
    if (!PAIRS || rank == 0) {
      constexpr int MM = LN_ROWS * CTAS;
      const uint32_t idesc = I8 ? dense::idesc_s8_s32(MM, BT) : tc05::idesc_bf16_f32(MM, BT);
      uint32_t g = 0, c = 0;   // steps, accumulator slots used
      bool ok = true;
      for (int i = first; i < ntiles && ok; i += step) {
        for (int s = k0; s < k1; ++s, ++g) {
          const bool fresh = SEG ? (s - k0) % LN_SEG == 0 : s == k0;
          const bool ends = SEG ? (s - k0) % LN_SEG == LN_SEG - 1 || s == k1 - 1 : s == k1 - 1;
          const int slot = c & 1, st = g % STAGES;
          if (fresh && !ln_wait_warp(&b->acc_empty[slot], ((c >> 1) & 1) ^ 1, b, a.status)) {
            ok = false;
            break;
          }
          if (!ln_wait_warp(&b->full[st], (g / STAGES) & 1, b, a.status)) {
            ok = false;
            break;
          }
          tc05::fence_after_sync();
          const uint32_t d = tmem + slot * BT;
          if (tc05::elect_one()) {
            const uint64_t da = tc05::sw128_desc(smem_u32(sm + st * STAGE));
            const uint64_t db = tc05::sw128_desc(smem_u32(sm + st * STAGE + LN_A_BYTES));
#pragma unroll
            for (int kk = 0; kk < LN_KB / 32; ++kk) {
              const uint32_t more = !fresh || kk > 0;
              if (PAIRS) dense::mma_pair<I8>(d, da + 2 * kk, db + 2 * kk, idesc, more);
              else if (I8) dense::mma_s8(d, da + 2 * kk, db + 2 * kk, idesc, more);
              else tc05::mma_bf16(d, da + 2 * kk, db + 2 * kk, idesc, more);
            }
            if (PAIRS) {
              dense::commit_pair(&b->empty[st]);
              if (ends) dense::commit_pair(&b->acc_full[slot]);
            } else {
              tc05::commit(&b->empty[st]);
              if (ends) tc05::commit(&b->acc_full[slot]);
            }
          }
          __syncwarp();
          if (ends) ++c;
        }
      }
      // every issued product has finished before tensor memory is freed
      if (tc05::elect_one()) {
        if (PAIRS) dense::commit_pair(&b->fin);
        else tc05::commit(&b->fin);
      }
      __syncwarp();
      if (!mbar_wait(&b->fin, 0, clock64() + WAIT_BUDGET_CYCLES)) set_status(a.status, DEV_TIMEOUT);
    }
  } else if (warp >= LN_W_EPI && (PAIRS || a.split == 1)) {
    const int w = warp - LN_W_EPI, q = warp & 3, part = w >> 2;   // (a warp reads the TMEM lanes of its number mod 4)
    const int col0 = BT < 32 ? 0 : part * EPI_COLS;
    const bool works = BT >= 32 || part == 0;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const uint32_t empty0 = PAIRS ? dense::peer_addr(&b->acc_empty[0], 0) : 0;
    uint32_t c = 0;   // accumulator slots read
    bool ok = true;
    auto wait_slot = [&](int slot) {
      const bool good = ln_wait_warp(&b->acc_full[slot], (c >> 1) & 1, b, a.status);
      tc05::fence_after_sync();
      return good;
    };
    auto release = [&](int slot) {
      tc05::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (PAIRS) dense::mbar_arrive_peer(empty0 + slot * 8);
        else mbar_arrive(&b->acc_empty[slot]);
      }
      ++c;
    };
    if constexpr (FEATURES) {
      constexpr int NCH = EPI_COLS / 16;
      for (int i = first; i < ntiles && ok; i += step) {
        int ta, tb;
        ln_tile(a, i, ta, tb);
        const int n = ta * LN_ROWS + q * 32 + lane, m0 = tb * BT + col0;
        float v[NCH][16];
        if (n < a.N) {   // on their way while the products run
          if (I8) touch(a.s_w + n);
          if (a.bias) touch(a.bias + n);
        }
        if (I8 && lane < EPI_COLS && m0 + lane < a.M) touch(a.s_a + m0 + lane);
        for (int sg = 0; sg < segs; ++sg) {
          const int slot = c & 1;
          ok = wait_slot(slot);
          if (!ok) break;
          if (works) {
#pragma unroll
            for (int h = 0; h < NCH; ++h) {
              float x[16];
              tc05::ld16(tmem + slot * BT + lanes + col0 + 16 * h, x);
#pragma unroll
              for (int j = 0; j < 16; ++j) v[h][j] = sg == 0 ? x[j] : __fadd_rn(v[h][j], x[j]);
            }
          }
          release(slot);
        }
        if (ok && works)
#pragma unroll
          for (int h = 0; h < NCH; ++h) ln_out_features<I8>(a, v[h], n, m0 + 16 * h);
        __syncwarp();
      }
    } else {
      // the warp's staging boxes in turn: box (column group) by box through all
      // tiles, the residual of the next box loaded while this one is formed
      constexpr int NBOX = 16 / N_EPI;
      const int es = a.out_f32 ? 4 : 2, bcols = 128 / es, ngroups = EPI_COLS / bcols;
      uint8_t *box0 = boxes + w * NBOX * LN_BOX;
      uint64_t *rbar = &b->res_full[w * NBOX];
      uint32_t n_used = 0;         // boxes stored so far
      struct Tile {
        int m, n;   // the warp's first row and column
      };
      auto tile_at = [&](int i) {
        int ta, tb;
        ln_tile(a, i, ta, tb);
        return Tile{ta * a_row + (PAIRS ? rank * LN_ROWS : 0) + q * 32, tb * BT + col0};
      };
      // (lane 0, once the box's last store has been read; nothing past the matrix)
      auto load_res = [&](int m, int n, uint32_t k) {
        if (m >= a.M || n >= a.N) return false;
        mbar_arrive_expect_tx(&rbar[k % NBOX], LN_BOX);
        dense::tma_load_2d(box0 + k % NBOX * LN_BOX, &a.tm_res, n, m, &rbar[k % NBOX]);
        return true;
      };
      uint32_t phase[NBOX] = {};   // residual loads waited for, per box
      bool pending = false;        // box n_used has a residual under way
      Tile next = tile_at(first);
      if (a.res && lane == 0) pending = load_res(next.m, next.n, 0);
      pending = __shfl_sync(0xffffffffu, pending, 0);
      for (int i = first; i < ntiles && ok; i += step) {
        constexpr int NCH = EPI_COLS / 16;
        float acc[SEG ? NCH : 1][16];
        const Tile here = next;
        const bool last_tile = i + step >= ntiles;
        next = tile_at(last_tile ? i : i + step);
        const float sa = I8 && here.m + lane < a.M ? __ldg(a.s_a + here.m + lane) : 1.0f;
        // the columns' bias and scales into L1 while the products run: every 16
        // columns would wait for them otherwise
        for (int n = here.n + 8 * lane; n < min(a.N, here.n + EPI_COLS); n += 256) {
          if (a.bias) touch(a.bias + n);
          if (I8) touch(a.s_w + n);
        }
        int slot = c & 1;
        if constexpr (SEG) {
          for (int sg = 0; sg < segs; ++sg) {
            slot = c & 1;
            ok = wait_slot(slot);
            if (!ok) break;
#pragma unroll
            for (int h = 0; h < NCH; ++h) {
              float x[16];
              tc05::ld16(tmem + slot * BT + lanes + col0 + 16 * h, x);
#pragma unroll
              for (int j = 0; j < 16; ++j) acc[h][j] = sg == 0 ? x[j] : __fadd_rn(acc[h][j], x[j]);
            }
            release(slot);
          }
        } else {
          ok = wait_slot(slot);
        }
        if (!ok) break;
        auto one_box = [&](int g, auto values) {   // values(h): 16 columns of the group
          const int m0 = here.m, n0 = here.n + g * bcols;
          const bool live = m0 < a.M && n0 < a.N;
          const uint32_t k = n_used % NBOX;
          uint8_t *box = box0 + k * LN_BOX;
          if (live && a.res) {
            uint32_t ph = phase[0];
            if (NBOX > 1 && k == 1) ph = phase[NBOX - 1];
            ok = ln_wait_warp(&rbar[k], ph & 1, b, a.status);
            if (k == 0) ++phase[0];
            else ++phase[NBOX - 1];
          } else if (live) {
            if (lane == 0) dense::store_wait_read<NBOX - 1>();
            __syncwarp();
          }
          pending = false;
          if (!ok) return;
          if (live) {
            values(box + lane * 128, n0);
            tc05::fence_async_smem();
            __syncwarp();
            if (lane == 0) dense::tma_store_2d(&a.tm_out, n0, m0, box);
            ++n_used;
          }
          if (a.res) {
            // the next box: of this tile or of the next
            const bool more = g + 1 < ngroups;
            if (lane == 0 && (more || !last_tile)) {
              dense::store_wait_read<NBOX - 1>();
              pending = load_res(more ? m0 : next.m, more ? n0 + bcols : next.n, n_used);
            }
            pending = __shfl_sync(0xffffffffu, pending, 0);
          }
        };
        if constexpr (SEG) {   // fp32: a box is 32 columns
#pragma unroll
          for (int g = 0; g < EPI_COLS / 32; ++g)
            one_box(g, [&](uint8_t *row, int n0) {
              ln_stage_tokens<I8>(a, acc[2 * g], n0, sa, row, 0);
              ln_stage_tokens<I8>(a, acc[2 * g + 1], n0 + 16, sa, row, 4);
            });
        } else {
#pragma unroll 1
          for (int g = 0; g < ngroups; ++g)
            one_box(g, [&](uint8_t *row, int n0) {
#pragma unroll 1
              for (int h = 0; h < bcols / 32; ++h) {
                const uint32_t from = tmem + slot * BT + lanes + col0 + g * bcols + 32 * h;
                float v[16], v2[16];
                __syncwarp();
                tc05::ld16x2(from, from + 16, v, v2);
                ln_stage_tokens<I8>(a, v, n0 + 32 * h, sa, row, 2 * h * es);
                ln_stage_tokens<I8>(a, v2, n0 + 32 * h + 16, sa, row, (2 * h + 1) * es);
              }
            });
          release(slot);
        }
      }
      // a residual load that nobody waited for (after an error) still lands
      if (pending && lane == 0) {
        const uint32_t k = n_used % NBOX;
        if (!mbar_wait(&rbar[k], (k == 0 ? phase[0] : phase[NBOX - 1]) & 1, clock64() + WAIT_BUDGET_CYCLES))
          set_status(a.status, DEV_TIMEOUT);
      }
      if (lane == 0) dense::store_wait_all();
      __syncwarp();
    }
  }
  __syncwarp();

  if constexpr (FEATURES && BT <= 64) {
    if (a.split > 1) {
      // one tile per cluster. The accumulators of feature f go to CTA
      // f / (128 / split), [source CTA][token][its features], through
      // distributed shared memory.
      const int fs = 7 - (31 - __clz(a.split)), fl = 1 << fs;   // features per CTA: 128 / split
      int ta, tb;
      ln_tile(a, first, ta, tb);
      const int q = warp & 3, half = (warp - LN_W_EPI) >> 2, f = q * 32 + lane;
      const int col0 = BT < 32 ? 0 : half * EPI_COLS;
      constexpr int NCH = EPI_COLS / 16;
      float v[NCH][16];
      bool have = false;
      if (warp >= LN_W_EPI) {
        have = true;
        // what the values that end here need, on its way while the products run
        const int ends = min(BT, a.M - tb * BT) << fs;
        for (int i = threadIdx.x - 32 * LN_W_EPI; i < ends; i += 32 * N_EPI) {
          const int m = tb * BT + (i >> fs), n = ta * LN_ROWS + (rank << fs) + (i & (fl - 1));
          if (n >= a.N) continue;
          if (I8) touch(a.s_a + m), touch(a.s_w + n);
          if (a.bias) touch(a.bias + n);
          if (a.res) prefetch_l2(static_cast<const uint8_t *>(a.res) + ((long long)m * a.ldr + n) * (a.out_f32 ? 4 : 2));
        }
        for (int sg = 0; sg < segs && have; ++sg) {
          const int slot = sg & 1;
          have = ln_wait_warp(&b->acc_full[slot], (sg >> 1) & 1, b, a.status);
          if (!have) break;
          tc05::fence_after_sync();
          if (BT >= 32 || half == 0)
#pragma unroll
            for (int h = 0; h < NCH; ++h) {
              float x[16];
              tc05::ld16(tmem + slot * BT + ((uint32_t)(q * 32) << 16) + col0 + 16 * h, x);
#pragma unroll
              for (int j = 0; j < 16; ++j) v[h][j] = sg == 0 ? x[j] : __fadd_rn(v[h][j], x[j]);
            }
          tc05::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b->acc_empty[slot]);
        }
      }
      dense::cluster_wait();   // every CTA of the cluster is running
      if (have && (BT >= 32 || half == 0)) {
        float *dst = dense::peer(xch, f >> fs) + ((rank * BT) << fs) + (f & (fl - 1));
        const int mm = min(EPI_COLS, a.M - tb * BT - col0);
#pragma unroll
        for (int h = 0; h < NCH; ++h)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (16 * h + i < mm) dst[(col0 + 16 * h + i) << fs] = v[h][i];
      }
      __syncwarp();
      dense::cluster_sync();
      const int m0 = tb * BT, total = min(BT, a.M - m0) << fs, n0 = ta * LN_ROWS + (rank << fs);
      // four values a thread at once: their loads in flight together
      for (int i0 = threadIdx.x; i0 < total; i0 += 4 * THREADS) {
        float x[4], res[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = min(i0 + j * THREADS, total - 1), m = i >> fs, n = min(n0 + (i & (fl - 1)), a.N - 1);
          float acc = 0.0f;
          int sum = 0;
          for (int r = 0; r < a.split; ++r) {
            const float y = xch[((r * BT + m) << fs) + (i & (fl - 1))];
            if (I8) sum += __float_as_int(y);
            else acc = __fadd_rn(acc, y);
          }
          x[j] = ln_acc<I8>(I8 ? __int_as_float(sum) : acc, I8 ? __ldg(a.s_a + m0 + m) : 1.0f, I8 ? __ldg(a.s_w + n) : 1.0f) +
                 (a.bias ? __ldg(a.bias + n) : 0.0f);
          res[j] = a.res ? ln_load(a.res, (long long)(m0 + m) * a.ldr + n, a.out_f32) : 0.0f;
        }
        ln_act_all(x, a.act);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = i0 + j * THREADS, n = n0 + (i & (fl - 1));
          if (i < total && n < a.N) {
            const float y = a.res ? x[j] + res[j] : x[j];
            ln_store(a.out, (long long)(m0 + (i >> fs)) * a.ldo + n, a.out_f32, y);
          }
        }
      }
    }
  }

  tc05::fence_before_sync();
  __syncthreads();
  // The pair's other CTA issues no products: it waits for the end of theirs only now, when its
  // epilogue has read the last of them (from the kernel's start the wait would span the whole
  // kernel, and one that works for longer than a wait's budget would be taken for a hang).
  if (PAIRS && rank && warp == LN_W_MMA && !mbar_wait(&b->fin, 0, clock64() + 2 * WAIT_BUDGET_CYCLES))
    set_status(a.status, DEV_TIMEOUT);
  if (PAIRS) dense::cluster_sync();   // neither CTA's memory is in use by the other any more
  if (warp == LN_W_MMA) {
    tc05::fence_after_sync();
    if (PAIRS) dense::tmem_dealloc_pair(tmem, ln_tmem_cols(BT));
    else tc05::tmem_dealloc(tmem, ln_tmem_cols(BT));
  }
}

// ---------------------------------------------------------------- host side --
// [rows][cols] with row stride ld (elements) of 1, 2 or 4 bytes, boxes of
// box_rows x 128 bytes in the 128-byte swizzle.
bool ln_map(CUtensorMap *m, const void *base, int es, int cols, int rows, long long ld, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = dense::tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * es};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / es), (cuuint32_t)box_rows};
  const cuuint32_t st[2] = {1, 1};
  return enc(m,
             es == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
             : es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
             2, const_cast<void *>(base), dims, strides, box, st, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int BT>
const void *ln_kernel(bool i8, bool f32) {
  if (i8) return (const void *)linear_kernel<MODE, BT, true, false>;
  // (fp32 results from wide pairs: a thread's sums do not fit its registers)
  if (f32) return (const void *)linear_kernel<MODE, MODE == LN_PAIRS ? 128 : BT, false, true>;
  return (const void *)linear_kernel<MODE, BT, false, false>;
}

int ln_max_clusters(int size) {
  static dense::ClusterCounts known;   // (of one kernel that stands for all that split K: they take an SM a CTA)
  return dense::max_clusters(known, size, (const void *)linear_kernel<LN_FEATURES, 16, true, false>, ln_threads(LN_FEATURES, 16),
                             ln_smem_bytes(LN_FEATURES, 16));
}

qmoe_status ln_launch(const void *fn, int smem, int threads, const LnArgs &a, int grid, int cluster, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return dense::launched(e);
  LnArgs args = a;
  void *params[] = {&args};
  return dense::launch(fn, grid, threads, smem, cluster, params, s);
}

}  // namespace
}  // namespace qmoe

using namespace qmoe;

extern "C" qmoe_status qmoe_linear(const void *a, int in_dtype, const void *w, int M, int N, int K, const float *a_scale,
                                   const float *w_scale, const float *bias, int act, const void *residual, void *out,
                                   int out_dtype, int64_t lda, int64_t ldw, int64_t ldr, int64_t ldo,
                                   int32_t *dev_status, qmoe_stream_t stream) {
  if (!a || !w || !out || !dev_status || M < 1 || N < 1 || K < 1) return QMOE_ERR_INVALID_ARG;
  if (in_dtype != QMOE_BF16 && in_dtype != QMOE_I8) return QMOE_ERR_INVALID_ARG;
  if (out_dtype != QMOE_F32 && out_dtype != QMOE_BF16) return QMOE_ERR_INVALID_ARG;
  if (act < QMOE_ACT_NONE || act > QMOE_ACT_GELU) return QMOE_ERR_INVALID_ARG;
  const bool i8 = in_dtype == QMOE_I8;
  if (i8 != (a_scale != nullptr) || i8 != (w_scale != nullptr)) return QMOE_ERR_INVALID_ARG;
  const int es = i8 ? 1 : 2, os = out_dtype == QMOE_F32 ? 4 : 2;
  if (lda == 0) lda = K;
  if (ldw == 0) ldw = K;
  if (ldo == 0) ldo = N;
  if (ldr == 0) ldr = N;
  if (lda < K || ldw < K || ldo < N || (residual && ldr < N)) return QMOE_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(w) || !aligned16(out) || !aligned16(residual) || !aligned16(a_scale) ||
      !aligned16(w_scale) || !aligned16(bias) || (reinterpret_cast<uintptr_t>(dev_status) & 3))
    return QMOE_ERR_INVALID_ARG;
  // rows of a and w start on 16 bytes (the copy engine's rule); strides below 2^40 bytes
  if (lda > LN_MAX_LD || ldw > LN_MAX_LD || ldo > LN_MAX_LD || (residual && ldr > LN_MAX_LD)) return QMOE_ERR_UNSUPPORTED;
  if (lda * es % 16 || ldw * es % 16 || K > LN_MAX_K || M > LN_MAX_MN || N > LN_MAX_MN) return QMOE_ERR_UNSUPPORTED;
  // a residual that is overwritten in place: row by row, or results would be read as residuals
  if (residual == out && ldr != ldo && M > 1) return QMOE_ERR_INVALID_ARG;
  LnArgs g{};
  g.s_a = a_scale;
  g.s_w = w_scale;
  g.bias = bias;
  g.res = residual;
  g.out = out;
  g.ldo = ldo;
  g.ldr = ldr;
  g.M = M;
  g.N = N;
  g.kelems = LN_KB / es;
  g.ksteps = (K + g.kelems - 1) / g.kelems;
  g.act = act;
  g.out_f32 = out_dtype == QMOE_F32;
  g.split = 1;
  g.status = dev_status;
  const int sms = num_sms();
  // a tensor store ends on 16 bytes: a row whose end does not would be overwritten past it
  const bool vec = (long long)N * os % 16 == 0 && ldo * os % 16 == 0 && (!residual || ldr * os % 16 == 0);
  const bool f32 = g.out_f32;
  // tokens or pairs where they fill half the machine (and rows can be stored
  // 16 bytes at a time); else narrow tiles of features, with K split
  int mode = LN_FEATURES;
  if (vec && M > 64) {
    const long long alone = (long long)((M + 127) / 128) * ((N + 127) / 128);
    const long long pairs = (long long)((M + 255) / 256) * ((N + 255) / 256);
    if (pairs * 2 >= sms) mode = LN_PAIRS;
    else if (alone * 2 >= sms) mode = LN_TOKENS;
  }
  int BT = mode == LN_PAIRS && (i8 || !f32) ? 256 : 128;
  if (mode == LN_FEATURES && (vec || M <= 64)) {
    // the tile width and split of K with the least time in cycles: a step takes
    // 2.9 per operand row (measured: 45 bytes a cycle and SM), an exchange and
    // the values' way out 3000 + 40 per token of the tile
    double best = 0.0;
    for (int bt = 16; bt <= 64; bt *= 2) {
      const long long tiles = (long long)((N + LN_ROWS - 1) / LN_ROWS) * ((M + bt - 1) / bt);
      int split = 1;
      for (int s = 2; s <= LN_MAX_SPLIT && tiles * s <= sms && g.ksteps >= 2 * s; s *= 2)
        if (tiles <= ln_max_clusters(s)) split = s;
      const double waves = (double)((tiles * split + sms - 1) / sms);
      const double t = waves * ((g.ksteps + split - 1) / split * 2.9 * (LN_ROWS + bt)) + 3000.0 + 40.0 * bt;
      if (bt == 16 || t < best) {
        best = t;
        BT = bt;
        g.split = split;
      }
      if (bt >= M) break;
    }
  }
  const int rows_a = mode == LN_FEATURES ? N : M, rows_b = mode == LN_FEATURES ? M : N;
  const int tile_a = mode == LN_PAIRS ? 2 * LN_ROWS : LN_ROWS;
  g.tiles_a = (rows_a + tile_a - 1) / tile_a;
  g.tiles_b = (rows_b + BT - 1) / BT;
  const long long nt = (long long)g.tiles_a * g.tiles_b;
  if (nt > 0x1fffffffLL) return QMOE_ERR_UNSUPPORTED;
  if (!ln_map(&g.tm_a, mode == LN_FEATURES ? w : a, es, K, rows_a, mode == LN_FEATURES ? ldw : lda, LN_ROWS) ||
      !ln_map(&g.tm_b, mode == LN_FEATURES ? a : w, es, K, rows_b, mode == LN_FEATURES ? lda : ldw, ln_b_rows(mode, BT)))
    return QMOE_ERR_CUDA;
  if (mode != LN_FEATURES) {
    if (!ln_map(&g.tm_out, out, os, N, M, ldo, 32)) return QMOE_ERR_CUDA;
    if (residual && !ln_map(&g.tm_res, residual, os, N, M, ldr, 32)) return QMOE_ERR_CUDA;
  }
  const void *fn;
  if (mode == LN_FEATURES) {
    switch (BT) {
      case 16: fn = ln_kernel<LN_FEATURES, 16>(i8, f32); break;
      case 32: fn = ln_kernel<LN_FEATURES, 32>(i8, f32); break;
      case 64: fn = ln_kernel<LN_FEATURES, 64>(i8, f32); break;
      default: fn = ln_kernel<LN_FEATURES, 128>(i8, f32); break;
    }
  } else {
    fn = mode == LN_PAIRS ? ln_kernel<LN_PAIRS, 256>(i8, f32) : ln_kernel<LN_TOKENS, 128>(i8, f32);
  }
  const int smem = ln_smem_bytes(mode, BT), threads = ln_threads(mode, BT);
  if ((size_t)smem > max_smem_optin()) return QMOE_ERR_UNSUPPORTED;
  const int cluster = mode == LN_PAIRS ? 2 : g.split;
  const int grid = cluster * (int)(nt < sms / cluster || g.split > 1 ? nt : sms / cluster);
  return ln_launch(fn, smem, threads, g, grid, cluster, (cudaStream_t)stream);
}
