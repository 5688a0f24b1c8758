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
//   tokens   - the 128 rows are tokens, a thread holds 32 neighbouring features
//     of its token per load and writes them with 16-byte stores: large batches.
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
constexpr int LN_W_TMA = 0, LN_W_MMA = 1, LN_W_EPI = 4, LN_N_EPI = 8;
constexpr int LN_THREADS = 32 * (LN_W_EPI + LN_N_EPI);
constexpr int LN_MAX_STAGES = 10;
constexpr int LN_MAX_SPLIT = 8;
constexpr int LN_MAX_K = 65536;                  // keeps |int32 sums| below 2^31
constexpr int LN_SMEM = 200 * 1024;              // ring budget
constexpr int LN_GROUP = 8;                      // A tiles that share B tiles in L2
constexpr int LN_SEG = 4;                        // steps per accumulator slot of fp32 results

enum { LN_FEATURES, LN_TOKENS, LN_PAIRS };

struct LnBars {
  uint64_t full[LN_MAX_STAGES], empty[LN_MAX_STAGES];
  uint64_t acc_full[2], acc_empty[2], fin;
  uint32_t tmem_base;
  int abort;
};

struct LnArgs {
  CUtensorMap tm_a, tm_b;        // the 128-row operand and the BT-row operand
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

// Rows of the B operand that one CTA loads.
__host__ __device__ constexpr int ln_b_rows(int mode, int BT) { return mode == LN_PAIRS ? BT / 2 : BT; }
__host__ __device__ constexpr int ln_stage_bytes(int mode, int BT) { return LN_A_BYTES + ln_b_rows(mode, BT) * LN_KB; }
__host__ __device__ constexpr int ln_stages(int mode, int BT) {
  return LN_SMEM / ln_stage_bytes(mode, BT) < LN_MAX_STAGES ? LN_SMEM / ln_stage_bytes(mode, BT) : LN_MAX_STAGES;
}
constexpr int ln_smem_bytes(int mode, int BT) {
  return 1024 + ln_stages(mode, BT) * ln_stage_bytes(mode, BT) + (int)sizeof(LnBars);
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

// silu by the hardware exponential and quotient (relative error below 1e-6
// around the origin, where the values are), gelu by erfc, which keeps the
// negative tail's relative precision. One copy of erfc's code, called: inlined
// into every unrolled element it does not fit the instruction cache.
__device__ __noinline__ float ln_gelu(float v) { return 0.5f * v * erfcf(-0.70710678f * v); }
__device__ __forceinline__ float ln_relu(float v) { return v > 0.0f ? v : (v == v ? 0.0f : v); }
__device__ __forceinline__ float ln_silu(float v) { return __fdividef(v, 1.0f + __expf(-v)); }

__device__ __forceinline__ float ln_act(float v, int act) {
  if (act == QMOE_ACT_NONE) return v;
  if (act == QMOE_ACT_RELU) return ln_relu(v);
  return act == QMOE_ACT_SILU ? ln_silu(v) : ln_gelu(v);
}
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

// One value of the result from its accumulator.
template <bool I8>
__device__ __forceinline__ void ln_finish(const LnArgs &a, float bits, int m, int n, float sw, float bias) {
  float v = ln_acc<I8>(bits, I8 ? __ldg(a.s_a + m) : 1.0f, sw) + bias;
  v = ln_act(v, a.act);
  if (a.res) v += ln_load(a.res, (long long)m * a.ldr + n, a.out_f32);
  ln_store(a.out, (long long)m * a.ldo + n, a.out_f32, v);
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

// Residual values of W neighbouring features of a token, as stored.
template <int W>
struct LnRes {
  uint4 q[W / 4];
};
template <int W>
__device__ __forceinline__ void ln_load_res(const LnArgs &a, LnRes<W> &r, int m, int n0) {
  if (!a.res || m >= a.M || n0 + W > a.N) return;
  const long long at = (long long)m * a.ldr + n0;
  const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.res) + at * (a.out_f32 ? 4 : 2));
#pragma unroll
  for (int j = 0; j < W / 8; ++j) r.q[j] = p[j];
  if (a.out_f32)
#pragma unroll
    for (int j = W / 8; j < W / 4; ++j) r.q[j] = p[j];
}

// Epilogue of W neighbouring features (from n0) of token m.
template <bool I8, int W>
__device__ __forceinline__ void ln_out_tokens(const LnArgs &a, float (&v)[W], int m, int n0, float sa, const LnRes<W> &res) {
  if (m >= a.M) return;
  if (n0 + W > a.N) {
    for (int i = 0; i < W; ++i)
      if (n0 + i < a.N) {
        float x = v[0];   // v is indexed at compile time only
#pragma unroll
        for (int j = 1; j < W; ++j) x = j == i ? v[j] : x;
        ln_finish<I8>(a, x, m, n0 + i, I8 ? __ldg(a.s_w + n0 + i) : 1.0f, a.bias ? __ldg(a.bias + n0 + i) : 0.0f);
      }
    return;
  }
#pragma unroll
  for (int j = 0; j < W / 4; ++j) {
    const float4 sw = I8 ? __ldg(reinterpret_cast<const float4 *>(a.s_w + n0) + j) : make_float4(1.f, 1.f, 1.f, 1.f);
    const float4 bb = a.bias ? __ldg(reinterpret_cast<const float4 *>(a.bias + n0) + j) : make_float4(0.f, 0.f, 0.f, 0.f);
    v[4 * j] = ln_acc<I8>(v[4 * j], sa, sw.x) + bb.x;
    v[4 * j + 1] = ln_acc<I8>(v[4 * j + 1], sa, sw.y) + bb.y;
    v[4 * j + 2] = ln_acc<I8>(v[4 * j + 2], sa, sw.z) + bb.z;
    v[4 * j + 3] = ln_acc<I8>(v[4 * j + 3], sa, sw.w) + bb.w;
  }
  ln_act_all(v, a.act);
  const long long oo = (long long)m * a.ldo + n0;
  if (a.out_f32) {
    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + oo);
#pragma unroll
    for (int j = 0; j < W / 4; ++j) {
      float4 x = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      if (a.res) {
        const uint4 q = res.q[j];
        x.x += __uint_as_float(q.x);
        x.y += __uint_as_float(q.y);
        x.z += __uint_as_float(q.z);
        x.w += __uint_as_float(q.w);
      }
      o[j] = x;
    }
  } else {
    uint4 *o = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + oo);
#pragma unroll
    for (int j = 0; j < W / 8; ++j) {
      uint32_t rw[4] = {0, 0, 0, 0}, ow[4];
      if (a.res) {
        rw[0] = res.q[j].x;
        rw[1] = res.q[j].y;
        rw[2] = res.q[j].z;
        rw[3] = res.q[j].w;
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
      o[j] = make_uint4(ow[0], ow[1], ow[2], ow[3]);
    }
  }
}

// SEG: a slot holds LN_SEG steps, and the epilogue's threads add the slots.
template <int MODE, int BT, bool I8, bool SEG>
__global__ void __launch_bounds__(LN_THREADS, 1) linear_kernel(const __grid_constant__ LnArgs a) {
  extern __shared__ uint8_t ln_smem[];
  constexpr bool FEATURES = MODE == LN_FEATURES, PAIRS = MODE == LN_PAIRS;
  constexpr int STAGES = ln_stages(MODE, BT), STAGE = ln_stage_bytes(MODE, BT), BROWS = ln_b_rows(MODE, BT);
  constexpr int CTAS = PAIRS ? 2 : 1;                       // CTAs on one tile
  constexpr int EPI_COLS = BT < 32 ? BT : BT / 2;           // columns of an epilogue warp
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(ln_smem) + 1023) & ~(uintptr_t)1023);
  LnBars *b = reinterpret_cast<LnBars *>(sm + STAGES * STAGE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIRS || a.split > 1 ? (int)dense::cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&b->full[i], 1);
      mbar_init(&b->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b->acc_full[i], 1);
      mbar_init(&b->acc_empty[i], CTAS * LN_N_EPI);
    }
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
  tc05::fence_after_sync();
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
    }
    if (!mbar_wait(&b->fin, 0, clock64() + WAIT_BUDGET_CYCLES * (PAIRS && rank ? 2 : 1))) set_status(a.status, DEV_TIMEOUT);
  } else if (warp >= LN_W_EPI && (PAIRS || a.split == 1)) {
    const int w = warp - LN_W_EPI, q = w & 3, half = w >> 2;
    const int col0 = BT < 32 ? 0 : half * EPI_COLS;
    const bool works = BT >= 32 || half == 0;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const uint32_t empty0 = PAIRS ? dense::peer_addr(&b->acc_empty[0], 0) : 0;
    uint32_t c = 0;
    bool ok = true;
    for (int i = first; i < ntiles && ok; i += step) {
      int ta, tb;
      ln_tile(a, i, ta, tb);
      const int row = ta * a_row + (PAIRS ? rank * LN_ROWS : 0) + q * 32 + lane;   // feature, or token
      const int colb = tb * BT + col0;
      auto release = [&](int slot) {
        tc05::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (PAIRS) dense::mbar_arrive_peer(empty0 + slot * 8);
          else mbar_arrive(&b->acc_empty[slot]);
        }
      };
      if constexpr (FEATURES) {
        constexpr int NCH = EPI_COLS / 16;
        float v[NCH][16];
        for (int sg = 0; sg < segs && ok; ++sg, ++c) {
          const int slot = c & 1;
          ok = ln_wait_warp(&b->acc_full[slot], (c >> 1) & 1, b, a.status);
          if (!ok) break;
          tc05::fence_after_sync();
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
          for (int h = 0; h < NCH; ++h) ln_out_features<I8>(a, v[h], row, colb + 16 * h);
      } else {
        const float sa = I8 && row < a.M ? __ldg(a.s_a + row) : 1.0f;
        if constexpr (SEG) {
          constexpr int NCH = EPI_COLS / 16;
          float v[NCH][16];
          for (int sg = 0; sg < segs && ok; ++sg, ++c) {
            const int slot = c & 1;
            ok = ln_wait_warp(&b->acc_full[slot], (c >> 1) & 1, b, a.status);
            if (!ok) break;
            tc05::fence_after_sync();
#pragma unroll
            for (int h = 0; h < NCH; ++h) {
              float x[16];
              tc05::ld16(tmem + slot * BT + lanes + col0 + 16 * h, x);
#pragma unroll
              for (int j = 0; j < 16; ++j) v[h][j] = sg == 0 ? x[j] : __fadd_rn(v[h][j], x[j]);
            }
            release(slot);
          }
          if (ok)
#pragma unroll
            for (int h = 0; h < NCH; ++h) {
              LnRes<16> res;
              ln_load_res(a, res, row, colb + 16 * h);
              ln_out_tokens<I8>(a, v[h], row, colb + 16 * h, sa, res);
            }
        } else {
          constexpr int NCH = EPI_COLS / 32;
          LnRes<32> res, next;
          ln_load_res(a, next, row, colb);   // under way while the tile's products run
          const int slot = c & 1;
          ok = ln_wait_warp(&b->acc_full[slot], (c >> 1) & 1, b, a.status);
          if (!ok) break;
          tc05::fence_after_sync();
#pragma unroll 1
          for (int h = 0; h < NCH; ++h) {
            res = next;
            if (h + 1 < NCH) ln_load_res(a, next, row, colb + 32 * (h + 1));
            float v[32];
            __syncwarp();
            dense::tmem_ld32(tmem + slot * BT + lanes + col0 + 32 * h, v);
            if (h + 1 == NCH) release(slot);
            ln_out_tokens<I8>(a, v, row, colb + 32 * h, sa, res);
          }
          ++c;
        }
        __syncwarp();
      }
    }
  }
  __syncwarp();

  if constexpr (FEATURES && BT <= 64) {
    if (a.split > 1) {
      // one tile per cluster. The accumulators of feature f go to CTA
      // f / (128 / split), [source CTA][token][its features], through
      // distributed shared memory over the finished ring.
      const int fl = LN_ROWS / a.split;
      int ta, tb;
      ln_tile(a, first, ta, tb);
      float *xch = reinterpret_cast<float *>(sm);
      const int w = warp - LN_W_EPI, q = w & 3, half = w >> 2, f = q * 32 + lane;
      const int col0 = BT < 32 ? 0 : half * EPI_COLS;
      constexpr int NCH = EPI_COLS / 16;
      float v[NCH][16];
      bool have = false;
      if (warp >= LN_W_EPI) {
        have = true;
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
      __syncthreads();         // this CTA's products have read their ring (the MMA warp has waited for them)
      dense::cluster_sync();   // and every other CTA's
      if (have && (BT >= 32 || half == 0)) {
        float *dst = dense::peer(xch, f / fl) + rank * BT * fl + f % fl;
#pragma unroll
        for (int h = 0; h < NCH; ++h)
#pragma unroll
          for (int i = 0; i < 16; ++i) dst[(col0 + 16 * h + i) * fl] = v[h][i];
      }
      __syncwarp();
      dense::cluster_sync();
      const int m0 = tb * BT, mn = min(BT, a.M - m0), n0 = ta * LN_ROWS + rank * fl;
      for (int i = threadIdx.x; i < mn * fl; i += LN_THREADS) {
        const int m = i / fl, fi = i - m * fl, n = n0 + fi;
        if (n >= a.N) continue;
        float acc;
        if (I8) {
          int s = 0;
          for (int r = 0; r < a.split; ++r) s += __float_as_int(xch[(r * BT + m) * fl + fi]);
          acc = __int_as_float(s);
        } else {
          acc = 0.0f;
          for (int r = 0; r < a.split; ++r) acc = __fadd_rn(acc, xch[(r * BT + m) * fl + fi]);
        }
        ln_finish<I8>(a, acc, m0 + m, n, I8 ? __ldg(a.s_w + n) : 1.0f, a.bias ? __ldg(a.bias + n) : 0.0f);
      }
    }
  }

  tc05::fence_before_sync();
  __syncthreads();
  if (PAIRS) dense::cluster_sync();   // neither CTA's memory is in use by the other any more
  if (warp == LN_W_MMA) {
    tc05::fence_after_sync();
    if (PAIRS) dense::tmem_dealloc_pair(tmem, ln_tmem_cols(BT));
    else tc05::tmem_dealloc(tmem, ln_tmem_cols(BT));
  }
}

// ---------------------------------------------------------------- host side --
// [rows][K] with row stride ld (elements), boxes of box_rows x 128 bytes in the
// 128-byte swizzle.
bool ln_map(CUtensorMap *m, const void *base, bool i8, int K, int rows, long long ld, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = dense::tensor_map_encoder();
  if (!enc) return false;
  const int es = i8 ? 1 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * es};
  const cuuint32_t box[2] = {(cuuint32_t)(LN_KB / es), (cuuint32_t)box_rows};
  const cuuint32_t st[2] = {1, 1};
  return enc(m, i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base),
             dims, strides, box, st, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int BT>
const void *ln_kernel(bool i8, bool f32) {
  if (i8) return (const void *)linear_kernel<MODE, BT, true, false>;
  return f32 ? (const void *)linear_kernel<MODE, BT, false, true> : (const void *)linear_kernel<MODE, BT, false, false>;
}

qmoe_status ln_launch(const void *fn, int smem, const LnArgs &a, int grid, int cluster, cudaStream_t s) {
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return QMOE_ERR_CUDA;
  LnArgs args = a;
  void *params[] = {&args};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(LN_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, params);
  note_launch();
  return cuda_status(e);
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
  if (lda * es % 16 || ldw * es % 16 || K > LN_MAX_K || lda > (1LL << 38) || ldw > (1LL << 38)) return QMOE_ERR_UNSUPPORTED;
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
  const bool vec = ldo * os % 16 == 0 && (!residual || ldr * os % 16 == 0);
  const int mode = M <= 64 || !vec ? LN_FEATURES : M > 128 && N > 128 ? LN_PAIRS : LN_TOKENS;
  const int BT = mode == LN_FEATURES ? (M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128) : mode == LN_PAIRS ? 256 : 128;
  const int rows_a = mode == LN_FEATURES ? N : M, rows_b = mode == LN_FEATURES ? M : N;
  const int tile_a = mode == LN_PAIRS ? 2 * LN_ROWS : LN_ROWS;
  g.tiles_a = (rows_a + tile_a - 1) / tile_a;
  g.tiles_b = (rows_b + BT - 1) / BT;
  const long long nt = (long long)g.tiles_a * g.tiles_b;
  if (nt > 0x1fffffffLL) return QMOE_ERR_UNSUPPORTED;
  if (mode == LN_FEATURES && BT <= 64)
    while (g.split < LN_MAX_SPLIT && nt * g.split * 2 <= sms && g.ksteps >= g.split * 4) g.split *= 2;
  if (!ln_map(&g.tm_a, mode == LN_FEATURES ? w : a, i8, K, rows_a, mode == LN_FEATURES ? ldw : lda, LN_ROWS) ||
      !ln_map(&g.tm_b, mode == LN_FEATURES ? a : w, i8, K, rows_b, mode == LN_FEATURES ? lda : ldw, ln_b_rows(mode, BT)))
    return QMOE_ERR_CUDA;
  const void *fn;
  const bool f32 = g.out_f32;
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
  const int smem = ln_smem_bytes(mode, BT);
  if ((size_t)smem > max_smem_optin()) return QMOE_ERR_UNSUPPORTED;
  if (mode == LN_PAIRS) return ln_launch(fn, smem, g, 2 * (int)(nt < sms / 2 ? nt : sms / 2), 2, (cudaStream_t)stream);
  const int grid = g.split > 1 ? (int)nt * g.split : (int)(nt < sms ? nt : sms);
  return ln_launch(fn, smem, g, grid, g.split, (cudaStream_t)stream);
}
