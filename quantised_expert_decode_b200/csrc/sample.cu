// Sampling: one token per row of logits from a given uniform number, with
// temperature, top-k, min-p and top-p. For a row with largest logit m:
//   w_i = exp((l_i - m) / temperature), 1 where l_i = m, 0 below 2^-64
//   rank: logit descending, ties to the lower index; NaN and -inf never rank
//   kept: the first top_k ranks with w >= min_p, and of those the shortest
//         prefix of ranks whose sum of w reaches top_p x their whole sum
//   token: the lowest index whose running sum of kept w (in index order)
//         exceeds u x the whole kept sum;  prob = w_token / kept sum
// The pages sample nothing; the rule is self-defined.
//
// Every filter keeps a prefix of the ranks, so the kept set is described by its
// last element: a border (value, index). It is found without sorting the row.
//
// Where the row lives: few rows are each spread over a cluster of CTAs, every
// CTA with a contiguous slice of the row in shared memory (`RES`; one read from
// HBM). Many rows are read three times, twice out of L2, by two CTAs per SM; each
// row by as many of them as there are to spare.
// Bound: for few rows the chain of its steps (some ten cluster barriers and as
// many short sums of a few hundred cycles each: 1 x 131072 with top-k, top-p and
// min-p 16.4 us, 8 x 131072 bf16 with top-p 33 us); for many the issue of some 65
// instructions per logit (256 x 131072 fp32 with top-p 136 us, 15 % of the
// measured copy rate).
//
// How the border is found:
// quick - one pass builds a histogram over 2048 value bins (counts for top-k,
//   masses for top-p) beside the row's sum of fp32 weights with its error bound;
//   the few bins that the border can lie in are gathered, sorted, and summed in
//   rank order with float64 weights (a table and a polynomial, relative error
//   below 4e-12); what lies above those bins is summed in the same precision,
//   for each stretch of 256 logits apart, packed so that whole warps form the
//   weights of kept logits only; the stretch that the token falls into is then
//   gone through element by element. Every decision is checked to be further
//   from its border than the error bound of the sums; where the fp32 sum is too
//   coarse the row's sum is formed again in float64, and where that leaves it
//   open too, or the bins do not separate the row, the row is done the exact way.
// exact - float64 exp, sums over the row confirm every bin, and a bin that holds
//   more than a list is cut again, down to equal values ordered by index.
//
// Either way sums that decide are float64 in a fixed order: the same inputs give
// the same token on every run. Within a warp's part, elements go in rounds of
// 128, four neighbours per lane.
#include <cuda_bf16.h>
#include <math_constants.h>
#include <stddef.h>

#include "dense.cuh"

namespace qmoe {
namespace {

constexpr int SP_THREADS = 512;
constexpr int SP_WARPS = SP_THREADS / 32;
constexpr int SP_BINS = 1024;                 // exact way
constexpr int SQ_BINS = 2048;                 // quick way: 11 bits of bin, 12 bits of place within it (4096 bins: 6 % slower)
constexpr int SQ_SUB = 12;
constexpr int SQ_ROUND = 256;                 // logits of a warp whose sums are kept apart: two float4 per lane
constexpr int SQ_LIST = 2048;                 // elements that the quick way gathers and sorts
constexpr double SP_EPS = 1e-11;              // bound of the quick sums' error, relative to the row's sum
constexpr int SP_LIST = 512;                  // elements ranked one by one (one per thread)
constexpr int SP_MAX_CLUSTER = 8;             // CTAs per row
constexpr long long SP_L2_BYTES = 126ll << 20;
// More CTAs on fewer logits cost more barriers than they save (8 rows of 4000: 14.0 us
// by one CTA each, 16.4 by two; of 8000: 15.2 by one, 16.4 by two, 16.9 by four).
constexpr int SP_MIN_SLICE = 4096;
constexpr int SP_MAX_SLICE = 32768;           // 128 KB of fp32 logits per CTA
constexpr int SP_MAX_V = 393216, SP_MAX_T = 1 << 27;
constexpr double SP_W_MIN = 5.421010862427522e-20;   // 2^-64
constexpr int SP_FIX = 44;                    // histogram masses in units of 2^-44
constexpr float SP_LOWEST = -3.402823466e38f;
constexpr int SP_ROUNDS = 400;                // bound of the narrowing loop; every round drops elements, most all but one bin

struct SpArgs {
  const void *logits;
  const float *temperature, *top_p, *min_p, *u;
  const int32_t *top_k;
  int32_t *token;
  float *prob;
  int32_t *status;
  long long ld;
  int T, V, slice, nc;       // nc: CTAs per row
  int seg, rounds;           // a warp's part of the slice, a multiple of 128, and its rounds
};

// What one CTA contributes to a step of the exact way.
struct SpPart {
  double above, in;          // weight above the bin, in the bin
  float min_above, max_in, min_in, max_below;
  int n_in, pad;
};

// What a CTA pushes into every CTA of its cluster.
struct SpPush {
  double a, b;
  float c;
  int bad, listed, pad;
};

struct SpShared {
  SpPart part[2];
  SpPush push[7][SP_MAX_CLUSTER];
  double warp_d[2][SP_WARPS];
  double exp2_tab[32];       // 2^(i / 32)
  float warp_f[4][SP_WARPS];
  int warp_i[SP_WARPS];
  union {
    unsigned long long mass[SP_BINS];         // exact way
    alignas(16) unsigned int bins[SQ_BINS];   // quick way: histogram, read four at a time
    double w[SQ_LIST];                        // quick way: weights of the sorted list
  };
  union {
    struct {                                  // exact way
      float list_v[SP_LIST];
      int list_i[SP_LIST];
      float sort_v[SP_LIST];
      int sort_i[SP_LIST];
    };
    unsigned long long keys[SQ_LIST];         // quick way: sq_key of gathered elements
  };
  double rounds[SP_MAX_V / SQ_ROUND];           // a warp's rounds are neighbours
  unsigned int list_n;
  int found, last;
  float border_v;
  int border_i, bad;
  double open_sum;
  float live, q_lo, q_hi;
  double log_min_p;
};

static_assert(offsetof(SpShared, bins) % 16 == 0 && alignof(SpShared) == 16, "bins are read as uint4");

// A CTA's slice of a row: in shared memory (RES) or in global memory. NaN
// stays: it passes no comparison.
template <bool BF16, bool RES>
struct SpSrc {
  const void *row;
  const float *vals;
  int n;
  bool vec;   // rows of memory start where four logits can be read at once
  __device__ __forceinline__ float at(int i) const {
    if (RES) return vals[i];
    return BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[i]) : static_cast<const float *>(row)[i];
  }
  // Four neighbours from i (a multiple of 4) within a slice whose `vec` holds.
  __device__ __forceinline__ float4 all_four(int i) const {
    if (RES) return *reinterpret_cast<const float4 *>(vals + i);
    if (!BF16) return __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(row) + i));
    const uint2 q = __ldg(reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(row) + i));
    return make_float4(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u), __uint_as_float(q.y << 16),
                       __uint_as_float(q.y & 0xffff0000u));
  }
  // The same, -inf from `end` on.
  __device__ __forceinline__ float4 four(int i, int end) const {
    if (RES) {
      if (i >= end) return make_float4(-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F);
      return all_four(i);   // -inf behind the slice
    }
    if (vec && i + 4 <= end) return all_four(i);
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = i + j < end ? at(i + j) : -CUDART_INF_F;
    return make_float4(v[0], v[1], v[2], v[3]);
  }
};

__host__ __device__ constexpr size_t sp_head_bytes() { return (sizeof(SpShared) + 15) & ~(size_t)15; }

struct SpRow {
  float max;
  double temp;
  float live;                // smallest logit with a weight (and the min-p weight)
  float bv;                  // border: kept iff l > bv, or l == bv and index <= bi
  int bi;
};

__device__ __forceinline__ double sp_weight(float l, const SpRow &r) {
  return l == r.max ? 1.0 : exp(((double)l - (double)r.max) / r.temp);
}
__device__ __forceinline__ bool sp_kept(float l, int i, const SpRow &r) {
  return l >= r.live && (l > r.bv || (l == r.bv && i <= r.bi));
}

// Order-preserving integer of a finite float, and back.
__device__ __forceinline__ float key_float(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// Smallest logit whose weight is at least `least` (0 < least <= 1): a float64
// estimate and its neighbours; where the weights are so flat that the estimate
// is further off, a search over the floats.
__device__ float sp_live(const SpRow &r, double least) {
  if (r.max == CUDART_INF_F) return r.max;
  const double e = (double)r.max + r.temp * log(least);
  float v = fminf(e < (double)SP_LOWEST ? SP_LOWEST : __double2float_rn(e), r.max);
#pragma unroll 1
  for (int i = 0; i < 3; ++i) {
    const bool enough = sp_weight(v, r) >= least;
    if (!enough) {
      v = key_float(float_key(v) + 1u);   // r.max has weight 1, so this stays below it
      continue;
    }
    if (v == SP_LOWEST) return v;
    const float d = key_float(float_key(v) - 1u);
    if (sp_weight(d, r) < least) return v;
    v = d;
  }
  unsigned lo = float_key(SP_LOWEST), hi = float_key(r.max);   // the answer lies in [lo, hi]
#pragma unroll 1
  while (lo < hi) {
    const unsigned mid = lo + (hi - lo) / 2;
    if (sp_weight(key_float(mid), r) >= least) hi = mid;
    else lo = mid + 1;
  }
  return key_float(lo);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Sum of one double per thread over the CTA, in warp order; every thread gets it.
__device__ double sp_block_sum(double v, double *buf) {
  v = warp_sum_d(v);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < SP_WARPS; ++w) s += buf[w];
  __syncthreads();
  return s;
}

// Sum over the cluster in CTA order. `par` alternates between calls.
__device__ double sp_cluster_sum(double v, SpShared *sh, const SpArgs &a, int &par) {
  const double s = sp_block_sum(v, sh->warp_d[0]);
  if (threadIdx.x == 0) sh->part[par].in = s;
  dense::cluster_sync();
  double t = 0.0;
  for (int c = 0; c < a.nc; ++c) t += dense::peer(&sh->part[par], c)->in;
  par ^= 1;
  return t;
}

// The border of the shortest prefix of ranks whose sum of weights (COUNT: of
// ones) reaches `target`, among the kept elements. Leaves r as it is when the
// kept elements do not reach it.
template <bool COUNT, typename Src>
__device__ void sp_select(const Src &src, int n, int base, SpRow &r, double target, SpShared *sh, const SpArgs &a,
                          int rank, int &par) {
  const int tid = threadIdx.x;
  float vhi = r.max, vlo = fmaxf(r.live, r.bv);
  double A = 0.0;   // exact sum above vhi
  for (int round = 0; round < SP_ROUNDS; ++round) {
    // bins of equal width from vhi down; halves keep the differences finite
    const float hh = 0.5f * vhi, width = hh - 0.5f * vlo;
    const float scale = __fdiv_rn((float)SP_BINS, width);
    auto bin_of = [&](float l) {
      const float b = __fmul_rn(hh - 0.5f * l, scale);
      return l == vhi ? 0 : min(SP_BINS - 1, (int)fminf(b, (float)SP_BINS));
    };
    for (int i = tid; i < SP_BINS; i += SP_THREADS) sh->mass[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += SP_THREADS) {
      const float l = src.at(i);
      if (l <= vhi && l >= vlo && sp_kept(l, base + i, r)) {
        const unsigned long long q =
            COUNT ? 1ull : (unsigned long long)__double2ll_rn(sp_weight(l, r) * (double)(1ull << SP_FIX));
        atomicAdd(&sh->mass[bin_of(l)], q);
      }
    }
    dense::cluster_sync();
    // every CTA adds the histograms and finds the bin: the same integers everywhere
    constexpr int PER = SP_BINS / SP_THREADS;
    unsigned long long m[PER], run = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      m[j] = 0;
      for (int c = 0; c < a.nc; ++c) m[j] += dense::peer(&sh->mass[0], c)[tid * PER + j];
      run += m[j];
    }
    unsigned long long incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if ((tid & 31) >= o) incl += x;
    }
    unsigned long long *wsum = reinterpret_cast<unsigned long long *>(sh->warp_d[1]);
    if ((tid & 31) == 31) wsum[tid >> 5] = incl;
    if (tid == 0) sh->found = SP_BINS - 1;
    __syncthreads();
    unsigned long long pre = incl - run;
    for (int w = 0; w < (tid >> 5); ++w) pre += wsum[w];
    const double need = (target - A) * (COUNT ? 1.0 : (double)(1ull << SP_FIX));
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const unsigned long long after = pre + m[j];
      if (m[j] && (double)pre < need && (double)after >= need) atomicMin(&sh->found, tid * PER + j);
      pre = after;
    }
    __syncthreads();
    const int bin = vlo == vhi ? 0 : sh->found;

    // exact sums around the bin
    double above = 0.0, in = 0.0;
    float min_above = CUDART_INF_F, max_in = -CUDART_INF_F, min_in = CUDART_INF_F, max_below = -CUDART_INF_F;
    int n_in = 0;
    for (int i = tid; i < n; i += SP_THREADS) {
      const float l = src.at(i);
      if (l <= vhi && l >= vlo && sp_kept(l, base + i, r)) {
        const int b = bin_of(l);
        const double w = COUNT ? 1.0 : sp_weight(l, r);
        if (b < bin) {
          above += w;
          min_above = fminf(min_above, l);
        } else if (b == bin) {
          in += w;
          ++n_in;
          max_in = fmaxf(max_in, l);
          min_in = fminf(min_in, l);
        } else {
          max_below = fmaxf(max_below, l);
        }
      }
    }
    above = sp_block_sum(above, sh->warp_d[0]);
    in = sp_block_sum(in, sh->warp_d[0]);
    max_in = warp_max(max_in);
    max_below = warp_max(max_below);
    min_in = -warp_max(-min_in);
    min_above = -warp_max(-min_above);
    n_in = __reduce_add_sync(0xffffffffu, n_in);
    if ((tid & 31) == 0) {
      const int w = tid >> 5;
      sh->warp_f[0][w] = max_in;
      sh->warp_f[1][w] = max_below;
      sh->warp_f[2][w] = min_in;
      sh->warp_f[3][w] = min_above;
      sh->warp_i[w] = n_in;
    }
    __syncthreads();
    if (tid == 0) {
      SpPart p;
      p.above = above;
      p.in = in;
      p.max_in = p.max_below = -CUDART_INF_F;
      p.min_in = p.min_above = CUDART_INF_F;
      p.n_in = p.pad = 0;
      for (int w = 0; w < SP_WARPS; ++w) {
        p.max_in = fmaxf(p.max_in, sh->warp_f[0][w]);
        p.max_below = fmaxf(p.max_below, sh->warp_f[1][w]);
        p.min_in = fminf(p.min_in, sh->warp_f[2][w]);
        p.min_above = fminf(p.min_above, sh->warp_f[3][w]);
        p.n_in += sh->warp_i[w];
      }
      sh->part[par] = p;
      sh->list_n = 0;
    }
    dense::cluster_sync();
    above = in = 0.0;
    n_in = 0;
    max_in = max_below = -CUDART_INF_F;
    min_in = min_above = CUDART_INF_F;
    for (int c = 0; c < a.nc; ++c) {
      const SpPart p = *dense::peer(&sh->part[par], c);
      above += p.above;
      in += p.in;
      n_in += p.n_in;
      max_in = fmaxf(max_in, p.max_in);
      max_below = fmaxf(max_below, p.max_below);
      min_in = fminf(min_in, p.min_in);
      min_above = fminf(min_above, p.min_above);
    }
    par ^= 1;
    if (A + above >= target && min_above < CUDART_INF_F) {   // the border lies above the bin
      vlo = min_above;
      continue;
    }
    A += above;
    if (A + in < target) {                                   // below it
      if (max_below == -CUDART_INF_F) return;                // the kept elements do not reach the target
      A += in;
      vhi = max_below;
      continue;
    }
    vhi = max_in;
    vlo = min_in;
    if (n_in > SP_LIST && vlo < vhi) continue;

    if (n_in <= SP_LIST) {
      // rank the bin's elements: gathered in CTA 0, sorted by counting, summed in rank order
      SpShared *s0 = dense::peer(sh, 0);
      for (int i = tid; i < n; i += SP_THREADS) {
        const float l = src.at(i);
        if (l <= vhi && l >= vlo && sp_kept(l, base + i, r)) {
          const unsigned at = atomicAdd(&s0->list_n, 1u);
          s0->list_v[at] = l;
          s0->list_i[at] = base + i;
        }
      }
      dense::cluster_sync();
      if (rank == 0) {
        if (tid < n_in) {
          const float v = sh->list_v[tid];
          const int ix = sh->list_i[tid];
          int at = 0;
          for (int j = 0; j < n_in; ++j) {
            const float o = sh->list_v[j];
            at += o > v || (o == v && sh->list_i[j] < ix);
          }
          sh->sort_v[at] = v;
          sh->sort_i[at] = ix;
        }
        __syncthreads();
        if (tid < 32) {
          double run2 = A;
          int hit = -1;
          for (int c = 0; c < n_in && hit < 0; c += 32) {
            const int j = c + tid;
            double x = j < n_in ? (COUNT ? 1.0 : sp_weight(sh->sort_v[j], r)) : 0.0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const double y = __shfl_up_sync(0xffffffffu, x, o);
              if (tid >= o) x += y;
            }
            const unsigned ok = __ballot_sync(0xffffffffu, j < n_in && run2 + x >= target);
            if (ok) hit = c + __ffs(ok) - 1;
            run2 += __shfl_sync(0xffffffffu, x, 31);
          }
          if (tid == 0) {
            if (hit < 0) hit = n_in - 1;   // rounding at the very end of the bin
            sh->border_v = sh->sort_v[hit];
            sh->border_i = sh->sort_i[hit];
          }
        }
      }
      dense::cluster_sync();
      r.bv = s0->border_v;
      r.bi = s0->border_i;
      dense::cluster_sync();
      return;
    }

    // more equal elements than the list holds: the m-th of them by index
    const double w = COUNT ? 1.0 : sp_weight(vhi, r);
    double mth = ceil((target - A) / w);
    if (mth < 1.0) mth = 1.0;
    if (mth > (double)n_in) mth = (double)n_in;
    int want = (int)mth;
    // (floating-point division may be one off either way)
    if (want > 1 && A + (double)(want - 1) * w >= target) --want;
    else if (want < n_in && A + (double)want * w < target) ++want;
    // equal elements per CTA, then per warp segment, then element by element
    const int seg = (a.slice + SP_WARPS - 1) / SP_WARPS, wid = tid >> 5, lane = tid & 31;
    const int s0i = wid * seg, s1i = min(n, s0i + seg);
    int cnt = 0;
    for (int i = s0i + lane; i < s1i; i += 32) cnt += src.at(i) == vhi && sp_kept(src.at(i), base + i, r);
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if (lane == 0) sh->warp_i[wid] = cnt;
    __syncthreads();
    if (tid == 0) {
      int t = 0;
      for (int w2 = 0; w2 < SP_WARPS; ++w2) t += sh->warp_i[w2];
      sh->part[par].n_in = t;
      sh->part[par].pad = -1;
    }
    dense::cluster_sync();
    int before = 0, owner = -1;
    for (int c = 0; c < a.nc && owner < 0; ++c) {
      const int t = dense::peer(&sh->part[par], c)->n_in;
      if (before + t >= want || c == a.nc - 1) owner = c;
      else before += t;
    }
    if (rank == owner) {
      int b2 = before;
      for (int w2 = 0; w2 < wid; ++w2) b2 += sh->warp_i[w2];
      if (b2 < want && b2 + sh->warp_i[wid] >= want) {
        for (int i0 = s0i; i0 < s1i; i0 += 32) {
          const int i = i0 + lane;
          const bool eq = i < s1i && src.at(i) == vhi && sp_kept(src.at(i), base + i, r);
          const unsigned mask = __ballot_sync(0xffffffffu, eq);
          const int c = __popc(mask);
          if (b2 + c >= want) {
            if (eq && b2 + __popc(mask & ((2u << lane) - 1u)) == want) sh->part[par].pad = base + i;
            break;
          }
          b2 += c;
        }
      }
    }
    dense::cluster_sync();
    r.bv = vhi;
    r.bi = dense::peer(&sh->part[par], owner)->pad;
    par ^= 1;
    dense::cluster_sync();
    return;
  }
  set_status(a.status, DEV_TIMEOUT);
}

// ------------------------------------------------------------------ quick way --
struct SqRow {
  float m;          // largest logit, finite
  double c, mc;     // log2(e) / temperature, and its product with m
  float cut;        // logits below have no weight
  float low;        // smallest logit with one
  float scale;      // bins: place = (m - l) * scale, in [0, 2^23) from `low` up
};

__device__ const double SQ_EXP2[32] = {   // 2^(i / 32)
    1.0, 1.0218971486541166, 1.0442737824274138, 1.0671404006768237,
    1.0905077326652577, 1.1143867425958924, 1.1387886347566916, 1.1637248587775775,
    1.189207115002721, 1.215247359980469, 1.241857812073484, 1.2690509571917332,
    1.2968395546510096, 1.3252366431597413, 1.3542555469368927, 1.383909881963832,
    1.4142135623730951, 1.4451808069770467, 1.4768261459394993, 1.5091644275934228,
    1.5422108254079407, 1.5759808451078865, 1.6104903319492543, 1.645755478153965,
    1.681792830507429, 1.718619298122478, 1.7562521603732995, 1.7947090750031072,
    1.8340080864093424, 1.8741676341103, 1.9152065613971474, 1.9571441241754002,
};

// 2^z for z = (l - m) log2(e) / temperature: z to the nearest 1/32, a table for
// that and the Taylor polynomial of degree 4 for the rest (|r| <= 1/64, so the
// next term is below (ln2 / 64)^5 / 120 = 1.3e-12).
__device__ __forceinline__ double sq_weight(float l, const SqRow &r, const double *tab) {
  const double z = fma((double)fmaxf(l, r.cut), r.c, -r.mc);
  const double magic = 211106232532992.0;   // 1.5 * 2^47: the sum's low word is z in units of 1/32
  const double t = z + magic;
  const int k = __double2loint(t);
  const double f = z - (t - magic);
  double p = fma(f, 0.009618129107628477, 0.05550410866482158);
  p = fma(f, p, 0.2402265069591007);
  p = fma(f, p, 0.6931471805599453);
  const double T = tab[k & 31];
  const double S = __hiloint2double(__double2hiint(T) + (k >> 5) * 0x100000, __double2loint(T));
  const double w = fma(S, f * p, S);
  return l >= r.cut ? w : 0.0;
}

// The same in fp32 and y = -z: the hardware exponential (2^-22 relative) of a
// product with three roundings, one of them that of c (c32).
__device__ __forceinline__ float sq_exp2(float z) {
  float w;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(z));
  return w;
}
__device__ __forceinline__ float sq_fast(float l, float c32, const SqRow &r, float &y) {
  y = fminf(__fmul_rn(__fsub_rn(r.m, l), c32), 64.0f);
  return sq_exp2(-y);
}

// Place of a logit >= low among the bins: 11 bits of bin, 12 bits inside it.
// Grows monotonically as the logit falls (two roundings of monotone operations).
// As a float it is 2^23 + place, exactly: the low 23 bits hold the place.
__device__ __forceinline__ float sq_place(float l, const SqRow &r) {
  return __fmaf_rn(__fsub_rn(r.m, l), r.scale, 8388608.0f);
}
__device__ __forceinline__ unsigned sq_bin(float place) { return (__float_as_uint(place) & 0x7fffffu) >> SQ_SUB; }
// The place where bin b begins (b up to SQ_BINS).
__device__ __forceinline__ float sq_bin_at(unsigned b) { return 8388608.0f + (float)(1 << SQ_SUB) * (float)b; }

// The smallest logit whose place is below `at` (+inf where there is none): a
// guess and its neighbours, else a search by 32 parts. Whole warps; every lane gets it.
__device__ __forceinline__ float sq_logit_at(float at, const SqRow &r) {
  if (!(sq_place(r.m, r) < at)) return CUDART_INF_F;
  const unsigned lane = threadIdx.x & 31, top = float_key(r.m), bottom = float_key(SP_LOWEST);
  const float guess = fminf(fmaxf(__fsub_rn(r.m, __fdiv_rn(__fsub_rn(at, 8388608.0f), r.scale)), SP_LOWEST), r.m);
  unsigned lo = bottom, hi = top;   // the answer's key lies in [lo, hi]
  unsigned k = min(max(float_key(guess), bottom + 16u) - 16u + lane, top);
  unsigned below = __ballot_sync(0xffffffffu, sq_place(key_float(k), r) < at);   // (grows with the lane)
  if (below != 0u && below != 0xffffffffu) return key_float(__shfl_sync(0xffffffffu, k, __ffs(below) - 1));
  for (int step = 0; step < 12 && lo < hi; ++step) {   // (7 or 8: 2^32 keys)
    const unsigned part = (hi - lo) / 32u + 1u;
    k = min(lo + lane * part, hi);
    below = __ballot_sync(0xffffffffu, sq_place(key_float(k), r) < at);
    const int f = below ? __ffs(below) - 1 : 32;   // the first part that begins with the answer or behind it
    const unsigned from = f ? min(lo + (unsigned)(f - 1) * part, hi) + 1u : lo;
    hi = f < 32 ? min(lo + (unsigned)f * part, hi) : hi;
    lo = f ? from : hi;
  }
  return key_float(hi);
}

// Adds v to a histogram's counter where l >= hi (no branch around it).
__device__ __forceinline__ void sq_count(uint32_t at, unsigned v, float l, float hi) {
  asm volatile("{\n .reg .pred p;\n setp.ge.f32 p, %2, %3;\n @p red.shared.add.u32 [%0], %1;\n}" ::"r"(at), "r"(v), "f"(l), "f"(hi)
               : "memory");
}
// Stores l where l >= hi, and moves on then.
__device__ __forceinline__ void sq_stack(uint32_t &at, float l, float hi) {
  asm volatile("{\n .reg .pred p;\n setp.ge.f32 p, %1, %2;\n @p st.shared.f32 [%0], %1;\n @p add.u32 %0, %0, 4;\n}"
               : "+r"(at) : "f"(l), "f"(hi) : "memory");
}

// By one whole warp with the same v in all lanes: a lane per CTA.
template <typename T>
__device__ __forceinline__ void push_all(T *at, const T &v, int nc) {
  const int lane = threadIdx.x & 31;
  if (lane < nc) *dense::peer(at, lane) = v;
}

// Ascending keys are ascending ranks: logit descending, then index. (-0 + 0 is 0: zeros
// of either sign are one logit.)
__device__ __forceinline__ unsigned long long sq_key(float l, int i) {
  return ((unsigned long long)~float_key(__fadd_rn(l, 0.0f)) << 32) | (unsigned)i;
}
__device__ __forceinline__ float sq_key_logit(unsigned long long k) { return key_float(~(unsigned)(k >> 32)); }

// Sorts the n keys, ascending (all threads of the CTA; a bitonic network, a pair
// per thread and turn).
__device__ void sq_sort(SpShared *sh, int n) {
  const int tid = threadIdx.x;
  int size = 2;
  while (size < n) size *= 2;
  for (int i = n + tid; i < size; i += SP_THREADS) sh->keys[i] = ~0ull;
  __syncthreads();
  for (int k = 2; k <= size; k *= 2)
    for (int j = k / 2; j > 0; j /= 2) {
      for (int p = tid; p < size / 2; p += SP_THREADS) {
        const int a = 2 * p - (p & (j - 1)), b = a + j;
        const unsigned long long x = sh->keys[a], y = sh->keys[b];
        if ((x > y) == ((a & k) == 0)) {
          sh->keys[a] = y;
          sh->keys[b] = x;
        }
      }
      if (j > 32) __syncthreads();
      else __syncwarp();   // up to there a warp's pairs stay within its own 64 keys (of each turn)
      if (j == 1) __syncthreads();
    }
}

// The gathered keys in rank order, and their weights.
__device__ void sq_rank(SpShared *sh, int n, const SqRow &r) {
  sq_sort(sh, n);
  for (int i = threadIdx.x; i < n; i += SP_THREADS) sh->w[i] = sq_weight(sq_key_logit(sh->keys[i]), r, sh->exp2_tab);
  __syncthreads();
}

// The element of a list of n weights where the running sum (from A) first
// reaches `target`: its place, or -1; `sure` is false where a running sum on
// either side of it is within eps of the target. One warp.
template <typename W>
__device__ int sq_cross(W weight, int n, double A, double target, double eps, bool &sure) {
  const int lane = threadIdx.x & 31;
  double run = A;
  for (int c = 0; c < n; c += 32) {
    const int j = c + lane;
    double x = j < n ? weight(j) : 0.0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const double after = run + x;
    const unsigned ok = __ballot_sync(0xffffffffu, j < n && after >= target);
    if (ok) {
      const int h = __ffs(ok) - 1;
      const double up = __shfl_sync(0xffffffffu, after, h), prev = __shfl_sync(0xffffffffu, after, h > 0 ? h - 1 : 0);
      const double below = h > 0 ? prev : run;
      sure = up - target > eps && target - below > eps;
      return c + h;
    }
    run += __shfl_sync(0xffffffffu, x, 31);
  }
  sure = false;
  return -1;
}

// Running sums over the warps of a CTA, in warp order, of a value per warp that
// lanes 0 bring: the sum before warp w in lane w, the whole sum in every lane.
// Between two uses of one buf lies a CTA barrier.
__device__ __forceinline__ void sq_cta_scan(double v, double *buf, double &before, double &whole) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  const double own = lane < SP_WARPS ? buf[lane] : 0.0;
  double x = own;
#pragma unroll
  for (int o = 1; o < SP_WARPS; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  before = x - own;
  whole = __shfl_sync(0xffffffffu, x, SP_WARPS - 1);
}

__device__ __forceinline__ double sq_cta_sum(double v, double *buf) {
  double before, whole;
  sq_cta_scan(v, buf, before, whole);
  return whole;
}

// f(i, l): a warp's part of a row in rounds of 256, i the place of the round in
// the part. Lane's elements: l[0..3] at i + 4 lane, l[4..7] at i + 128 + 4 lane;
// -inf behind the part. The next round's loads are under way meanwhile.
template <bool BF16, bool RES, typename F>
__device__ __forceinline__ void sq_each(const SpSrc<BF16, RES> &src, int s0, int own, F f) {
  const int at = s0 + 4 * (threadIdx.x & 31), end = s0 + own, easy = RES || src.vec ? own - SQ_ROUND : -1;
  float4 a, b;
  auto fetch = [&](int i) {
    if (i <= easy) {   // (a whole round)
      a = src.all_four(at + i);
      b = src.all_four(at + i + 128);
    } else {
      a = src.four(at + i, end);
      b = src.four(at + i + 128, end);
    }
  };
  fetch(0);
#pragma unroll 1
  for (int i = 0; i < own; i += SQ_ROUND) {
    const float l[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    fetch(i + SQ_ROUND);
    f(i, l);
  }
}

// The lane's elements (as sq_each gives them) whose bits are set, to the CTA's list.
template <typename Src>
__device__ __forceinline__ void sq_gather(const Src &src, SpShared *sh, int i, unsigned bits, int base) {
  for (; bits; bits &= bits - 1) {
    const int j = __ffs(bits) - 1, e = i + 4 * (threadIdx.x & 31) + (j & 3) + 32 * (j & 4);
    const unsigned k = atomicAdd(&sh->list_n, 1u);
    if (k < SQ_LIST) sh->keys[k] = sq_key(src.at(e), base + e);
  }
}

// CTA 0 fetches what the others have listed behind its own list (their counts came
// with `push`, before the last cluster barrier), unless it is too much. All threads; the
// count of all CTAs' elements. (Listing straight into CTA 0's memory, a remote atomic
// per element, held up its rounds, and read by CTA 0 alone it needs no barrier.)
__device__ int sq_collect(SpShared *sh, const SpPush *push, const SpArgs &a, int rank) {
  int all = 0;
  for (int c = 0; c < a.nc; ++c) all += push[c].listed;
  if (rank == 0 && all <= SQ_LIST) {
    int from = push[0].listed;
    for (int c = 1; c < a.nc; ++c) {
      const SpShared *o = dense::peer(sh, c);
      for (int i = threadIdx.x; i < push[c].listed; i += SP_THREADS) sh->keys[from + i] = o->keys[i];
      from += push[c].listed;
    }
    __syncthreads();
  }
  return all;
}

// Top-k: everything down to rank k's bin goes to CTA 0, which finishes the row.
template <bool BF16, bool RES>
__device__ bool sq_finish_k(const SpSrc<BF16, RES> &src, int s0, int own, int base, float from, int top_k, float top_p, float u,
                            const SqRow &r, SpShared *sh, const SpArgs &a, int t, int rank) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  sq_each(src, s0, own, [&](int i, const float(&l)[8]) {
    unsigned in = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) in |= l[j] >= from ? 1u << j : 0u;
    sq_gather(src, sh, s0 + i, in, base);
  });
  __syncthreads();
  if (wid == 0) push_all(&sh->push[1][rank], SpPush{0.0, 0.0, 0.0f, 0, (int)sh->list_n, 0}, a.nc);
  dense::cluster_sync();
  int kept = sq_collect(sh, sh->push[1], a, rank);
  if (rank == 0) {
    bool good = kept <= SQ_LIST;
    if (good) {
      sq_rank(sh, kept, r);
      kept = min(kept, top_k);
      if (tid < 32) {
        double tot = 0.0;
        for (int j = lane; j < kept; j += 32) tot += sh->w[j];
        tot = warp_sum_d(tot);
        if (top_p < 1.0f) {
          const double need = (double)fmaxf(top_p, 0.0f) * tot;
          int h = 0;
          if (need > 0.0) {
            bool sure = true;
            h = sq_cross([&](int j) { return sh->w[j]; }, kept, 0.0, need, SP_EPS * tot, sure);
            good = sure && h >= 0;
          }
          kept = h + 1;
          tot = 0.0;
          for (int j = lane; j < kept; j += 32) tot += sh->w[j];
          tot = warp_sum_d(tot);
        }
        if (lane == 0) {
          sh->warp_d[0][0] = tot;
          sh->warp_i[0] = good ? kept : 0;
        }
      }
      __syncthreads();
      kept = sh->warp_i[0];
      // by index: the kept elements as (index, rank)
      constexpr int EACH = SQ_LIST / SP_THREADS;
      unsigned long long mine[EACH];
#pragma unroll
      for (int c = 0; c < EACH; ++c) {
        const int j = c * SP_THREADS + tid;
        mine[c] = j < kept ? (sh->keys[j] << 32) | (unsigned)j : ~0ull;
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < EACH; ++c) sh->keys[c * SP_THREADS + tid] = mine[c];
      sq_sort(sh, kept);
      if (tid < 32) {
        const double tot = sh->warp_d[0][0];
        bool sure = true;
        const int h = sq_cross([&](int j) { return sh->w[(unsigned)sh->keys[j]]; }, kept, 0.0, (double)u * tot, SP_EPS * tot, sure);
        good = sure && h >= 0;
        if (good && lane == 0) {
          a.token[t] = (int)(sh->keys[h] >> 32);
          if (a.prob) a.prob[t] = (float)(sh->w[(unsigned)sh->keys[h]] / tot);
        }
      }
    }
    if (wid == 0) push_all(&sh->push[4][0], SpPush{0.0, 0.0, 0.0f, good ? 0 : 1}, a.nc);
  }
  dense::cluster_sync();
  return sh->push[4][0].bad == 0;
}

// Samples the row by the quick way. Returns false (in every thread of the
// cluster) where it cannot be sure. Its last step is a cluster barrier.
template <bool BF16, bool RES>
__device__ bool sq_row(const SpSrc<BF16, RES> &src, float *stack, int base, float m, float lmin, float temp,
                       int top_k, float top_p, float min_p, float u, SpShared *sh, const SpArgs &a, int t, int rank) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, n = src.n;
  SqRow r;
  r.m = m;
  r.c = 1.4426950408889634 / (double)temp;
  r.mc = (double)m * r.c;
  const bool k_on = top_k > 0 && top_k < a.V, p_on = top_p < 1.0f, mp_on = min_p > 0.0f;
  // weights below 2^-63.9 are left out (their sum stays far below SP_EPS)
  const double cut = (double)m - 44.29 * (double)temp;
  r.cut = cut > (double)SP_LOWEST ? __double2float_ru(cut) : SP_LOWEST;
  // top-p: what lies below `tail` weighs less than 1 - top_p in all, and the row's sum is
  // at least 1, so the border is above and the bins need not reach further
  const float few = fmaxf(1.0f - fmaxf(top_p, 0.0f), 5e-8f);
  const double tail = k_on || !p_on ? (double)r.cut : (double)m - (double)temp * 0.6932 * (double)(__log2f((float)a.V / few) + 0.01f);
  const float low = fmaxf(fmaxf(lmin, r.cut), tail > (double)SP_LOWEST ? __double2float_rd(tail) : SP_LOWEST);
  const float range = __fsub_rn(m, low);
  r.scale = __fdiv_rn(8380000.0f, range);   // a little below 2^23 / range
  if (!(range > 0.0f && r.scale < 1e30f && r.scale > 1e-30f && r.c < 1e30 && r.c > 1e-30)) return false;
  // min-p: kept from `hi` up, undecided from `lo` up
  if (mp_on && tid == 0) {
    const double at = (double)m + (double)temp * sh->log_min_p, d = 1e-10 * (double)temp + 1e-14 * fabs(at);
    sh->q_hi = __double2float_ru(at + d);
    sh->q_lo = __double2float_ru(at - d);
  }
  if (k_on || p_on)
    for (int i = tid; i < SQ_BINS; i += SP_THREADS) sh->bins[i] = 0;
  __syncthreads();
  float lo = r.cut, hi = r.cut;
  if (mp_on) {
    lo = fmaxf(lo, sh->q_lo);
    hi = fminf(fmaxf(hi, sh->q_hi), m);   // the largest logit is always kept
  }
  const float counted = fmaxf(hi, low);                 // these have a bin
  const int s0 = wid * a.seg;                           // this warp's part, in index order
  const int own = max(0, min(n, s0 + a.seg) - s0);      // elements of it
  int bad = 0;

  const float c32 = (float)r.c;
  unsigned first = SQ_BINS, last = SQ_BINS - 1;   // the border lies in these bins
  double S = 0.0, SY = 0.0;   // the row's sum of fp32 weights, and of weights times y
  if (k_on || p_on) {
    const float per_bin = (float)(r.c * (double)(1 << SQ_SUB) / (double)r.scale);   // log2 of the weights' fall over a bin
    // a mass is 32768 at its bin's top, less by the weights' fall towards the bin's end
    const unsigned slope = (unsigned)(32768.0f * (1.0f - exp2f(-per_bin)));
    const uint32_t bins = (uint32_t)__cvta_generic_to_shared(&sh->bins[0]);
    double s = 0.0;
    float sy = 0.0f;
    sq_each(src, s0, own, [&](int, const float(&l)[8]) {
      if (mp_on)
#pragma unroll
        for (int j = 0; j < 8; ++j) bad |= l[j] >= lo && l[j] < hi;
      if (k_on) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          sq_count(bins + 4 * sq_bin(sq_place(l[j], r)), 1u, l[j], counted);
        return;
      }
      // the sum of fp32 weights beside the histogram, two at a time in fp32 (what is
      // left out has a weight of 2^-64 here: too small to count)
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        float w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float d = __fsub_rn(r.m, l[j + k]), y = l[j + k] >= hi ? __fmul_rn(d, c32) : 64.0f;
          w[k] = sq_exp2(-y);
          sy = __fmaf_rn(w[k], y, sy);
          const unsigned at = __float_as_uint(__fmaf_rn(d, r.scale, 8388608.0f));
          sq_count(bins + (at >> (SQ_SUB - 2) & 4u * (SQ_BINS - 1)),
                   ((32768u << SQ_SUB) - (at & ((1u << SQ_SUB) - 1u)) * slope) >> SQ_SUB, l[j + k], counted);
        }
        s += (double)(w[0] + w[1]);
      }
    });
    bad = __syncthreads_or(bad);
    if (!k_on) {
      s = sq_cta_sum(warp_sum_d(s), sh->warp_d[0]);
      sy = (float)sq_cta_sum((double)warp_sum(sy), sh->warp_d[1]);
    }
    if (wid == 0) push_all(&sh->push[0][rank], SpPush{s, (double)sy, 0.0f, bad}, a.nc);
    if (tid == 0) {
      sh->found = sh->last = SQ_BINS;
      sh->list_n = 0;
    }
    dense::cluster_sync();
#pragma unroll 1
    for (int c = 0; c < a.nc; ++c) {
      S += sh->push[0][c].a;
      SY += sh->push[0][c].b;
      bad |= sh->push[0][c].bad;
    }
    if (bad) return false;
    // every CTA adds its share of the bins over the cluster (PER neighbouring
    // bins per thread), then the shares' sums go round
    constexpr int PER = SQ_BINS / SP_THREADS;
    static_assert(PER % 4 == 0, "whole uint4 of bins per thread");
    const int share = SP_THREADS / a.nc;   // threads with bins; nc is a power of two
    const int b0 = PER * (rank * share + tid);
    unsigned long long hh[PER] = {};
    if (tid < share) {
#pragma unroll
      for (int q = 0; q < PER; q += 4) {
        uint4 x[SP_MAX_CLUSTER];
#pragma unroll
        for (int c = 0; c < SP_MAX_CLUSTER; ++c)   // all loads in flight together
          if (c < a.nc) x[c] = reinterpret_cast<const uint4 *>(dense::peer(&sh->bins[0], c))[(b0 + q) / 4];
#pragma unroll
        for (int c = 0; c < SP_MAX_CLUSTER; ++c)
          if (c < a.nc) {
            hh[q] += x[c].x;
            hh[q + 1] += x[c].y;
            hh[q + 2] += x[c].z;
            hh[q + 3] += x[c].w;
          }
      }
    }
    double f[PER], run = 0.0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      f[j] = (double)hh[j];
      if (!k_on) f[j] *= (double)exp2f(-per_bin * (float)(b0 + j));
      run += f[j];
    }
    double incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    double before, all;
    __syncthreads();
    sq_cta_scan(__shfl_sync(0xffffffffu, incl, 31), sh->warp_d[1], before, all);
    double pre = __shfl_sync(0xffffffffu, before, wid) + incl - run;
    if (a.nc > 1) {
      if (wid == 0) push_all(&sh->push[5][rank], SpPush{all, 0.0, 0.0f, 0}, a.nc);
      dense::cluster_sync();
      all = 0.0;
#pragma unroll 1
      for (int c = 0; c < a.nc; ++c) {
        if (c < rank) pre += sh->push[5][c].a;
        all += sh->push[5][c].a;
      }
    }
    if (!k_on) all = 32768.0 * S;   // (what lies below the bins too)
    // top-k: the bin of rank k. top-p: the bins that the histogram's masses,
    // good to 1.3e-4, leave open.
    const double want = k_on ? fmin((double)top_k, all) : (double)fmaxf(top_p, 0.0f) * all;
    const double early = k_on ? want : want * (1.0 - 3e-4), late = k_on ? want : want * (1.0 + 3e-4);
    int at_first = SQ_BINS, at_last = SQ_BINS;
    double upto = pre;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      upto += f[j];
      if (hh[j] && upto >= early) at_first = min(at_first, b0 + j);
      if (hh[j] && upto >= late) at_last = min(at_last, b0 + j);
    }
    at_first = __reduce_min_sync(0xffffffffu, at_first);
    at_last = __reduce_min_sync(0xffffffffu, at_last);
    if (lane < a.nc) {
      if (at_first < SQ_BINS) atomicMin(&dense::peer(sh, lane)->found, at_first);
      if (at_last < SQ_BINS) atomicMin(&dense::peer(sh, lane)->last, at_last);
    }
    dense::cluster_sync();
    first = (unsigned)sh->found;
    last = (unsigned)min(sh->last, SQ_BINS - 1);
    if (first >= SQ_BINS) return false;
  }
  // logits from `above` up lie above the open bins, from `from` up in them
  float above = hi, from = lo;
  if (k_on || p_on) {
    above = fmaxf(hi, sq_logit_at(sq_bin_at(first), r));
    from = fmaxf(hi, sq_logit_at(sq_bin_at(last + 1), r));
  }
  if (k_on) return sq_finish_k(src, s0, own, base, from, top_k, top_p, u, r, sh, a, t, rank);

  // The sum above the open bins, for each of the warp's rounds; the open bins'
  // elements to CTA 0. What is kept of a round is stacked, lane behind lane.
  const float *mine = stack + wid * SQ_ROUND;
  const uint32_t mine_at = (uint32_t)__cvta_generic_to_shared(mine);
  double ws = 0.0, a_fast = 0.0;   // exact weights; fp32 weights of the same
  float a_sy = 0.0f;
  sq_each(src, s0, own, [&](int i, const float(&l)[8]) {
    int held = 0;   // of this lane
    float rest = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = l[j] >= above;
      held += in ? 1 : 0;
      rest = fmaxf(rest, in ? -CUDART_INF_F : l[j]);
    }
    if (rest >= from) {
      bad |= !p_on;   // min-p alone leaves nothing open
      unsigned opens = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) opens |= l[j] >= from && l[j] < above ? 1u << j : 0u;
      if (p_on) sq_gather(src, sh, s0 + i, opens, base);
    }
    int upto = held;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      upto += lane >= o ? y : 0;
    }
    const int all = __shfl_sync(0xffffffffu, upto, 31);
    uint32_t at = mine_at + 4 * (upto - held);
#pragma unroll
    for (int j = 0; j < 8; ++j) sq_stack(at, l[j], above);
    __syncwarp();
    double x = 0.0;
#pragma unroll 1
    for (int k = lane; k - lane < all; k += 32) {
      const float v = k < all ? mine[k] : -CUDART_INF_F;
      x += sq_weight(v, r, sh->exp2_tab);
      float y;
      const float w = sq_fast(v, c32, r, y);   // (2^-64 where there is none)
      a_fast += (double)w;
      a_sy = __fmaf_rn(w, y, a_sy);
    }
    __syncwarp();
    x = all ? warp_sum_d(x) : 0.0;
    if (lane == 0) sh->rounds[wid * a.rounds + i / SQ_ROUND] = x;
    ws += x;
  });
  bad = __syncthreads_or(bad);
  double warps_before, sum;
  sq_cta_scan(ws, sh->warp_d[0], warps_before, sum);
  if (p_on) {
    a_fast = sq_cta_sum(warp_sum_d(a_fast), sh->warp_d[1]);
    __syncthreads();
    a_sy = (float)sq_cta_sum((double)warp_sum(a_sy), sh->warp_d[1]);
  }
  if (wid == 0) push_all(&sh->push[1][rank], SpPush{sum, a_fast, a_sy, bad, (int)sh->list_n, 0}, a.nc);
  dense::cluster_sync();
  double total = 0.0;
#pragma unroll 1
  for (int c = 0; c < a.nc; ++c) {
    total += sh->push[1][c].a;
    S -= sh->push[1][c].b;       // what is left is below the border's bins, or in them
    SY -= sh->push[1][c].c;
    bad |= sh->push[1][c].bad;
  }
  if (bad) return false;

  float bv = hi;
  int bi = a.V;
  if (p_on) {
    const double p = (double)fmaxf(top_p, 0.0f);
    const SpShared *lists = dense::peer(sh, 0);
    const int listed = sq_collect(sh, sh->push[1], a, rank);
    if (listed > SQ_LIST) return false;
    // The row's sum: exact weights down to the open bins, fp32 weights below
    // them, freed of what c's fp32 value is off by (y times that, relatively). Its
    // error: two roundings of y (9e-8 of it) and 2.4e-7 of each weight below, and
    // the roundings of two weights added in fp32 of the whole first sum.
    double whole = total + S, err = 0.0;
    if (rank == 0) {
      sq_rank(sh, listed, r);
      double open_fast = 0.0, open_sum = 0.0;
      float open_sy = 0.0f;
      for (int j = tid; j < listed; j += SP_THREADS) {
        float y;
        const float v = sq_fast(sq_key_logit(sh->keys[j]), c32, r, y);
        open_fast += (double)v;
        open_sum += sh->w[j];
        open_sy += v * y;
      }
      open_fast = sq_cta_sum(warp_sum_d(open_fast), sh->warp_d[0]);
      open_sum = sq_cta_sum(warp_sum_d(open_sum), sh->warp_d[1]);
      __syncthreads();
      open_sy = (float)sq_cta_sum((double)warp_sum(open_sy), sh->warp_d[0]);
      S -= open_fast;
      SY -= (double)open_sy;
      S += 0.6931471805599453 * ((double)c32 - r.c) / r.c * SY;
      whole = total + open_sum + S;
      err = p * (9e-8 * fmax(SY, 0.0) + 2.6e-7 * fmax(S, 0.0) + 8e-8 * whole);
    }
    for (int round = 0; round < 2; ++round) {   // (uniform over the cluster)
      if (rank == 0 && tid < 32) {
        bool sure = true;
        int h = 0;
        if (p > 0.0) h = sq_cross([&](int j) { return sh->w[j]; }, listed, total, p * whole, err, sure);
        const int good = sure && h >= 0;
        double x = 0.0;   // the open bins' kept weights
        for (int j = lane; j <= h; j += 32) x += sh->w[j];
        x = warp_sum_d(x);
        if (lane < a.nc) {
          SpShared *o = dense::peer(sh, lane);
          o->border_v = good ? sq_key_logit(sh->keys[h]) : 0.0f;
          o->border_i = good ? (int)(unsigned)sh->keys[h] : 0;
          o->found = h;
          o->open_sum = x;
          o->bad = !good;
        }
      }
      dense::cluster_sync();
      if (!sh->bad) break;
      if (round == 1) return false;
      // the fp32 sum leaves it open: the row's sum again, in float64
      double s = 0.0;
#pragma unroll 4
      for (int i = lane; i < own; i += 32) {
        const float l = src.at(s0 + i);
        s += sq_weight(l >= hi ? l : -CUDART_INF_F, r, sh->exp2_tab);
      }
      s = sq_cta_sum(warp_sum_d(s), sh->warp_d[1]);
      if (wid == 0) push_all(&sh->push[2][rank], SpPush{s, 0.0, 0.0f, 0}, a.nc);
      dense::cluster_sync();
      whole = 0.0;
#pragma unroll 1
      for (int c = 0; c < a.nc; ++c) whole += sh->push[2][c].a;
      err = SP_EPS * whole;
    }
    bv = sh->border_v;
    bi = sh->border_i;
    total += sh->open_sum;
    // the open bins' kept weights to the rounds that they lie in (what these
    // sums decide is checked against SP_EPS, so their order does not matter)
    for (int j = tid; j <= sh->found; j += SP_THREADS) {
      const int i = (int)(unsigned)lists->keys[j] - base;
      if (i >= 0 && i < n) atomicAdd(&sh->rounds[i / a.seg * a.rounds + i % a.seg / SQ_ROUND], lists->w[j]);
    }
    __syncthreads();
    ws = 0.0;
    for (int i = lane; i * SQ_ROUND < own; i += 32) ws += sh->rounds[wid * a.rounds + i];
    ws = warp_sum_d(ws);
    sq_cta_scan(ws, sh->warp_d[1], warps_before, sum);
    if (wid == 0) push_all(&sh->push[3][rank], SpPush{sum, 0.0, 0.0f, 0}, a.nc);
    dense::cluster_sync();
  }

  // the token, by index: the CTA, the warp, the round, the lane's elements, the element
  const SpPush *sums = p_on ? sh->push[3] : sh->push[1];
  const double aim = (double)u * total, eps = SP_EPS * total;
  double before = 0.0;
  int owner = -1;
#pragma unroll 1
  for (int c = 0; c < a.nc && owner < 0; ++c) {
    const double x = sums[c].a;
    if (before + x > aim) owner = c;
    else before += x;
  }
  if (owner < 0) return false;
  if (rank == owner) {
    // the last warp that begins at or below the target (the first begins at `before`)
    const unsigned starts = __ballot_sync(0xffffffffu, lane < SP_WARPS && before + warps_before <= aim);
    if (wid == (starts ? 31 - __clz(starts) : 0)) {
      auto scan = [&](double v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += y;
        }
        return v;
      };
      auto weight_at = [&](int i) -> double {
        const float l = i < own ? src.at(s0 + i) : -CUDART_INF_F;
        const bool in = l >= hi && (l > bv || (l == bv && base + s0 + i <= bi));
        return sq_weight(in ? l : -CUDART_INF_F, r, sh->exp2_tab);
      };
      double b2 = before + __shfl_sync(0xffffffffu, warps_before, wid);
      // the round: the first whose end passes the target, else the last
      int i0 = 0;
      for (int k = 0; k < own; k += 32 * SQ_ROUND) {
        const int i = k + lane * SQ_ROUND;
        const double own_r = i < own ? sh->rounds[wid * a.rounds + i / SQ_ROUND] : 0.0, z = scan(own_r);
        const unsigned pass = __ballot_sync(0xffffffffu, own_r > 0.0 && b2 + z > aim);
        if (pass) {
          const int c = __ffs(pass) - 1;
          i0 = k + c * SQ_ROUND;
          b2 += __shfl_sync(0xffffffffu, z, c) - __shfl_sync(0xffffffffu, own_r, c);
          break;
        }
        b2 += __shfl_sync(0xffffffffu, z, 31);
      }
      // its eight elements per lane, from another one in each lane: no bank twice
      constexpr int EACH = SQ_ROUND / 32;
      double x = 0.0;
#pragma unroll 1
      for (int j = 0; j < EACH; ++j) x += weight_at(i0 + EACH * lane + ((j + lane) & (EACH - 1)));
      const double own_x = x;
      x = scan(x);
      const unsigned pass = __ballot_sync(0xffffffffu, own_x > 0.0 && b2 + x > aim);
      int hit = -1;
      double w_hit = 0.0;
      bool sure = false;
      if (pass) {   // (else the target is within rounding of the round's end: not sure)
        const int c = __ffs(pass) - 1;
        const double b3 = b2 + __shfl_sync(0xffffffffu, x, c) - __shfl_sync(0xffffffffu, own_x, c);
        const double w = lane < EACH ? weight_at(i0 + EACH * c + lane) : 0.0, z = scan(w);
        const unsigned over = __ballot_sync(0xffffffffu, w > 0.0 && b3 + z > aim);
        if (over) {
          const int h = __ffs(over) - 1;
          hit = i0 + EACH * c + h;
          const double after = b3 + __shfl_sync(0xffffffffu, z, h);
          w_hit = __shfl_sync(0xffffffffu, w, h);
          // both ends of the token's interval are clear of the target
          sure = after - aim > eps && aim - (after - w_hit) > eps;
        }
      }
      const bool good = hit >= 0 && sure;
      if (good && lane == 0) {
        a.token[t] = base + s0 + hit;
        if (a.prob) a.prob[t] = (float)(w_hit / total);
      }
      push_all(&sh->push[4][0], SpPush{0.0, 0.0, 0.0f, good ? 0 : 1}, a.nc);
    }
  }
  dense::cluster_sync();
  return sh->push[4][0].bad == 0;
}

// The thread's largest and smallest logit of a slice, which goes into shared
// memory on the way (RES), -inf behind its end.
template <bool BF16, bool RES>
__device__ void sp_load(const SpSrc<BF16, RES> &src, float *vals, int padded, float &mx, float &mn) {
  const int tid = threadIdx.x;
  mx = -CUDART_INF_F;
  mn = CUDART_INF_F;
  const SpSrc<BF16, false> mem{src.row, nullptr, src.n, src.vec};
  constexpr int U = 8;
  const int full = src.n / 4 * 4;
  for (int i0 = 0; i0 < full; i0 += 4 * U * SP_THREADS) {
    float4 q[U];
    const int at = i0 + 4 * tid;
    if (src.vec && i0 + 4 * U * SP_THREADS <= full) {
#pragma unroll
      for (int c = 0; c < U; ++c) q[c] = mem.all_four(at + 4 * c * SP_THREADS);
    } else {
#pragma unroll
      for (int c = 0; c < U; ++c) q[c] = mem.four(at + 4 * c * SP_THREADS, full);
    }
#pragma unroll
    for (int c = 0; c < U; ++c) {
      const int i = at + 4 * c * SP_THREADS;
      mx = fmaxf(fmaxf(mx, fmaxf(q[c].x, q[c].y)), fmaxf(q[c].z, q[c].w));
      if (i < full) {
        mn = fminf(fminf(mn, fminf(q[c].x, q[c].y)), fminf(q[c].z, q[c].w));
        if (RES) *reinterpret_cast<float4 *>(vals + i) = q[c];
      }
    }
  }
  for (int i = full + tid; i < src.n; i += SP_THREADS) {
    const float v = mem.at(i);
    mx = fmaxf(mx, v);
    mn = fminf(mn, v);
    if (RES) vals[i] = v;
  }
  if (RES)
    for (int i = src.n + tid; i < padded; i += SP_THREADS) vals[i] = -CUDART_INF_F;
}

template <bool BF16, bool RES>
__global__ void __launch_bounds__(SP_THREADS, RES ? 1 : 2) sample_kernel(SpArgs a) {
  extern __shared__ __align__(16) uint8_t sp_smem[];
  SpShared *sh = reinterpret_cast<SpShared *>(sp_smem);
  float *stack = reinterpret_cast<float *>(sp_smem + sp_head_bytes());   // a round's logits per warp
  float *vals = stack + SP_WARPS * SQ_ROUND;                             // RES: the slice
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int rank = (int)dense::cluster_rank(), t = blockIdx.x / a.nc;
  const int base = min(a.V, rank * a.slice), n = min(a.V, base + a.slice) - base;

  dense::cluster_arrive();   // (waited for before the first store into another CTA)
  pdl_wait();
  pdl_launch_dependents();
  const float temp = a.temperature ? a.temperature[t] : 1.0f;
  const int top_k = a.top_k ? a.top_k[t] : 0;
  const float top_p = a.top_p ? a.top_p[t] : 1.0f;
  const float min_p = a.min_p ? a.min_p[t] : 0.0f;
  const float u = a.u[t];

  const void *row = static_cast<const uint8_t *>(a.logits) + ((size_t)t * a.ld + base) * (BF16 ? 2 : 4);
  const SpSrc<BF16, RES> src{row, vals, n, (reinterpret_cast<uintptr_t>(row) & (BF16 ? 7 : 15)) == 0};
  float mx, mn;
  if (wid == SP_WARPS - 1) {   // beside the others' loads
    if (lane == 0) sh->log_min_p = min_p > 0.0f ? log((double)min_p) : 0.0;
  }
  sp_load(src, vals, SP_WARPS * a.seg, mx, mn);
  if (tid < 32) sh->exp2_tab[tid] = SQ_EXP2[tid];
  mx = warp_max(mx);
  mn = -warp_max(-mn);
  if (lane == 0) {
    sh->warp_f[0][wid] = mx;
    sh->warp_f[1][wid] = mn;
  }
  __syncthreads();
  dense::cluster_wait();   // every CTA of the cluster is running: its shared memory may be written
  if (wid == 0) {
    mx = warp_max(sh->warp_f[0][lane % SP_WARPS]);
    mn = -warp_max(-sh->warp_f[1][lane % SP_WARPS]);
    push_all(&sh->push[6][rank], SpPush{(double)mx, (double)mn, 0.0f, 0}, a.nc);
  }
  dense::cluster_sync();
  SpRow r;
  r.max = -CUDART_INF_F;
  mn = CUDART_INF_F;
#pragma unroll 1
  for (int c = 0; c < a.nc; ++c) {
    r.max = fmaxf(r.max, (float)sh->push[6][c].a);
    mn = fminf(mn, (float)sh->push[6][c].b);
  }
  int par = 0;
  r.temp = (double)temp;
  r.bv = -CUDART_INF_F;
  r.bi = a.V;

  // parameters outside their ranges, and rows without a finite candidate (every
  // branch up to here and below is uniform over the cluster)
  const bool ok = temp >= 0.0f && temp < CUDART_INF_F && top_p == top_p && min_p <= 1.0f && u >= 0.0f && u < 1.0f;
  if (!ok || r.max == -CUDART_INF_F) {
    if (rank == 0 && tid == 0) {
      if (!ok) set_status(a.status, DEV_BAD_PARAM);
      a.token[t] = -1;
      if (a.prob) a.prob[t] = 0.0f;
    }
    dense::cluster_sync();
    return;
  }
  if (temp == 0.0f) {   // greedy: the lowest index of the largest logit
    int at = 0x7fffffff;
    for (int i = tid; i < n; i += SP_THREADS)
      if (src.at(i) == r.max) at = min(at, base + i);
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) sh->warp_i[wid] = at;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < SP_WARPS; ++w) at = min(at, sh->warp_i[w]);
      sh->part[par].n_in = at;
    }
    dense::cluster_sync();
    if (rank == 0 && tid == 0) {
#pragma unroll 1
      for (int c = 0; c < a.nc; ++c) at = min(at, dense::peer(&sh->part[par], c)->n_in);
      a.token[t] = at;
      if (a.prob) a.prob[t] = 1.0f;
    }
    dense::cluster_sync();
    return;
  }
  if (r.max < CUDART_INF_F) {
    if (sq_row<BF16, RES>(src, stack, base, r.max, mn, temp, top_k, top_p, min_p, u, sh, a, t, rank)) return;
    dense::cluster_sync();
  }
  if (tid == 0) sh->live = sp_live(r, min_p > 0.0f ? fmax((double)min_p, SP_W_MIN) : SP_W_MIN);
  __syncthreads();
  r.live = sh->live;

  if (top_k > 0 && top_k < a.V) sp_select<true>(src, n, base, r, (double)top_k, sh, a, rank, par);
  if (top_p < 1.0f) {
    double s = 0.0;
    for (int i = tid; i < n; i += SP_THREADS)
      if (sp_kept(src.at(i), base + i, r)) s += sp_weight(src.at(i), r);
    s = sp_cluster_sum(s, sh, a, par);
    // (at least the smallest weight: top_p <= 0 keeps the first rank)
    sp_select<false>(src, n, base, r, fmax(SP_W_MIN, (double)top_p * s), sh, a, rank, par);
  }

  // the token, by index: sums per warp segment, per CTA, over the cluster
  const int seg = (a.slice + SP_WARPS - 1) / SP_WARPS;
  const int s0 = wid * seg, s1 = min(n, s0 + seg);
  double ws = 0.0;
  for (int i = s0 + lane; i < s1; i += 32)
    if (sp_kept(src.at(i), base + i, r)) ws += sp_weight(src.at(i), r);
  ws = warp_sum_d(ws);
  if (lane == 0) sh->warp_d[1][wid] = ws;
  __syncthreads();
  if (tid == 0) {
    double s = 0.0;
    for (int w = 0; w < SP_WARPS; ++w) s += sh->warp_d[1][w];
    sh->part[par].in = s;
  }
  dense::cluster_sync();
  double total = 0.0;
#pragma unroll 1
  for (int c = 0; c < a.nc; ++c) total += dense::peer(&sh->part[par], c)->in;
  const double target = (double)u * total;
  double before = 0.0;
  int owner = -1, last = 0;
#pragma unroll 1
  for (int c = 0; c < a.nc && owner < 0; ++c) {
    const double s = dense::peer(&sh->part[par], c)->in;
    if (s > 0.0) last = c;
    if (before + s > target) owner = c;
    else before += s;
  }
  if (owner < 0) owner = last;
  if (rank == owner) {
    // the first warp whose running sum passes the target; the last with any
    // weight if rounding leaves none
    int ow = -1, lw = 0;
    double b2 = before, bw = before;
    for (int w = 0; w < SP_WARPS && ow < 0; ++w) {
      const double s = sh->warp_d[1][w];
      if (s > 0.0) lw = w, bw = b2;
      if (b2 + s > target) ow = w;
      else b2 += s;
    }
    if (ow < 0) ow = lw, b2 = bw;
    if (wid == ow) {
      int hit = -1, lastk = -1;
      for (int i0 = s0; i0 < s1 && hit < 0; i0 += 32) {
        const int i = i0 + lane;
        double x = i < s1 && sp_kept(src.at(i), base + i, r) ? sp_weight(src.at(i), r) : 0.0;
        const unsigned some = __ballot_sync(0xffffffffu, x > 0.0);
        const bool mine = x > 0.0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const unsigned over = __ballot_sync(0xffffffffu, mine && b2 + x > target);
        if (over) hit = i0 + __ffs(over) - 1;
        if (some) lastk = i0 + 31 - __clz(some);
        b2 += __shfl_sync(0xffffffffu, x, 31);
      }
      if (hit < 0) hit = lastk;
      if (lane == 0) {
        a.token[t] = base + hit;
        if (a.prob) a.prob[t] = (float)(sp_weight(src.at(hit), r) / total);
      }
    }
  }
  dense::cluster_sync();   // no CTA leaves while another may read its shared memory
}

}  // namespace
}  // namespace qmoe

using namespace qmoe;

extern "C" qmoe_status qmoe_sample(const void *logits, int dtype, int T, int V, int64_t ld, const float *temperature,
                                   const int32_t *top_k, const float *top_p, const float *min_p, const float *u,
                                   int32_t *token, float *prob, int32_t *dev_status, qmoe_stream_t stream) {
  if (!logits || !u || !token || !dev_status || T < 1 || V < 1) return QMOE_ERR_INVALID_ARG;
  if (dtype != QMOE_F32 && dtype != QMOE_BF16) return QMOE_ERR_INVALID_ARG;
  if (ld == 0) ld = V;
  if (ld < V) return QMOE_ERR_INVALID_ARG;
  const uintptr_t a4 = reinterpret_cast<uintptr_t>(temperature) | reinterpret_cast<uintptr_t>(top_k) |
                       reinterpret_cast<uintptr_t>(top_p) | reinterpret_cast<uintptr_t>(min_p) |
                       reinterpret_cast<uintptr_t>(u) | reinterpret_cast<uintptr_t>(token) |
                       reinterpret_cast<uintptr_t>(prob) | reinterpret_cast<uintptr_t>(dev_status);
  if ((a4 & 3) || !aligned16(logits)) return QMOE_ERR_INVALID_ARG;
  if (V > SP_MAX_V || T > SP_MAX_T) return QMOE_ERR_UNSUPPORTED;
  const auto smem_of = [](bool res, int seg) { return (int)(sp_head_bytes() + (size_t)SP_WARPS * (SQ_ROUND + (res ? seg : 0)) * 4); };
  const auto kernel = [&](bool res) {
    return dtype == QMOE_BF16 ? (res ? (const void *)sample_kernel<true, true> : (const void *)sample_kernel<true, false>)
                              : (res ? (const void *)sample_kernel<false, true> : (const void *)sample_kernel<false, false>);
  };
  // In shared memory, by as many CTAs per row as run at once, where they can hold it
  // (131072 fp32 logits, top-p: 12 rows by 8 CTAs 30 us, 18 to 30 rows by 4 33 us, where
  // 8, in two turns, take 46 and reading again and again 38). Else two CTAs per SM read rows
  // out of L2 (40 rows 50 us, in shared memory in turns 75; 73 rows 67 and 124), and at
  // least two per row where the rows under way do not fit there (256 rows of 131072:
  // 139 us, one each 148; of 60000: one each 72 us, two 82).
  static dense::ClusterCounts known[2];   // by type
  const int sms = num_sms();
  int nc = SP_MAX_CLUSTER;
  while (nc > 1 && (V < nc * SP_MIN_SLICE || T * (long long)nc > sms ||
                    T > dense::max_clusters(known[dtype == QMOE_BF16], nc, kernel(true), SP_THREADS, smem_of(true, SP_MAX_SLICE / SP_WARPS))))
    nc /= 2;
  const bool res = T <= sms && (V + nc - 1) / nc <= SP_MAX_SLICE;
  if (!res) {
    nc = 1;
    while (nc < SP_MAX_CLUSTER && T * (long long)nc <= sms && V >= 2 * nc * SP_MIN_SLICE) nc *= 2;
    if (nc == 1 && 2LL * sms * V * (dtype == QMOE_BF16 ? 2 : 4) > SP_L2_BYTES) nc = 2;
  }
  const int slice = ((V + nc - 1) / nc + 7) / 8 * 8;
  const int seg = (slice + SP_WARPS * 128 - 1) / (SP_WARPS * 128) * 128;
  const int smem = smem_of(res, seg);
  SpArgs args{logits, temperature, top_p, min_p, u,     top_k, token, prob, dev_status,
              ld,     T,           V,     slice, nc,    seg,   (seg + SQ_ROUND - 1) / SQ_ROUND};
  const void *fn = kernel(res);
  // (the largest a call can need, not this call's: the limit is the kernel's, for all host threads)
  const cudaError_t e =
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(res, SP_MAX_SLICE / SP_WARPS));
  if (e != cudaSuccess) return dense::launched(e);
  void *params[] = {&args};
  return dense::launch(fn, T * nc, SP_THREADS, smem, nc, params, (cudaStream_t)stream);
}
