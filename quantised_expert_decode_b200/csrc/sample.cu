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
// last element: a border (value, index). The row is read from HBM once, into
// the shared memory of a cluster of CTAs (a contiguous slice each), and the
// border is found there without sorting: a histogram over the value range
// locates the bin that the border falls into, exact sums over the row confirm
// it, and the bin's few elements are ranked one by one; a bin that is still
// too large is cut again. Sums that decide are float64, formed in a fixed
// order, so the same inputs give the same token on every run.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "dense.cuh"

namespace qmoe {
namespace {

constexpr int SP_THREADS = 512;
constexpr int SP_WARPS = SP_THREADS / 32;
constexpr int SP_BINS = 1024;
constexpr int SP_LIST = SP_THREADS;           // elements ranked one by one (one per thread)
constexpr int SP_MAX_CLUSTER = 8;
constexpr int SP_MAX_SLICE = 49152;           // 192 KB of fp32 logits per CTA
constexpr int SP_MAX_V = SP_MAX_CLUSTER * SP_MAX_SLICE;
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
};

// What one CTA contributes to a sum over the cluster.
struct SpPart {
  double above, in;          // weight above the bin, in the bin
  float min_above, max_in, min_in, max_below;
  int n_in, pad;
};

struct SpShared {
  SpPart part[2];
  double warp_d[2][SP_WARPS];
  float warp_f[4][SP_WARPS];
  int warp_i[SP_WARPS];
  unsigned long long mass[SP_BINS];
  unsigned int list_n;
  int found;
  float list_v[SP_LIST];
  int list_i[SP_LIST];
  float sort_v[SP_LIST];
  int sort_i[SP_LIST];
  float border_v;
  int border_i;
  float live;
};

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
template <bool COUNT>
__device__ void sp_select(const float *vals, int n, int base, SpRow &r, double target, SpShared *sh, const SpArgs &a,
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
      const float l = vals[i];
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
      const float l = vals[i];
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
        const float l = vals[i];
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
    for (int i = s0i + lane; i < s1i; i += 32) cnt += vals[i] == vhi && sp_kept(vals[i], base + i, r);
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
          const bool eq = i < s1i && vals[i] == vhi && sp_kept(vals[i], base + i, r);
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

template <bool BF16>
__global__ void __launch_bounds__(SP_THREADS) sample_kernel(SpArgs a) {
  extern __shared__ __align__(16) uint8_t sp_smem[];
  SpShared *sh = reinterpret_cast<SpShared *>(sp_smem);
  float *vals = reinterpret_cast<float *>(sp_smem + ((sizeof(SpShared) + 15) & ~(size_t)15));
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int rank = (int)dense::cluster_rank(), t = blockIdx.x / a.nc;
  const int base = min(a.V, rank * a.slice), n = min(a.V, base + a.slice) - base;

  const float temp = a.temperature ? a.temperature[t] : 1.0f;
  const int top_k = a.top_k ? a.top_k[t] : 0;
  const float top_p = a.top_p ? a.top_p[t] : 1.0f;
  const float min_p = a.min_p ? a.min_p[t] : 0.0f;
  const float u = a.u[t];

  // the slice into shared memory, NaN as -inf
  float mx = -CUDART_INF_F;
  auto put = [&](int i, float v) {
    v = v == v ? v : -CUDART_INF_F;
    vals[i] = v;
    mx = fmaxf(mx, v);
  };
  const size_t row = (size_t)t * a.ld + base;
  if (BF16) {
    const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(a.logits) + row;
    const int nv = (reinterpret_cast<uintptr_t>(p) & 15) == 0 ? n / 8 : 0;
    for (int i = tid; i < nv; i += SP_THREADS) {
      const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        put(8 * i + 2 * j, __uint_as_float(w[j] << 16));
        put(8 * i + 2 * j + 1, __uint_as_float(w[j] & 0xffff0000u));
      }
    }
    for (int i = 8 * nv + tid; i < n; i += SP_THREADS) put(i, __bfloat162float(p[i]));
  } else {
    const float *p = static_cast<const float *>(a.logits) + row;
    const int nv = (reinterpret_cast<uintptr_t>(p) & 15) == 0 ? n / 4 : 0;
    for (int i = tid; i < nv; i += SP_THREADS) {
      const float4 q = __ldcs(reinterpret_cast<const float4 *>(p) + i);
      put(4 * i, q.x);
      put(4 * i + 1, q.y);
      put(4 * i + 2, q.z);
      put(4 * i + 3, q.w);
    }
    for (int i = 4 * nv + tid; i < n; i += SP_THREADS) put(i, p[i]);
  }
  int par = 0;
  mx = warp_max(mx);
  if (lane == 0) sh->warp_f[0][wid] = mx;
  __syncthreads();
  if (tid == 0) {
    for (int w = 0; w < SP_WARPS; ++w) mx = fmaxf(mx, sh->warp_f[0][w]);
    sh->part[par].max_in = mx;
  }
  dense::cluster_sync();
  SpRow r;
  r.max = -CUDART_INF_F;
  for (int c = 0; c < a.nc; ++c) r.max = fmaxf(r.max, dense::peer(&sh->part[par], c)->max_in);
  par ^= 1;
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
      if (vals[i] == r.max) at = min(at, base + i);
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) sh->warp_i[wid] = at;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < SP_WARPS; ++w) at = min(at, sh->warp_i[w]);
      sh->part[par].n_in = at;
    }
    dense::cluster_sync();
    if (rank == 0 && tid == 0) {
      for (int c = 0; c < a.nc; ++c) at = min(at, dense::peer(&sh->part[par], c)->n_in);
      a.token[t] = at;
      if (a.prob) a.prob[t] = 1.0f;
    }
    dense::cluster_sync();
    return;
  }
  if (tid == 0) sh->live = sp_live(r, min_p > 0.0f ? fmax((double)min_p, SP_W_MIN) : SP_W_MIN);
  __syncthreads();
  r.live = sh->live;

  if (top_k > 0 && top_k < a.V) sp_select<true>(vals, n, base, r, (double)top_k, sh, a, rank, par);
  if (top_p < 1.0f) {
    double s = 0.0;
    for (int i = tid; i < n; i += SP_THREADS)
      if (sp_kept(vals[i], base + i, r)) s += sp_weight(vals[i], r);
    s = sp_cluster_sum(s, sh, a, par);
    // (at least the smallest weight: top_p <= 0 keeps the first rank)
    sp_select<false>(vals, n, base, r, fmax(SP_W_MIN, (double)top_p * s), sh, a, rank, par);
  }

  // the token, by index: sums per warp segment, per CTA, over the cluster
  const int seg = (a.slice + SP_WARPS - 1) / SP_WARPS;
  const int s0 = wid * seg, s1 = min(n, s0 + seg);
  double ws = 0.0;
  for (int i = s0 + lane; i < s1; i += 32)
    if (sp_kept(vals[i], base + i, r)) ws += sp_weight(vals[i], r);
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
  for (int c = 0; c < a.nc; ++c) total += dense::peer(&sh->part[par], c)->in;
  const double target = (double)u * total;
  double before = 0.0;
  int owner = -1, last = 0;
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
        double x = i < s1 && sp_kept(vals[i], base + i, r) ? sp_weight(vals[i], r) : 0.0;
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
        if (a.prob) a.prob[t] = (float)(sp_weight(vals[hit], r) / total);
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
  if (V > SP_MAX_V || T > (1 << 27)) return QMOE_ERR_UNSUPPORTED;
  int nc = 1;
  // enough CTAs to hold the row, then enough to fill the machine
  while (nc < SP_MAX_CLUSTER && ((V + nc - 1) / nc > SP_MAX_SLICE / 3 || (long long)T * nc * 2 <= num_sms())) nc *= 2;
  const int slice = ((V + nc - 1) / nc + 7) / 8 * 8;
  const size_t smem = ((sizeof(SpShared) + 15) & ~(size_t)15) + (size_t)slice * 4;
  if (smem > max_smem_optin()) return QMOE_ERR_UNSUPPORTED;
  SpArgs args{logits, temperature, top_p, min_p, u, top_k, token, prob, dev_status, ld, T, V, slice, nc};
  const void *fn = dtype == QMOE_BF16 ? (const void *)sample_kernel<true> : (const void *)sample_kernel<false>;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return QMOE_ERR_CUDA;
  void *params[] = {&args};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)T * (unsigned)nc);
  cfg.blockDim = dim3(SP_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = nc;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, params);
  note_launch();
  return cuda_status(e);
}
