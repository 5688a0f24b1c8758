// Residual RMSNorm with an 8-bit output, and the same row quantiser without
// the norm. For every row t (z, p and A as real numbers after z's rounding):
//   z = fl32(x + y),  r = 1 / sqrt(mean(z^2) + eps),  p = z * gain
//   A = max |p| over the scale's columns (the row, or a group of 32/64/128)
//   codes = rint(127 p / A) (ties to even),  scale = A r / 127
// r cancels in the codes, so they follow from p alone, and they are formed
// exactly: a code is taken from fp32 arithmetic (five roundings of 2^-24
// relative) unless that lies within its error of a rounding border. Such a code
// (8 in a million) is decided by two float64 products with A's fp32 value, and
// where that value's own rounding leaves it open by the exact A, the largest
// exact product (of two 24-bit factors).
// r and the scales are fp32 values from an fp32 sum of squares; rows whose
// fp32 sum or products leave the normal range are repeated in float64.
//
// Bound: HBM bandwidth for fp32 rows (one read of x and y, one write per output; z
// waits in shared memory between the statistics and the codes: 8192 x 2048 with
// x, y and z in fp32 41.4 us, 80 % of the measured copy rate), for bf16 rows the
// issue of some 40 instructions a column (8192 x 2048 with the normed rows too 34.3 us,
// 67 %). One CTA per row at a time, 8 neighbouring columns per thread and round, CTAs
// loop over rows, two rows' z in turn, so that one CTA barrier per row carries all
// statistics; the next row is fetched into L2 meanwhile. What is rare follows the
// loop as loops of its own: called, or inlined where it is found, it took registers
// from every row (a third of the speed).
#include <cuda_bf16.h>

#include "dense.cuh"

namespace qmoe {
namespace {

constexpr int NQ_VEC = 8;                    // columns per thread and chunk: 16 bytes of bf16, 8 bytes of codes
constexpr int NQ_MAX_THREADS = 512;
constexpr int NQ_SMEM = 220 * 1024;          // of an SM, for rows
constexpr int NQ_MAX_CTA_SMEM = NQ_SMEM / 2; // of a CTA: two rows in turn only where two CTAs fit
constexpr int NQ_MAX_H = 16384, NQ_MAX_T = 1 << 30;
constexpr float NQ_MAGIC = 12582912.0f;      // 1.5 * 2^23: adding it rounds to an integer, ties to even
constexpr float NQ_ERR = 3.1e-7f;            // bound of a code's fp32 error relative to it: five roundings of 2^-24
// fp32 statistics outside these are formed again in float64
constexpr float NQ_LO = 1e-25f, NQ_HI = 1e25f;

struct NqArgs {
  const void *x, *y;          // [T][H] fp32 or bf16; y may be null
  const float *gain;          // [H] or null
  void *z;                    // [T][H] like x, or null
  __nv_bfloat16 *norm;        // [T][H] or null
  int8_t *codes;              // [T][H]
  float *scales;              // [T] or [T][H / group]
  float eps;
  int T, H, group;            // group 0: one scale per row
};

template <bool BF16>
__device__ __forceinline__ void nq_load(const void *p, size_t e, float (&v)[NQ_VEC]) {
  if (BF16) {
    const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + e);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + e);
    const float4 a = f[0], b = f[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

__device__ __forceinline__ uint4 nq_bf16x8(const float (&v)[NQ_VEC]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Magnitude bits: unsigned order is the order of |v|, infinities above every
// finite value and NaNs above those.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Largest |p| in float64 over `width` adjacent lanes; magnitudes' bits order
// like the magnitudes, NaN above everything.
__device__ __forceinline__ double lanes_max_abs(double v, int width) {
  unsigned long long m = (unsigned long long)__double_as_longlong(fabs(v));
  for (int o = width >> 1; o > 0; o >>= 1) {
    const unsigned long long n = __shfl_xor_sync(0xffffffffu, m, o);
    m = n > m ? n : m;
  }
  return __longlong_as_double((long long)m);
}

__device__ __forceinline__ double wider(double a, double b) {
  return (unsigned long long)__double_as_longlong(a) > (unsigned long long)__double_as_longlong(b) ? a : b;
}

__device__ __forceinline__ bool in_range(float v) { return v >= NQ_LO && v <= NQ_HI; }

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

struct NqShared {
  float ss[2][NQ_MAX_THREADS / 32];
  uint32_t hi[2][NQ_MAX_THREADS / 32];
  double d[NQ_MAX_THREADS / 32];
};

__device__ __forceinline__ void nq_get(const float *zs, int ch, float (&z)[NQ_VEC]) {
  nq_load<false>(zs, (size_t)ch * NQ_VEC, z);
}

// ---- what is rare

__device__ __forceinline__ float nq_gain1(const NqArgs &a, int h) { return a.gain ? __ldg(a.gain + h) : 1.0f; }

// The float64 quotient's code.
__device__ __forceinline__ int code_exact(double p, double A) { return (int)rint(__ddiv_rn(__dmul_rn(p, 127.0), A)); }

// Largest |p| in float64 of the columns h0 .. h1 - 1, step by step (one thread).
__device__ __forceinline__ double cols_max_abs(const NqArgs &a, const float *zs, int h0, int h1, int step) {
  double m = 0.0;
#pragma unroll 1
  for (int h = h0; h < h1; h += step) m = wider(m, fabs((double)zs[h] * (double)nq_gain1(a, h)));
  return m;
}

// The codes near a border of one warp's chunks, from z's exact products with the
// gain. A code between k and k + 1 is k + 1 where 254 |p| > (2 k + 1) A, two
// float64 products; where A's fp32 value (known to 2^-24; exact without a gain)
// does not decide it the exact A does: its fp32 value plus the largest remainder
// among the products that round to it; and what that leaves open the quotient.
// (The scan for that remainder takes 4 columns a lane with 4 loads in flight: in
// single columns it took as long as several rows, 42 us for the 8192 x 2048 case.)
__device__ __forceinline__ void settle(const NqArgs &a, const float *zs, int t, int ch, float Af, bool near) {
  const int h0 = ch * NQ_VEC, lane = threadIdx.x & 31;
  if (a.group != 0) {   // the group's largest |p| in fp32
    uint32_t m = 0;
    if (h0 < a.H) {
      float z[NQ_VEC], g[NQ_VEC];
      nq_get(zs, ch, z);
#pragma unroll
      for (int i = 0; i < NQ_VEC; ++i) g[i] = 1.0f;
      if (a.gain) nq_load<false>(a.gain, h0, g);
#pragma unroll
      for (int i = 0; i < NQ_VEC; ++i) m = max(m, mag(__fmul_rn(z[i], g[i])));
    }
    __syncwarp();
    for (int o = a.group / NQ_VEC >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    Af = __uint_as_float(m);
  }
  const float r = __fmul_rn(127.0f, __frcp_rn(Af));
  double A = (double)Af;
  bool exact = !a.gain;
  unsigned ties = 0;
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    bool open = false;
    if (near) {
      float z[NQ_VEC], g[NQ_VEC];
      nq_get(zs, ch, z);
#pragma unroll
      for (int i = 0; i < NQ_VEC; ++i) g[i] = 1.0f;
      if (a.gain) nq_load<false>(a.gain, h0, g);
#pragma unroll
      for (int i = 0; i < NQ_VEC; ++i) {
        const float v = __fmul_rn(__fmul_rn(z[i], g[i]), r);
        if (__fmaf_rn(fabsf(v), NQ_ERR, fabsf(v - rintf(v))) <= 0.499999f) continue;
        const double p = (double)z[i] * (double)g[i];
        const float f = floorf(fabsf(v));
        const double left = 254.0 * fabs(p), right = (double)(2.0f * f + 1.0f) * A;
        // (without a gain both sides are exact, and a tie goes to the even code)
        int k = (int)f + (left > right || (!a.gain && left == right && ((int)f & 1)) ? 1 : 0);
        k = v < 0.0f ? -k : k;
        if (a.gain && fabs(left - right) <= (exact ? 1e-14 : 1.3e-7) * right) {
          if (exact) ties |= 1u << i;
          else open = true;
        }
        a.codes[(size_t)t * a.H + h0 + i] = (int8_t)k;
      }
#pragma unroll 1
      for (; ties; ties &= ties - 1) {
        const int h = h0 + __ffs(ties) - 1;
        a.codes[(size_t)t * a.H + h] = (int8_t)code_exact((double)zs[h] * (double)nq_gain1(a, h), A);
      }
    }
    if (exact || !__any_sync(0xffffffffu, open)) break;
    float lo = -INFINITY;
    const int c0 = a.group ? h0 : 4 * lane, c1 = a.group ? min(h0 + NQ_VEC, a.H) : a.H, cs = a.group ? 4 : 128;
#pragma unroll 4
    for (int h = c0; h < c1; h += cs) {
      const float4 z = *reinterpret_cast<const float4 *>(zs + h), g = __ldg(reinterpret_cast<const float4 *>(a.gain + h));
      const float zz[4] = {z.x, z.y, z.z, z.w}, gg[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float rem = __fmaf_rn(fabsf(zz[i]), fabsf(gg[i]), -Af);
        lo = fmaxf(lo, mag(__fmul_rn(zz[i], gg[i])) == mag(Af) ? rem : -INFINITY);
      }
    }
    __syncwarp();
    for (int o = (a.group ? a.group / NQ_VEC : 32) >> 1; o > 0; o >>= 1) lo = fmaxf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    A = (double)Af + (double)lo;
    exact = true;
  }
}

// A chunk of one warp in float64: the row's A (or its own groups'), 1 / rms.
__device__ __forceinline__ void chunk_slow(const NqArgs &a, const float *zs, int t, int ch, double A, double r) {
  const int gl = a.group / NQ_VEC, h0 = ch * NQ_VEC, h1 = min(h0 + NQ_VEC, a.H);
  if (a.group != 0) A = lanes_max_abs(cols_max_abs(a, zs, h0, h1, 1), gl);
  const bool finite = A <= 1.7e308 && r == r;   // neither NaN nor infinite
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    const double p = (double)zs[h] * (double)nq_gain1(a, h);
    if (a.norm) a.norm[(size_t)t * a.H + h] = __float2bfloat16_rn(__double2float_rn(p * r));
    if (a.codes) a.codes[(size_t)t * a.H + h] = (int8_t)(finite && A > 0.0 ? code_exact(p, A) : 0);
  }
  if (!a.codes || h0 >= a.H) return;
  const float sc = finite ? __double2float_rn(A * r / 127.0) : __uint_as_float(0x7fffffffu);
  if (a.group == 0) {
    if (ch == 0) a.scales[t] = sc;
  } else if ((ch & (gl - 1)) == 0) {
    a.scales[((size_t)t * a.H + h0) / a.group] = sc;
  }
}

// 1 / rms of a row in float64 (whole CTA). A NaN or an infinity makes it NaN.
__device__ __forceinline__ double row_inverse(const NqArgs &a, const float *zs, NqShared *sh) {
  double d = 0.0;
  // (each thread its own columns: the others' may not be there yet)
  for (int ch = threadIdx.x; ch < a.H / NQ_VEC; ch += blockDim.x)
#pragma unroll 1
    for (int i = 0; i < NQ_VEC; ++i) d = fma((double)zs[ch * NQ_VEC + i], (double)zs[ch * NQ_VEC + i], d);
  d = warp_sum_d(d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh->d[threadIdx.x >> 5] = d;
  __syncthreads();
  d = 0.0;
  for (int w = 0; w < (int)blockDim.x >> 5; ++w) d += sh->d[w];
  const double m = d / a.H + (double)a.eps;
  return d <= 1.7e308 ? (m > 0.0 ? 1.0 / sqrt(m) : 0.0) : __longlong_as_double(0x7ff8000000000000ll);
}

template <bool BF16, bool NORM>
__global__ void __launch_bounds__(NQ_MAX_THREADS, 2) norm_q8_kernel(const __grid_constant__ NqArgs a) {
  extern __shared__ __align__(16) float z_rows[];   // two rows' z, in turn
  __shared__ NqShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int nchunk = a.H / NQ_VEC, step = blockDim.x;
  const bool row_scale = a.group == 0 && a.codes, gain = NORM && a.gain;
  const int gl = a.group / NQ_VEC;   // lanes per group
  const float inv_h = 1.0f / (float)a.H;

  pdl_wait();   // (the next kernel is let in at the end only: its waiting CTAs took places unevenly, 4 % at 1003 x 5248)
  int par = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, par ^= 1) {
    const size_t row = (size_t)t * a.H;
    float *zs = z_rows + par * a.H;
    float ss = 0.0f;
    uint32_t hi = 0;   // magnitude bits of this thread's largest |p| in fp32
#pragma unroll 2
    for (int ch = tid; ch < nchunk; ch += step) {
      const size_t e = row + (size_t)ch * NQ_VEC;
      float z[NQ_VEC];
      nq_load<BF16>(a.x, e, z);
      if (NORM && a.y) {
        float y[NQ_VEC];
        nq_load<BF16>(a.y, e, y);
#pragma unroll
        for (int i = 0; i < NQ_VEC; ++i) z[i] = __fadd_rn(z[i], y[i]);
      }
      float4 *q = reinterpret_cast<float4 *>(zs + ch * NQ_VEC);
      q[0] = make_float4(z[0], z[1], z[2], z[3]);
      q[1] = make_float4(z[4], z[5], z[6], z[7]);
      if (NORM && a.z) {   // the updated residual stream
        if (BF16) {
          *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.z) + e) = nq_bf16x8(z);
        } else {
          float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.z) + e);
          o[0] = make_float4(z[0], z[1], z[2], z[3]);
          o[1] = make_float4(z[4], z[5], z[6], z[7]);
        }
      }
      if (NORM)
#pragma unroll
        for (int i = 0; i < NQ_VEC; ++i) ss = __fmaf_rn(z[i], z[i], ss);
      if (row_scale) {
        if (gain) {
          float g[NQ_VEC];
          nq_load<false>(a.gain, (size_t)ch * NQ_VEC, g);
#pragma unroll
          for (int i = 0; i < NQ_VEC; ++i) z[i] = __fmul_rn(z[i], g[i]);
        }
#pragma unroll
        for (int i = 0; i < NQ_VEC; ++i) hi = max(hi, mag(z[i]));
      }
    }

    // the CTA's next row on its way into L2 while this one is worked on
    if (t + (int)gridDim.x < a.T && (lane & (BF16 ? 7 : 3)) == 0)   // (a 128-byte line per 8 or 4 lanes)
      for (int ch = tid; ch < nchunk; ch += step) {
        const size_t e = row + (size_t)gridDim.x * a.H + (size_t)ch * NQ_VEC;
        prefetch_l2(static_cast<const uint8_t *>(a.x) + e * (BF16 ? 2 : 4));
        if (NORM && a.y) prefetch_l2(static_cast<const uint8_t *>(a.y) + e * (BF16 ? 2 : 4));
      }

    // row statistics
    if (NORM) {
      ss = warp_sum(ss);
      if (lane == 0) sh.ss[par][warp] = ss;
    }
    if (row_scale) {
      hi = __reduce_max_sync(0xffffffffu, hi);
      if (lane == 0) sh.hi[par][warp] = hi;
    }
    __syncthreads();
    uint32_t rhi = 0;
    float rss = 0.0f;
    for (int w = 0; w < nw; ++w) {
      if (NORM) rss += sh.ss[par][w];
      rhi = max(rhi, sh.hi[par][w]);
    }
    float Af = __uint_as_float(rhi), r = __fmul_rn(127.0f, __frcp_rn(Af));   // the scale's largest |p| in fp32
    // (uniform) rows whose fp32 sum of squares or largest product leaves the normal
    // range - tiny, huge, not finite - are done again below
    const bool odd = (NORM && !in_range(rss)) || (row_scale && !in_range(Af));
    const float inv = NORM ? rsqrtf(__fmaf_rn(rss, inv_h, a.eps)) : 1.0f;

    unsigned near = 0, slow = 0, bit = 1;   // rounds whose chunks are not settled yet
#pragma unroll 1
    for (int ch = tid; ch - lane < nchunk; ch += step, bit <<= 1) {   // (whole warps)
      const bool live = ch < nchunk;
      const size_t e = row + (size_t)ch * NQ_VEC;
      float p[NQ_VEC];
      nq_get(zs, live ? ch : 0, p);
      if (NORM && !a.codes) {
        // the normed row alone: (z r) gain, as |z r| is at most sqrt(H), while z gain may leave
        // the fp32 range where the normed row does not
#pragma unroll
        for (int i = 0; i < NQ_VEC; ++i) p[i] = __fmul_rn(p[i], inv);
        if (gain) {
          float g[NQ_VEC];
          nq_load<false>(a.gain, (size_t)(live ? ch : 0) * NQ_VEC, g);
#pragma unroll
          for (int i = 0; i < NQ_VEC; ++i) p[i] = __fmul_rn(p[i], g[i]);
        }
        const uint4 o = nq_bf16x8(p);
        if (live) *reinterpret_cast<uint4 *>(a.norm + e) = o;
        continue;
      }
      if (gain) {
        float g[NQ_VEC];
        nq_load<false>(a.gain, (size_t)(live ? ch : 0) * NQ_VEC, g);
#pragma unroll
        for (int i = 0; i < NQ_VEC; ++i) p[i] = __fmul_rn(p[i], g[i]);
      }
      if (NORM && a.norm) {
        // (z gain) r, as the codes need z gain: the columns whose largest product leaves the range
        // below are done again; a product below 2^-126 among larger ones is off by up to 2^-150
        float v[NQ_VEC];
#pragma unroll
        for (int i = 0; i < NQ_VEC; ++i) v[i] = __fmul_rn(p[i], inv);
        const uint4 o = nq_bf16x8(v);
        if (live) *reinterpret_cast<uint4 *>(a.norm + e) = o;
      }

      if (a.group != 0) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < NQ_VEC; ++i) m = max(m, mag(p[i]));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));   // (at least 4 lanes)
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        if (gl > 4) m = max(m, __shfl_xor_sync(0xffffffffu, m, 4));
        if (gl > 8) m = max(m, __shfl_xor_sync(0xffffffffu, m, 8));
        Af = __uint_as_float(m);
        r = __fmul_rn(127.0f, __frcp_rn(Af));
        slow |= live && !in_range(Af) ? bit : 0u;
      }
      uint2 codes;
      float far = 0.0f;
      {
        uint32_t m[NQ_VEC];
#pragma unroll
        for (int i = 0; i < NQ_VEC; ++i) {
          const float v = __fmul_rn(p[i], r), q = __fadd_rn(v, NQ_MAGIC);
          far = fmaxf(far, __fmaf_rn(fabsf(v), NQ_ERR, fabsf(__fsub_rn(v, __fsub_rn(q, NQ_MAGIC)))));
          m[i] = __float_as_uint(q);
        }
        codes.x = __byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410);
        codes.y = __byte_perm(__byte_perm(m[4], m[5], 0x0040), __byte_perm(m[6], m[7], 0x0040), 0x5410);
      }
      near |= live && far > 0.499999f ? bit : 0u;
      const float sc = __fmul_rn(__fmul_rn(Af, inv), 1.0f / 127.0f);
      if (live) {
        *reinterpret_cast<uint2 *>(a.codes + e) = codes;
        if (a.group == 0) {
          if (ch == 0) a.scales[t] = sc;
        } else if ((ch & (gl - 1)) == 0) {
          a.scales[((size_t)t * nchunk + ch) / gl] = sc;
        }
      }
    }
    // now and then: what the fp32 arithmetic left open, or could not do
    const unsigned all = odd ? bit - 1u : 0u;   // (a warp's rounds so far)
    unsigned m = __reduce_or_sync(0xffffffffu, near | slow | all);
    if (m == 0) continue;
    double A = 0.0, rd = (double)inv;
    if (odd) {
      if (NORM) rd = row_inverse(a, zs, &sh);
      if (row_scale) A = lanes_max_abs(cols_max_abs(a, zs, lane, a.H, 32), 32);
    }
    for (; m; m &= m - 1) {
      const int k = __ffs(m) - 1, ch = tid + k * step;
      if (odd || __any_sync(0xffffffffu, slow >> k & 1)) chunk_slow(a, zs, t, ch, A, rd);
      else settle(a, zs, t, ch, Af, near >> k & 1);
    }
  }
}

qmoe_status nq_launch(const NqArgs &a, int dtype, bool norm, cudaStream_t s) {
  // Threads per row: many rows 128, so that a thread's part of the reductions is
  // shared by more columns; fewer rows than the SMs hold at once more, for the shorter
  // chain (800 x 2048 bf16: 5.8 us with 128, 6.3 with 256; 8192 x 2048: 33.5, 38.5; 400 x
  // 4096: 6.5 with 256, 7.1 with 512; one row: 2.6 with 512, 3.3 with 128); and enough to
  // fill an SM with as many CTAs as its shared memory holds (2000 x 4096: 19 us with 256,
  // 25 with 128; 1100 x 8192: 23 with 512, 32 with 256).
  const int nchunk = a.H / NQ_VEC, sms = num_sms(), row = a.H * (int)sizeof(float);
  const int fit = NQ_SMEM / (2 * row);   // CTAs per SM with two rows in turn
  const int want = a.T > 4 * sms ? 128 : a.T > 2 * sms ? 256 : NQ_MAX_THREADS;
  const int least = fit >= 8 ? 128 : fit >= 4 ? 256 : NQ_MAX_THREADS, most = want > least ? want : least;
  const int threads = nchunk >= most ? most : (nchunk + 31) / 32 * 32;
  const void *fn = norm ? (dtype == QMOE_BF16 ? (const void *)norm_q8_kernel<true, true> : (const void *)norm_q8_kernel<false, true>)
                        : (dtype == QMOE_BF16 ? (const void *)norm_q8_kernel<true, false> : (const void *)norm_q8_kernel<false, false>);
  // CTAs that run at once and loop over rows; the widest rows one each (600 x 16384 bf16: 30 us, in turn 58)
  const long long cap = fit >= 2 ? (long long)(1024 / threads < fit ? 1024 / threads : fit) * sms : a.T;
  const int grid = a.T < cap ? a.T : (int)cap, smem = (grid < a.T ? 2 : 1) * row;
  cudaError_t e = cudaSuccess;
  // (the largest a call can need, not this call's: the limit is the kernel's, for all host threads)
  static_assert(NQ_MAX_H * sizeof(float) <= NQ_MAX_CTA_SMEM, "one of the widest rows");
  if (smem > 40 * 1024) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, NQ_MAX_CTA_SMEM);
  if (e != cudaSuccess) return dense::launched(e);
  NqArgs args = a;
  void *params[] = {&args};
  return dense::launch(fn, grid, threads, smem, 1, params, s);
}

bool nq_group_ok(int group, int H) { return group == 0 || ((group == 32 || group == 64 || group == 128) && H % group == 0); }

}  // namespace
}  // namespace qmoe

using namespace qmoe;

extern "C" qmoe_status qmoe_rmsnorm_residual_q8(const void *x_in, const void *y, int dtype, const float *gain, float eps,
                                                int T, int H, int group, void *z_out, void *norm_out, int8_t *codes,
                                                float *scales, qmoe_stream_t stream) {
  if (!x_in || T < 1 || H < 1 || (dtype != QMOE_F32 && dtype != QMOE_BF16)) return QMOE_ERR_INVALID_ARG;
  if ((codes == nullptr) != (scales == nullptr) || (!codes && !norm_out)) return QMOE_ERR_INVALID_ARG;
  if (!aligned16(x_in) || !aligned16(y) || !aligned16(gain) || !aligned16(z_out) || !aligned16(norm_out) ||
      !aligned16(codes) || (reinterpret_cast<uintptr_t>(scales) & 3))
    return QMOE_ERR_INVALID_ARG;
  if (!(eps >= 0.0f)) return QMOE_ERR_INVALID_ARG;
  if (T > NQ_MAX_T || H % 16 || H > NQ_MAX_H || !nq_group_ok(group, H)) return QMOE_ERR_UNSUPPORTED;
  NqArgs a{x_in, y, gain, z_out, static_cast<__nv_bfloat16 *>(norm_out), codes, scales, eps, T, H, group};
  return nq_launch(a, dtype, true, (cudaStream_t)stream);
}

extern "C" qmoe_status qmoe_quantise_rows(const void *x, int dtype, int T, int H, int group, int8_t *codes,
                                          float *scales, qmoe_stream_t stream) {
  if (!x || !codes || !scales || T < 1 || H < 1 || (dtype != QMOE_F32 && dtype != QMOE_BF16))
    return QMOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || (reinterpret_cast<uintptr_t>(scales) & 3)) return QMOE_ERR_INVALID_ARG;
  if (T > NQ_MAX_T || H % 16 || H > NQ_MAX_H || !nq_group_ok(group, H)) return QMOE_ERR_UNSUPPORTED;
  NqArgs a{x, nullptr, nullptr, nullptr, nullptr, codes, scales, 0.0f, T, H, group};
  return nq_launch(a, dtype, false, (cudaStream_t)stream);
}
