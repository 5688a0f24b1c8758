// Residual RMSNorm with an 8-bit output, and the same row quantiser without
// the norm. For every row t (z, p and A as real numbers after z's rounding):
//   z = fl32(x + y),  r = 1 / sqrt(mean(z^2) + eps),  p = z * gain
//   A = max |p| over the scale's columns (the row, or a group of 32/64/128)
//   codes = rint(127 p / A) (ties to even),  scale = A r / 127
// r cancels in the codes, so they follow from p alone, and they are formed
// exactly: a code is taken from fp32 arithmetic (off by at most 3.1e-5 at
// |127 p / A| <= 127: four roundings of 2^-24 relative) unless that value lies
// within 1e-4 of a rounding border, where the thread repeats its columns with
// the exact float64 products (two 24-bit factors) and a float64 division.
// r and the scales are fp32 values from an fp32 sum of squares; rows whose
// fp32 sum or products leave the normal range are repeated in float64.
//
// Bound: HBM bandwidth (one read of x and y, one write per output; z stays in
// registers between the statistics and the codes). One CTA per row at a time,
// 8 columns per thread and load, CTAs loop over rows with the gain in
// registers, and one CTA barrier per row carries both statistics.
#include <cuda_bf16.h>

#include "common.cuh"

namespace qmoe {
namespace {

constexpr int NQ_VEC = 8;                    // columns per thread and chunk: 16 bytes of bf16, 8 bytes of codes
constexpr int NQ_MAX_THREADS = 512;
constexpr int NQ_MAX_CHUNKS = 4;
constexpr int NQ_MAX_H = NQ_VEC * NQ_MAX_THREADS * NQ_MAX_CHUNKS;
constexpr float NQ_MAGIC = 12582912.0f;      // 1.5 * 2^23: adding it rounds to an integer, ties to even
constexpr float NQ_NEAR = 0.4999f;           // fp32 codes this close to a border are settled in float64
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

// A product's exact magnitude is its fp32 value plus this remainder (exact by
// fused multiply-add for products well inside the fp32 range).
__device__ __forceinline__ float remainder_of(float z, float g, float hi) { return __fmaf_rn(fabsf(z), fabsf(g), -hi); }

__device__ __forceinline__ float lanes_max(float m, int width) {
  for (int o = width >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

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

template <int N>
__device__ __forceinline__ double thread_max_abs(const float (&z)[N], const float *g) {
  unsigned long long m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const double p = g ? (double)z[i] * (double)g[i] : (double)z[i];
    const unsigned long long n = (unsigned long long)__double_as_longlong(fabs(p));
    m = n > m ? n : m;
  }
  return __longlong_as_double((long long)m);
}

__device__ __forceinline__ double wider(double a, double b) {
  return (unsigned long long)__double_as_longlong(a) > (unsigned long long)__double_as_longlong(b) ? a : b;
}

__device__ __forceinline__ bool in_range(float v) { return v >= NQ_LO && v <= NQ_HI; }

// One code from the exact quotient.
__device__ __forceinline__ int code_exact(double p, double A) { return (int)rint(__ddiv_rn(__dmul_rn(p, 127.0), A)); }

template <bool BF16, int C, bool NORM>
__global__ void __launch_bounds__(NQ_MAX_THREADS) norm_q8_kernel(NqArgs a) {
  __shared__ float s_ss[2][NQ_MAX_THREADS / 32];
  __shared__ uint32_t s_hi[2][NQ_MAX_THREADS / 32];
  __shared__ float s_lo[2][NQ_MAX_THREADS / 32];
  __shared__ double s_d[NQ_MAX_THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int nchunk = a.H / NQ_VEC;
  const bool has_gain = NORM && a.gain;

  float g[C][NQ_VEC];
  if (NORM) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int ch = c * blockDim.x + tid;
#pragma unroll
      for (int i = 0; i < NQ_VEC; ++i) g[c][i] = 1.0f;
      if (has_gain && ch < nchunk) nq_load<false>(a.gain, (size_t)ch * NQ_VEC, g[c]);
    }
  }

  int par = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, par ^= 1) {
    const size_t row = (size_t)t * a.H;
    float z[C][NQ_VEC];
    float ss = 0.0f;
    uint32_t hi = 0;      // this thread's largest |p| in fp32 (all chunks; used for a row scale)
    uint32_t hic[C];      // per chunk (used for group scales)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int ch = c * blockDim.x + tid;
      if (ch < nchunk) nq_load<BF16>(a.x, row + (size_t)ch * NQ_VEC, z[c]);
      else
#pragma unroll
        for (int i = 0; i < NQ_VEC; ++i) z[c][i] = 0.0f;
    }
    if (NORM && a.y) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int ch = c * blockDim.x + tid;
        if (ch < nchunk) {
          float yv[NQ_VEC];
          nq_load<BF16>(a.y, row + (size_t)ch * NQ_VEC, yv);
#pragma unroll
          for (int i = 0; i < NQ_VEC; ++i) z[c][i] = __fadd_rn(z[c][i], yv[i]);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      hic[c] = 0;
#pragma unroll
      for (int i = 0; i < NQ_VEC; ++i) {
        if (NORM) ss = __fmaf_rn(z[c][i], z[c][i], ss);
        hic[c] = max(hic[c], mag(NORM ? __fmul_rn(z[c][i], g[c][i]) : z[c][i]));
      }
      hi = max(hi, hic[c]);
    }
    // the updated residual stream leaves as early as it can
    if (NORM && a.z) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int ch = c * blockDim.x + tid;
        if (ch < nchunk) {
          if (BF16) {
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.z) + row + (size_t)ch * NQ_VEC) = nq_bf16x8(z[c]);
          } else {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.z) + row + (size_t)ch * NQ_VEC);
            o[0] = make_float4(z[c][0], z[c][1], z[c][2], z[c][3]);
            o[1] = make_float4(z[c][4], z[c][5], z[c][6], z[c][7]);
          }
        }
      }
    }

    // row statistics: the sum of squares, and for a row scale the exact
    // largest |p|: the largest remainder among the products whose fp32 value
    // is the warp's largest, then among the warps that hold the row's largest
    float inv = 1.0f;
    double invd = 1.0;    // the same in float64 where `wide`
    bool wide = false;
    const bool row_scale = a.group == 0 && a.codes;
    const uint32_t whi = __reduce_max_sync(0xffffffffu, hi);
    if (row_scale) {
      float lo = -INFINITY;
      if (hi == whi) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < NQ_VEC; ++i) {
            const float gv = NORM ? g[c][i] : 1.0f;
            if (mag(__fmul_rn(z[c][i], gv)) == whi) lo = fmaxf(lo, remainder_of(z[c][i], gv, __uint_as_float(whi)));
          }
      }
      lo = lanes_max(lo, 32);
      if (lane == 0) s_lo[par][warp] = lo;
    }
    if (NORM) {
      ss = warp_sum(ss);
      if (lane == 0) s_ss[par][warp] = ss;
    }
    if (lane == 0) s_hi[par][warp] = whi;
    __syncthreads();
    uint32_t rhi = 0;
    float rss = 0.0f, rlo = -INFINITY;
    for (int w = 0; w < nw; ++w) {
      rhi = max(rhi, s_hi[par][w]);
      if (NORM) rss += s_ss[par][w];
    }
    double Arow = 0.0;
    if (row_scale) {
      for (int w = 0; w < nw; ++w)
        if (s_hi[par][w] == rhi) rlo = fmaxf(rlo, s_lo[par][w]);
      Arow = (double)__uint_as_float(rhi) + (double)rlo;
      if (!in_range(__uint_as_float(rhi))) {   // uniform over the CTA: fp32 products cannot be trusted
        double m = 0.0;
#pragma unroll
        for (int c = 0; c < C; ++c) m = wider(m, thread_max_abs(z[c], NORM ? g[c] : nullptr));
        m = lanes_max_abs(m, 32);
        __syncthreads();
        if (lane == 0) s_d[warp] = m;
        __syncthreads();
        Arow = 0.0;
        for (int w = 0; w < nw; ++w) Arow = wider(Arow, s_d[w]);
      }
    }
    if (NORM) {
      if (in_range(rss)) {
        inv = rsqrtf(__fdiv_rn(rss, (float)a.H) + a.eps);
      } else {   // tiny, huge or non-finite rows: the sum of squares and r in float64
        wide = true;
        double d = 0.0;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < NQ_VEC; ++i) d = fma((double)z[c][i], (double)z[c][i], d);
        d = warp_sum_d(d);
        __syncthreads();
        if (lane == 0) s_d[warp] = d;
        __syncthreads();
        d = 0.0;
        for (int w = 0; w < nw; ++w) d += s_d[w];
        // a NaN or an infinity in the row makes every value of it NaN
        const double m = d / a.H + (double)a.eps;
        invd = d <= 1.7e308 ? (m > 0.0 ? 1.0 / sqrt(m) : 0.0) : __longlong_as_double(0x7ff8000000000000ll);
        inv = __double2float_rn(invd);
      }
    }
    if (NORM && a.norm) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int ch = c * blockDim.x + tid;
        if (ch < nchunk) {
          float v[NQ_VEC];
#pragma unroll
          for (int i = 0; i < NQ_VEC; ++i) v[i] = __fmul_rn(__fmul_rn(z[c][i], inv), g[c][i]);
          if (wide)
#pragma unroll
            for (int i = 0; i < NQ_VEC; ++i) v[i] = __double2float_rn((double)z[c][i] * (double)g[c][i] * invd);
          *reinterpret_cast<uint4 *>(a.norm + row + (size_t)ch * NQ_VEC) = nq_bf16x8(v);
        }
      }
    }
    if (!a.codes) continue;

    const int gl = a.group / NQ_VEC;   // lanes per group
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int ch = c * blockDim.x + tid;
      if (c * blockDim.x + (tid & ~31) >= nchunk) break;   // the whole warp is past the row
      double Ad = Arow;   // the scale's exact largest |p|
      if (a.group != 0) {
        uint32_t m = hic[c];
        for (int o = gl >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        float lo = -INFINITY;
        if (hic[c] == m) {
#pragma unroll
          for (int i = 0; i < NQ_VEC; ++i) {
            const float gv = NORM ? g[c][i] : 1.0f;
            if (mag(__fmul_rn(z[c][i], gv)) == m) lo = fmaxf(lo, remainder_of(z[c][i], gv, __uint_as_float(m)));
          }
        }
        lo = lanes_max(lo, gl);
        Ad = (double)__uint_as_float(m) + (double)lo;
        const bool odd = !in_range(__uint_as_float(m));
        if (__any_sync(0xffffffffu, odd)) {
          const double e = lanes_max_abs(thread_max_abs(z[c], NORM ? g[c] : nullptr), gl);
          if (odd) Ad = e;
        }
      }
      const float A = __double2float_rn(Ad);
      const bool plain = in_range(A) && !wide;
      const bool finite = Ad <= 1.7e308 && inv == inv;   // neither NaN nor infinite
      uint32_t lo4 = 0, hi4 = 0;
      if (plain && finite) {
        const float r = __fdiv_rn(127.0f, A);
        float far = 0.0f;
#pragma unroll
        for (int i = 0; i < NQ_VEC; ++i) {
          const float v = __fmul_rn(NORM ? __fmul_rn(z[c][i], g[c][i]) : z[c][i], r);
          const float m = __fadd_rn(v, NQ_MAGIC);
          far = fmaxf(far, fabsf(__fsub_rn(v, __fsub_rn(m, NQ_MAGIC))));
          const uint32_t b = __float_as_uint(m) & 0xffu;
          if (i < 4) lo4 |= b << (8 * i);
          else hi4 |= b << (8 * (i - 4));
        }
        if (far > NQ_NEAR) {
          lo4 = hi4 = 0;
#pragma unroll
          for (int i = 0; i < NQ_VEC; ++i) {
            const float gv = NORM ? g[c][i] : 1.0f;
            const uint32_t b = (uint32_t)code_exact((double)z[c][i] * (double)gv, Ad) & 0xffu;
            if (i < 4) lo4 |= b << (8 * i);
            else hi4 |= b << (8 * (i - 4));
          }
        }
      } else if (finite && Ad > 0.0) {
#pragma unroll
        for (int i = 0; i < NQ_VEC; ++i) {
          const float gv = NORM ? g[c][i] : 1.0f;
          const uint32_t b = (uint32_t)code_exact((double)z[c][i] * (double)gv, Ad) & 0xffu;
          if (i < 4) lo4 |= b << (8 * i);
          else hi4 |= b << (8 * (i - 4));
        }
      }
      if (ch < nchunk) {
        *reinterpret_cast<uint2 *>(a.codes + row + (size_t)ch * NQ_VEC) = make_uint2(lo4, hi4);
        float sc;
        if (!finite) sc = __uint_as_float(0x7fffffffu);
        else if (plain) sc = __fdiv_rn(__fmul_rn(A, inv), 127.0f);
        else sc = __double2float_rn(Ad * (wide ? invd : (double)inv) / 127.0);
        if (a.group == 0) {
          if (ch == 0) a.scales[t] = sc;
        } else if (ch % gl == 0) {
          a.scales[(size_t)t * (a.H / a.group) + ch / gl] = sc;
        }
      }
    }
  }
}

template <bool BF16, bool NORM>
const void *nq_kernel(int C) {
  switch (C) {
    case 1: return (const void *)norm_q8_kernel<BF16, 1, NORM>;
    case 2: return (const void *)norm_q8_kernel<BF16, 2, NORM>;
    default: return (const void *)norm_q8_kernel<BF16, 4, NORM>;
  }
}

qmoe_status nq_launch(const NqArgs &a, int dtype, bool norm, cudaStream_t s) {
  const int nchunk = a.H / NQ_VEC;
  int C = 1;
  while (C < NQ_MAX_CHUNKS && nchunk > C * 256) C *= 2;
  const int threads = ((nchunk + C - 1) / C + 31) / 32 * 32;
  const void *fn = norm ? (dtype == QMOE_BF16 ? nq_kernel<true, true>(C) : nq_kernel<false, true>(C))
                        : (dtype == QMOE_BF16 ? nq_kernel<true, false>(C) : nq_kernel<false, false>(C));
  const int per_sm = 2048 / threads < 16 ? 2048 / threads : 16;
  const long long cap = (long long)num_sms() * per_sm;
  const int grid = a.T < cap ? a.T : (int)cap;
  NqArgs args = a;
  void *params[] = {&args};
  const cudaError_t e = cudaLaunchKernel(fn, dim3(grid), dim3(threads), params, 0, s);
  note_launch();
  return cuda_status(e);
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
  if (H % 16 || H > NQ_MAX_H || !nq_group_ok(group, H)) return QMOE_ERR_UNSUPPORTED;
  NqArgs a{x_in, y, gain, z_out, static_cast<__nv_bfloat16 *>(norm_out), codes, scales, eps, T, H, group};
  return nq_launch(a, dtype, true, (cudaStream_t)stream);
}

extern "C" qmoe_status qmoe_quantise_rows(const void *x, int dtype, int T, int H, int group, int8_t *codes,
                                          float *scales, qmoe_stream_t stream) {
  if (!x || !codes || !scales || T < 1 || H < 1 || (dtype != QMOE_F32 && dtype != QMOE_BF16))
    return QMOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || (reinterpret_cast<uintptr_t>(scales) & 3)) return QMOE_ERR_INVALID_ARG;
  if (H % 16 || H > NQ_MAX_H || !nq_group_ok(group, H)) return QMOE_ERR_UNSUPPORTED;
  NqArgs a{x, nullptr, nullptr, nullptr, nullptr, codes, scales, 0.0f, T, H, group};
  return nq_launch(a, dtype, false, (cudaStream_t)stream);
}
