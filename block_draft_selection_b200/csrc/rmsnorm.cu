// Root-mean-square norm with the residual's addition, and rows to int8.
//
//   h = bf16(x + residual),  r = 1 / sqrt(mean h^2 + eps),  y = h gamma r
//   int8: a = max |h gamma|, scale = a r / 127, q = rint(127 h gamma / a)
//
// One CTA per row, or one warp where there are many short ones; the row stays
// in registers (VPT vectors of 8 channels per thread), so every input byte is
// read once.  r cancels in q, so the sum of squares and the maximum come out of
// one reduction and nothing waits for r before the second pass over the
// registers.  Memory bound: what counts is bytes in flight.  Many rows take few threads with up to 8 vectors each,
// all loaded before the first is used, and as many CTAs as fit on an SM; few
// rows take one vector per thread, where the shortest chain counts.
//
// q is decided exactly.  h and gamma are bf16, so p = h * gamma has at most 16
// significant bits, and p, 127 p and q a (7 more bits) are exact in fp32; so
// is their difference, which is below a.  q = rint(p (127 / a)), off by 2e-5
// at most, is then the right one wherever |127 p - q a| < a / 2; elsewhere
// (one value in 30000) the vector is divided out: 127 p / a differs from a
// halfway point, where it is not one, by a relative 2^-16 / 254 = 6.01e-8 or
// more (both sides are multiples of 2^-15 of their leading bits), above the
// 2^-24 = 5.96e-8 of a correctly rounded division, so rounding the IEEE
// quotient gives what rounding the real one gives.  Without gamma
// (dflash_quant_i8) the operands have 8 bits and the nearest miss is 2^-9 / 127
// of q away, so the product with 127 / a decides alone, provided that true
// halves stay halves or err upwards: those are x = a/2 (q = 63.5, even
// neighbour 64) and, where a is 127 times a power of two, exact products.
// 127 / a is therefore rounded up.
//
// Where the sum of squares overflows fp32, r is taken in fp64, and h, whose
// product with gamma may overflow too, goes on as h 2^-66, exact but for values
// that are nothing beside the row's, with r 2^66.  Elsewhere |h| < 2^64, so that
// |h gamma| is finite for every |gamma| < 2^64.
#include <cuda_bf16.h>

#include "common.cuh"
#include "host_util.cuh"
#include "pairs.cuh"

namespace dflash {
namespace norm {

constexpr unsigned FULL = 0xffffffffu;
constexpr int MAX_D = 32768;
constexpr float MAGIC = 12582912.f;   // 1.5 * 2^23: adding it rounds to an integer, ties to even, in the low bits

struct Args {
  const uint4* x;
  const uint4* res;
  const uint4* gamma;
  uint4* h;
  uint4* y;
  uint2* q;
  float* scale;
  float eps;
  float inv_d;
  int d8;
  int M;
};

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// |h gamma| of a vector's values joined to the maximum a; NaN if one is.
__device__ __forceinline__ float join_max(float a, const uint4& h, const uint4& g) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float u, v;
    mul2(widen2(word(h, i)), widen2(word(g, i))).get(u, v);
    a = max_nan(a, fabsf(u));
    a = max_nan(a, fabsf(v));
  }
  return a;
}

__device__ __forceinline__ uint32_t narrow2(F2 f) {
  float a, b;
  f.get(a, b);
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The low bytes of four words.
__device__ __forceinline__ uint32_t bytes4(float a, float b, float c, float d) {
  const uint32_t lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// q of 8 values of p, the slow and exact way.
__device__ __noinline__ uint2 divide8(uint4 h, uint4 g, float num, float den) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    mul2(widen2(word(h, i)), widen2(word(g, i))).get(a, b);
    const uint32_t qa = __float2int_rn(__fdiv_rn(num * a, den)) & 0xff, qb = __float2int_rn(__fdiv_rn(num * b, den)) & 0xff;
    w[i >> 1] |= (qa | (qb << 8)) << (16 * (i & 1));
  }
  return make_uint2(w[0], w[1]);
}

// MINB: CTAs on an SM that the registers must allow.  ROWS: rows of a CTA,
// one with all of its warps, or one for each warp (threadIdx.y).
template <int VPT, int MAXT, int MINB, int ROWS, bool NORM, bool I8>
__global__ void __launch_bounds__(MAXT, MINB) rmsnorm_kernel(const Args p) {
  __shared__ float red_s[MAXT / 32], red_a[MAXT / 32];
  __shared__ double red_d[MAXT / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = ROWS > 1 ? 1 : blockDim.x >> 5;
  const unsigned m = ROWS > 1 ? blockIdx.x * ROWS + threadIdx.y : blockIdx.x;
  if (ROWS > 1 && m >= static_cast<unsigned>(p.M)) return;   // no barrier follows with a row to each warp
  const size_t row = static_cast<size_t>(m) * p.d8;
  uint4 hv[VPT];
  {
    uint4 rv[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = tid + j * blockDim.x;
      hv[j] = rv[j] = make_uint4(0, 0, 0, 0);
      if (c < p.d8) {
        hv[j] = p.x[row + c];
        if (NORM && p.res != nullptr) rv[j] = p.res[row + c];
      }
    }
    if (NORM && p.res != nullptr) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = tid + j * blockDim.x;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = narrow2(add2(widen2(word(hv[j], i)), widen2(word(rv[j], i))));
        hv[j] = make_uint4(w[0], w[1], w[2], w[3]);
        if (p.h != nullptr && c < p.d8) p.h[row + c] = hv[j];
      }
    }
  }
  F2 s2(0.f, 0.f);
  float a = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = tid + j * blockDim.x;
    uint4 g = make_uint4(0, 0, 0, 0);
    if (NORM && I8 && c < p.d8) g = __ldg(p.gamma + c);
    __nv_bfloat162 m2 = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = word(hv[j], i);
      const F2 f = widen2(w);
      if (NORM) s2 = fma2(f, f, s2);
      if (I8 && !NORM) m2 = __hmax2_nan(m2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
    }
    if (I8 && NORM) a = join_max(a, hv[j], g);
    if (I8 && !NORM) a = max_nan(a, max_nan(__low2float(m2), __high2float(m2)));
  }
  float ss, s1;
  s2.get(ss, s1);
  ss += s1;
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    if (NORM) ss += __shfl_xor_sync(FULL, ss, off);
    if (I8) a = max_nan(a, __shfl_xor_sync(FULL, a, off));
  }
  if (nwarps > 1) {
    if (lane == 0) {
      red_s[warp] = ss;
      red_a[warp] = a;
    }
    __syncthreads();
    const int w = lane & (MAXT / 32 - 1);   // every group of MAXT / 32 lanes adds all warps'
    ss = w < nwarps ? red_s[w] : 0.f;
    a = w < nwarps ? red_a[w] : 0.f;
#pragma unroll
    for (int off = MAXT / 64; off; off >>= 1) {
      if (NORM) ss += __shfl_xor_sync(FULL, ss, off);
      if (I8) a = max_nan(a, __shfl_xor_sync(FULL, a, off));
    }
  }
  float r = 1.f;
  if (NORM) {
    if (ss < INFINITY) {
      r = rsqrtf(fmaf(ss, p.inv_d, p.eps));   // off by 2 units in the last place at most
    } else {
      // fp32 overflowed (or the row holds a NaN or an infinity), the same in every thread: again in fp64
      double s = 0.0;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float u, v;
          widen2(word(hv[j], i)).get(u, v);
          s = fma(static_cast<double>(u), static_cast<double>(u), fma(static_cast<double>(v), static_cast<double>(v), s));
        }
      }
#pragma unroll
      for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(FULL, s, off);
      if (nwarps > 1) {
        if (lane == 0) red_d[warp] = s;
        __syncthreads();
        s = 0.0;
        for (int w = 0; w < nwarps; ++w) s += red_d[w];
      }
      const double r64 = 1.0 / sqrt(s / (8 * p.d8) + static_cast<double>(p.eps));
      r = static_cast<float>(r64);
      if (!I8 || a == INFINITY) {   // a, the same in every thread, again too
        r = static_cast<float>(r64 * 0x1p66);
        a = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          const int c = tid + j * blockDim.x;
          const F2 k(0x1p-66f, 0x1p-66f);
          hv[j] = make_uint4(narrow2(mul2(widen2(hv[j].x), k)), narrow2(mul2(widen2(hv[j].y), k)),
                             narrow2(mul2(widen2(hv[j].z), k)), narrow2(mul2(widen2(hv[j].w), k)));
          if (I8 && c < p.d8) a = join_max(a, hv[j], __ldg(p.gamma + c));
        }
        if (I8) {
#pragma unroll
          for (int off = 16; off; off >>= 1) a = max_nan(a, __shfl_xor_sync(FULL, a, off));
          if (nwarps > 1) {
            if (lane == 0) red_a[warp] = a;   // the first ones were read before the last barrier
            __syncthreads();
            for (int w = 0; w < nwarps; ++w) a = max_nan(a, red_a[w]);
          }
        }
      }
    }
  }
  if (I8) {
    const bool bad = !(a < INFINITY);
    const bool zero = a < 7.8886091e-31f;   // 2^-100
    if (tid == 0) p.scale[m] = bad ? __int_as_float(0x7fc00000) : (zero ? 0.f : a * r / 127.f);
    const bool none = bad || zero;
    // 127 p must stay in fp32's range: both sides of the quotient times a power of two
    const float k = NORM && a > 1.2676506e30f ? 5.421010862e-20f : 1.f;   // 2^100, 2^-64
    const float num = 127.f * k, den = a * k;
    // the norm's is checked by its remainder, so that 1e-6 would do
    const float inv = none ? 0.f : (NORM ? num * __fdividef(1.f, den) : __fdiv_ru(127.f, a));
    const F2 inv2(inv, inv), num2(num, num), nden2(-den, -den), magic2(MAGIC, MAGIC), nmagic2(-MAGIC, -MAGIC);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = tid + j * blockDim.x;
      if (c >= p.d8) continue;
      if (none) {
        p.q[row + c] = make_uint2(0, 0);
        continue;
      }
      uint4 g = make_uint4(0, 0, 0, 0);
      if (NORM) g = __ldg(p.gamma + c);
      float t[8], worst = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        F2 v = widen2(word(hv[j], i));
        if (NORM) v = mul2(v, widen2(word(g, i)));
        const F2 tm = fma2(v, inv2, magic2);
        tm.get(t[2 * i], t[2 * i + 1]);
        if (NORM) {
          float e0, e1;
          fma2(add2(tm, nmagic2), nden2, mul2(v, num2)).get(e0, e1);
          worst = fmaxf(worst, fmaxf(fabsf(e0), fabsf(e1)));
        }
      }
      uint2 q = make_uint2(bytes4(t[0], t[1], t[2], t[3]), bytes4(t[4], t[5], t[6], t[7]));
      if (NORM && !(worst < 0.5f * den)) q = divide8(hv[j], g, num, den);
      p.q[row + c] = q;
    }
  } else {
    const F2 r2(r, r);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = tid + j * blockDim.x;
      if (c >= p.d8) continue;
      const uint4 g = __ldg(p.gamma + c);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = narrow2(mul2(mul2(widen2(word(hv[j], i)), widen2(word(g, i))), r2));
      p.y[row + c] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <int VPT, int MAXT, int MINB, int ROWS, bool NORM, bool I8>
static cudaError_t launch_as(const Args& a, cudaStream_t st) {
  const unsigned threads = ROWS > 1 ? 32 : ((a.d8 + VPT - 1) / VPT + 31) & ~31;
  const unsigned grid = (static_cast<unsigned>(a.M) + ROWS - 1) / ROWS;
  return launch_kernel(rmsnorm_kernel<VPT, MAXT, MINB, ROWS, NORM, I8>, dim3(grid), dim3(threads, ROWS), 0, st, a);
}

// At most one row per SM: one vector per thread ([8, 2560] int8 1.9 us; with two
// vectors 1.1 times that, with four 1.3).  More rows of up to 512 channels in the
// norm, 2048 in the quantiser: a warp each, eight in a CTA ([4352, 512] bf16 3.0
// us, with a CTA each 4.9; [70768, 384] to int8 20, with a CTA each 74, as fast as
// CTAs start; but [4352, 1024] in the norm 7.0 and 6.4).  Longer rows: two
// vectors in the norm ([512, 2560] int8 3.1 us, with one 1.3 times that, with
// four 1.2; [4352, 4096] int8 22, 1.6 and 1.05; bf16 23.7, 1.1, 1.02), four in the
// quantiser, which holds no sum and no residual ([151936, 2560] 191 us, with one
// 316, with two 207).
template <bool NORM, bool I8>
static int launch(const Args& a, cudaStream_t st) {
  cudaError_t e;
  if (a.d8 > 1024)
    e = launch_as<4, 1024, 1, 1, NORM, I8>(a, st);
  else if (a.M <= num_sms_current())
    e = launch_as<1, 1024, 1, 1, NORM, I8>(a, st);
  else if (a.d8 <= 32)
    e = launch_as<1, 256, 5, 8, NORM, I8>(a, st);
  else if (a.d8 <= 64)
    e = launch_as<2, 256, 5, 8, NORM, I8>(a, st);
  else if constexpr (NORM)
    e = launch_as<2, 512, 3, 1, NORM, I8>(a, st);
  else if (a.d8 <= 128)
    e = launch_as<4, 256, 5, 8, NORM, I8>(a, st);
  else if (a.d8 <= 256)
    e = launch_as<8, 256, 4, 8, NORM, I8>(a, st);
  else
    e = launch_as<4, 256, 5, 1, NORM, I8>(a, st);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

static bool misaligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

static bool bad_rows(int M, int d) { return M < 1 || d < 8 || d > MAX_D || d % 8 != 0; }

static bool bad_norm(const void* x, const void* residual, const void* gamma, float eps, int M, int d, const void* h) {
  if (!x || !gamma || bad_rows(M, d) || (h && !residual)) return true;
  if (!(eps >= 1e-20f) || !(eps < INFINITY)) return true;
  return misaligned(x, 16) || misaligned(residual, 16) || misaligned(gamma, 16) || misaligned(h, 16);
}

}  // namespace norm
}  // namespace dflash

extern "C" int dflash_rmsnorm(const dflash_bf16* x, const dflash_bf16* residual, const dflash_bf16* gamma, float eps,
                              int M, int d, dflash_bf16* h, dflash_bf16* y, void* stream) {
  using namespace dflash::norm;
  if (bad_norm(x, residual, gamma, eps, M, d, h) || !y || misaligned(y, 16) || y == h) return DFLASH_ERR_INVALID_ARG;
  Args a = {reinterpret_cast<const uint4*>(x), reinterpret_cast<const uint4*>(residual),
            reinterpret_cast<const uint4*>(gamma), reinterpret_cast<uint4*>(h), reinterpret_cast<uint4*>(y),
            nullptr, nullptr, eps, 1.f / static_cast<float>(d), d / 8, M};
  return launch<true, false>(a, static_cast<cudaStream_t>(stream));
}

extern "C" int dflash_rmsnorm_i8(const dflash_bf16* x, const dflash_bf16* residual, const dflash_bf16* gamma,
                                 float eps, int M, int d, dflash_bf16* h, int8_t* q, float* scale, void* stream) {
  using namespace dflash::norm;
  if (bad_norm(x, residual, gamma, eps, M, d, h) || !q || !scale || misaligned(q, 8) || misaligned(scale, 4))
    return DFLASH_ERR_INVALID_ARG;
  Args a = {reinterpret_cast<const uint4*>(x), reinterpret_cast<const uint4*>(residual),
            reinterpret_cast<const uint4*>(gamma), reinterpret_cast<uint4*>(h), nullptr,
            reinterpret_cast<uint2*>(q), scale, eps, 1.f / static_cast<float>(d), d / 8, M};
  return launch<true, true>(a, static_cast<cudaStream_t>(stream));
}

extern "C" int dflash_quant_i8(const dflash_bf16* x, int M, int d, int8_t* q, float* scale, void* stream) {
  using namespace dflash::norm;
  if (!x || !q || !scale || bad_rows(M, d) || misaligned(x, 16) || misaligned(q, 8) || misaligned(scale, 4))
    return DFLASH_ERR_INVALID_ARG;
  Args a = {reinterpret_cast<const uint4*>(x), nullptr, nullptr, nullptr, nullptr, reinterpret_cast<uint2*>(q),
            scale, 0.f, 0.f, d / 8, M};
  return launch<false, true>(a, static_cast<cudaStream_t>(stream));
}
