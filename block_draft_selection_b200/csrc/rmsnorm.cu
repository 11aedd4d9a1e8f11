// Root-mean-square norm with the residual's addition, and rows to int8.
//
//   h = bf16(x + residual),  r = 1 / sqrt(mean h^2 + eps),  y = h gamma r
//   int8: a = max |h gamma|, scale = a r / 127, q = rint(127 h gamma / a)
//
// One CTA per row; the row stays in registers (VPT vectors of 8 channels per
// thread), so every input byte is read once.  r cancels in q, so the sum of
// squares and the maximum come out of one block reduction and nothing waits
// for r before the second pass over the registers.
//
// q is decided exactly.  h and gamma are bf16, so p = h * gamma has at most 16
// significant bits and both p and 127 p are exact in fp32.  The quotient
// 127 p / a differs from a halfway point k + 1/2, where it is not one, by a
// relative 2^-15 / 254 or more (numerator and denominator are multiples of
// 2^-15 of their leading bits), i.e. 1.2e-7, above the 2^-24 of a correctly
// rounded division: rounding the IEEE quotient gives what rounding the real
// one gives.  Without gamma (dflash_quant_i8) the operands have 8 bits and the
// nearest miss is 2^-9 / 127 of q away, so a product with 127 / a decides as
// exactly, provided that true halves stay halves or err upwards: those are
// x = a/2 (q = 63.5, even neighbour 64) and, where a is 127 times a power of
// two, exact products.  127 / a is therefore rounded up.
#include <cuda_bf16.h>

#include "common.cuh"

namespace dflash {
namespace norm {

constexpr unsigned FULL = 0xffffffffu;
constexpr int MAX_D = 32768;

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t lo = __bfloat16_as_ushort(__float2bfloat16_rn(f[2 * k]));
    const uint32_t hi = __bfloat16_as_ushort(__float2bfloat16_rn(f[2 * k + 1]));
    w[k] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The larger one; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct Args {
  const uint4* x;
  const uint4* res;
  const uint4* gamma;
  uint4* h;
  uint4* y;
  uint2* q;
  float* scale;
  float eps;
  int d8;
};

template <int VPT, bool NORM, bool I8>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const Args p) {
  __shared__ float red_s[32], red_a[32];
  __shared__ double red_d[32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = blockDim.x >> 5;
  const size_t row = static_cast<size_t>(blockIdx.x) * p.d8;
  uint4 hv[VPT];
  float ss = 0.f, a = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = tid + j * blockDim.x;
    hv[j] = make_uint4(0, 0, 0, 0);
    if (c < p.d8) {
      hv[j] = p.x[row + c];
      float f[8];
      unpack8(hv[j], f);
      if (NORM && p.res != nullptr) {
        float g[8];
        unpack8(p.res[row + c], g);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] += g[k];
        hv[j] = pack8(f);
        if (p.h != nullptr) p.h[row + c] = hv[j];
        unpack8(hv[j], f);
      }
      if (NORM) {
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(f[k], f[k], ss);
      }
      if (I8) {
        if (NORM) {
          float g[8];
          unpack8(__ldg(p.gamma + c), g);
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] *= g[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) a = max_nan(a, fabsf(f[k]));
      }
    }
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    if (NORM) ss += __shfl_xor_sync(FULL, ss, off);
    if (I8) a = max_nan(a, __shfl_xor_sync(FULL, a, off));
  }
  if (lane == 0) {
    red_s[warp] = ss;
    red_a[warp] = a;
  }
  __syncthreads();
  ss = 0.f;
  a = 0.f;
  for (int w = 0; w < nwarps; ++w) {
    if (NORM) ss += red_s[w];
    if (I8) a = max_nan(a, red_a[w]);
  }
  const int d = p.d8 * 8;
  float r = 1.f;
  if (NORM) {
    if (ss < INFINITY) {
      r = 1.f / sqrtf(ss / static_cast<float>(d) + p.eps);
    } else {
      // fp32 overflowed (or the row holds a NaN or an infinity): again in fp64
      double s = 0.0;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float f[8];
        unpack8(hv[j], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) s = fma(static_cast<double>(f[k]), static_cast<double>(f[k]), s);
      }
#pragma unroll
      for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(FULL, s, off);
      if (lane == 0) red_d[warp] = s;
      __syncthreads();   // uniform: every thread holds the same ss
      s = 0.0;
      for (int w = 0; w < nwarps; ++w) s += red_d[w];
      r = static_cast<float>(1.0 / sqrt(s / d + static_cast<double>(p.eps)));
    }
  }
  if (I8) {
    const bool bad = !(a < INFINITY);
    const bool zero = a < 7.8886091e-31f;   // 2^-100
    if (tid == 0) p.scale[blockIdx.x] = bad ? __int_as_float(0x7fc00000) : (zero ? 0.f : a * r / 127.f);
    const bool none = bad || zero;
    const float inv = NORM || none ? 0.f : __fdiv_ru(127.f, a);
    // 127 p must stay in fp32's range: both sides of the quotient times a power of two
    const float k = a > 1.2676506e30f ? 5.421010862e-20f : 1.f;   // 2^100, 2^-64
    const float num = 127.f * k, den = a * k;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = tid + j * blockDim.x;
      if (c < p.d8) {
        float f[8];
        unpack8(hv[j], f);
        uint32_t w[2] = {0, 0};
        if (!none) {
          float g[8];
          if (NORM) unpack8(__ldg(p.gamma + c), g);
#pragma unroll
          for (int c8 = 0; c8 < 8; ++c8) {
            const float t = NORM ? __fdiv_rn(num * (f[c8] * g[c8]), den) : f[c8] * inv;
            w[c8 >> 2] |= (static_cast<uint32_t>(__float2int_rn(t)) & 0xffu) << (8 * (c8 & 3));
          }
        }
        p.q[row + c] = make_uint2(w[0], w[1]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = tid + j * blockDim.x;
      if (c < p.d8) {
        float f[8], g[8];
        unpack8(hv[j], f);
        unpack8(__ldg(p.gamma + c), g);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = f[k] * g[k] * r;
        p.y[row + c] = pack8(f);
      }
    }
  }
}

template <bool NORM, bool I8>
static int launch(const Args& a, int M, cudaStream_t st) {
  const int vpt = a.d8 <= 512 ? 1 : (a.d8 <= 1024 ? 2 : 4);
  const int threads = ((a.d8 + vpt - 1) / vpt + 31) & ~31;
  const dim3 grid(static_cast<unsigned>(M)), block(static_cast<unsigned>(threads));
  cudaError_t e;
  if (vpt == 1)
    e = launch_kernel(rmsnorm_kernel<1, NORM, I8>, grid, block, 0, st, a);
  else if (vpt == 2)
    e = launch_kernel(rmsnorm_kernel<2, NORM, I8>, grid, block, 0, st, a);
  else
    e = launch_kernel(rmsnorm_kernel<4, NORM, I8>, grid, block, 0, st, a);
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
            nullptr, nullptr, eps, d / 8};
  return launch<true, false>(a, M, static_cast<cudaStream_t>(stream));
}

extern "C" int dflash_rmsnorm_i8(const dflash_bf16* x, const dflash_bf16* residual, const dflash_bf16* gamma,
                                 float eps, int M, int d, dflash_bf16* h, int8_t* q, float* scale, void* stream) {
  using namespace dflash::norm;
  if (bad_norm(x, residual, gamma, eps, M, d, h) || !q || !scale || misaligned(q, 8) || misaligned(scale, 4))
    return DFLASH_ERR_INVALID_ARG;
  Args a = {reinterpret_cast<const uint4*>(x), reinterpret_cast<const uint4*>(residual),
            reinterpret_cast<const uint4*>(gamma), reinterpret_cast<uint4*>(h), nullptr,
            reinterpret_cast<uint2*>(q), scale, eps, d / 8};
  return launch<true, true>(a, M, static_cast<cudaStream_t>(stream));
}

extern "C" int dflash_quant_i8(const dflash_bf16* x, int M, int d, int8_t* q, float* scale, void* stream) {
  using namespace dflash::norm;
  if (!x || !q || !scale || bad_rows(M, d) || misaligned(x, 16) || misaligned(q, 8) || misaligned(scale, 4))
    return DFLASH_ERR_INVALID_ARG;
  Args a = {reinterpret_cast<const uint4*>(x), nullptr, nullptr, nullptr, nullptr, reinterpret_cast<uint2*>(q),
            scale, 0.f, d / 8};
  return launch<false, true>(a, M, static_cast<cudaStream_t>(stream));
}
