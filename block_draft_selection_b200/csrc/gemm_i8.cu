// Matrix product in 8-bit integers with a scale per token and per channel:
//   C[m,n] = float(sum_k A[m,k] B[n,k]) * sa[m] * sb[n]
#include <cuda_bf16.h>

#include "common.cuh"

namespace dflash {
namespace gi8 {

constexpr int T = 64;      // tile of C, and bytes of K per step
constexpr int MAX_K = 131071;   // 128 * 128 * K stays below 2^31

__device__ __forceinline__ void put(float* c, size_t i, float v) { c[i] = v; }
__device__ __forceinline__ void put(__nv_bfloat16* c, size_t i, float v) { c[i] = __float2bfloat16_rn(v); }

template <typename OUT>
__global__ void __launch_bounds__(256) gemm_i8_kernel(const int8_t* __restrict__ A, const float* __restrict__ sa,
                                                      const int8_t* __restrict__ B, const float* __restrict__ sb,
                                                      OUT* __restrict__ C, int M, int N, int K) {
  __shared__ int as[T][T / 4 + 1], bs[T][T / 4 + 1];
  pdl_wait();
  pdl_trigger();
  const int n_tiles = (N + T - 1) / T;
  const int mt = blockIdx.x / n_tiles, nt = blockIdx.x - mt * n_tiles;
  const int tid = threadIdx.x, ti = tid >> 4, tj = tid & 15;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += T) {
    const int r = tid >> 2, c = (tid & 3) * 16;
    int4 a = make_int4(0, 0, 0, 0), b = a;
    if (mt * T + r < M && k0 + c < K)
      a = __ldg(reinterpret_cast<const int4*>(A + static_cast<size_t>(mt * T + r) * K + k0 + c));
    if (nt * T + r < N && k0 + c < K)
      b = __ldg(reinterpret_cast<const int4*>(B + static_cast<size_t>(nt * T + r) * K + k0 + c));
    const int w = (tid & 3) * 4;
    as[r][w] = a.x; as[r][w + 1] = a.y; as[r][w + 2] = a.z; as[r][w + 3] = a.w;
    bs[r][w] = b.x; bs[r][w + 1] = b.y; bs[r][w + 2] = b.z; bs[r][w + 3] = b.w;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < T / 4; ++k) {
      int av[4], bv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        av[i] = as[ti + 16 * i][k];
        bv[i] = bs[tj + 16 * i][k];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(av[i], bv[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = mt * T + ti + 16 * i, n = nt * T + tj + 16 * j;
      if (m < M && n < N) put(C, static_cast<size_t>(m) * N + n, __int2float_rn(acc[i][j]) * sa[m] * sb[n]);
    }
}

}  // namespace gi8
}  // namespace dflash

extern "C" int dflash_gemm_i8(const int8_t* A, const float* sa, const int8_t* B, const float* sb, void* C, int c_bf16,
                              int M, int N, int K, int* dev_status, void* stream) {
  using namespace dflash::gi8;
  (void)dev_status;
  if (!A || !sa || !B || !sb || !C || M < 1 || N < 1 || K < 16 || K > MAX_K || K % 16 != 0 || (c_bf16 & ~1))
    return DFLASH_ERR_INVALID_ARG;
  auto mis = [](const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; };
  if (mis(A, 16) || mis(B, 16) || mis(sa, 4) || mis(sb, 4) || mis(C, c_bf16 ? 2 : 4)) return DFLASH_ERR_INVALID_ARG;
  const long long tiles = static_cast<long long>((M + T - 1) / T) * ((N + T - 1) / T);
  if (tiles > 0x7fffffffLL) return DFLASH_ERR_UNSUPPORTED;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(tiles)), block(256);
  const cudaError_t e =
      c_bf16 ? dflash::launch_kernel(gemm_i8_kernel<__nv_bfloat16>, grid, block, 0, st, A, sa, B, sb,
                                     static_cast<__nv_bfloat16*>(C), M, N, K)
             : dflash::launch_kernel(gemm_i8_kernel<float>, grid, block, 0, st, A, sa, B, sb, static_cast<float*>(C),
                                     M, N, K);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
