// Log-probabilities of given tokens, with entropy, rank and top alternatives.
//
//   lse = log sum exp(z/T),  logp = z_t/T - lse,  rank = 1 + #{z > z_t},
//   entropy = -sum p log p,  the K largest z (value desc, index asc)
//
// One pass over a row: each thread keeps a reference value `ref` (a maximum
// it has seen), s = sum exp2(t) and w = sum t exp2(t) with t = (z - ref) c,
// c = log2(e) / T, the count of values above z_t, and each warp keeps its K
// best entries sorted over its lanes.  The difference z - ref is taken first
// (exact near ref, where the terms that matter are), so values as large as
// the type's range need no care, and equal values give t = 0 exactly.
//
// c is rounded to fp32, i.e. the sums are those of a temperature off by a
// relative 2^-24; the log of the sum is corrected for that to first order with
// the mean of t, which the entropy needs anyway.
#include <cuda_bf16.h>

#include "common.cuh"

namespace dflash {
namespace lp {

constexpr unsigned FULL = 0xffffffffu;
constexpr int NT = 512;
constexpr int NW = NT / 32;
constexpr int MAX_K = 32;
constexpr int MAX_V = 1 << 24;
constexpr double LN2 = 0.69314718055994530942;

struct Args {
  const void* z;
  long long ld;
  int V;
  int K;
  float c;           // log2(e) / T in fp32
  double inv_t;      // 1 / T
  const int32_t* tokens;      // given tokens (or NULL)
  const int32_t* draft;       // emitted tokens: draft [B, L], accept_len, next_token [B]
  const int32_t* accept_len;
  const int32_t* next_token;
  int L;
  float* logp;
  int32_t* rank;
  float* entropy;
  float* lse;
  float* top_logp;
  int32_t* top_idx;
  int* status;
};

// (value, index) as one integer that orders as the alternatives do: larger
// value first, then the smaller index.  Never 0, so 0 is the empty entry.  -0
// counts as +0; a NaN as the largest value.
__device__ __forceinline__ uint64_t entry_of(float z, int idx) {
  const uint32_t b = __float_as_uint(z + 0.f);
  uint32_t key = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  if (z != z) key = 0xffffffffu;
  return (static_cast<uint64_t>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(idx));
}

__device__ __forceinline__ float value_of(uint64_t e) {
  const uint32_t key = static_cast<uint32_t>(e >> 32);
  return __uint_as_float((key & 0x80000000u) ? (key ^ 0x80000000u) : ~key);   // key 0xffffffff: a NaN
}

__device__ __forceinline__ int index_of(uint64_t e) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(e)); }

// A warp's best entries, sorted downwards over its lanes; kth = entry K - 1.
struct WarpTop {
  uint64_t ent, kth;

  // Every lane offers an entry (0: none).
  __device__ __forceinline__ void offer(uint64_t cand, int K, int lane) {
    unsigned todo = __ballot_sync(FULL, cand > kth);
    while (todo) {
      const uint64_t c = __shfl_sync(FULL, cand, __ffs(todo) - 1);
      const int pos = __popc(__ballot_sync(FULL, ent > c));
      const uint64_t up = __shfl_up_sync(FULL, ent, 1);
      ent = lane < pos ? ent : (lane == pos ? c : up);
      kth = __shfl_sync(FULL, ent, K - 1);
      todo &= todo - 1;
      todo &= __ballot_sync(FULL, cand > kth);
    }
  }
};

__device__ __forceinline__ float load(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }

// The token asked for in a row, and whether the row is asked for at all.
__device__ __forceinline__ bool row_token(const Args& p, int row, int& token) {
  token = -1;
  if (p.accept_len != nullptr) {
    const int b = row / (p.L + 1), i = row - b * (p.L + 1);
    int n = p.accept_len[b];
    if (n < 1 || n > p.L + 1) {
      if (threadIdx.x == 0) set_status(p.status, DFLASH_ERR_BAD_INDEX);
      n = n < 1 ? 1 : p.L + 1;
    }
    if (i >= n) return false;
    token = i == n - 1 ? p.next_token[b] : p.draft[static_cast<size_t>(b) * p.L + i];
    if (token < 0) token = 0x7fffffff;   // out of range, not padding
    return true;
  }
  if (p.tokens != nullptr) {
    token = p.tokens[row];
    return token >= 0;
  }
  return true;
}

template <typename Z>
__global__ void __launch_bounds__(NT) logprobs_kernel(const Args p) {
  __shared__ float sh_ref[NW];
  __shared__ double sh_s[NW], sh_w[NW];
  __shared__ int sh_cnt[NW];
  __shared__ uint64_t sh_top[NW * 32];
  __shared__ double sh_log;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x;
  int token;
  if (!row_token(p, row, token)) return;
  const Z* z = static_cast<const Z*>(p.z) + static_cast<size_t>(row) * p.ld;
  const bool bad_token = token >= p.V;
  if (bad_token && tid == 0) set_status(p.status, DFLASH_ERR_BAD_INDEX);
  const float zt = token >= 0 && !bad_token ? load(z + token) : 0.f;

  float ref = -INFINITY, s = 0.f, w = 0.f;
  int cnt = 0;
  WarpTop top{0, 0};
  for (int v0 = 0; v0 < p.V; v0 += NT) {
    const int v = v0 + tid;
    const float x = v < p.V ? load(z + v) : -INFINITY;
    if (x > ref) {
      if (ref != -INFINITY) {
        const float dlt = (ref - x) * p.c;
        const float f = exp2f(dlt);
        w = f > 0.f ? f * (w + dlt * s) : 0.f;
        s *= f;
      }
      ref = x;
    }
    const float t = ref == -INFINITY ? (x != x ? x : -INFINITY) : (x - ref) * p.c;
    const float e = exp2f(t);
    s += e;
    w += e == 0.f ? 0.f : e * t;
    cnt += x > zt ? 1 : 0;
    if (p.K > 0) top.offer(v < p.V ? entry_of(x, v) : 0, p.K, lane);
  }
  // one reference for the row, then the sums in fp64
  float m = ref;
#pragma unroll
  for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, off));
  if (lane == 0) sh_ref[warp] = m;
  sh_top[tid] = top.ent;
  __syncthreads();
  for (int k = 0; k < NW; ++k) m = fmaxf(m, sh_ref[k]);
  double sd = s, wd = w;
  if (ref != -INFINITY) {
    const double dlt = (static_cast<double>(ref) - m) * p.c;   // NaN where both are +inf
    const double f = exp2(dlt);
    wd = f == 0.0 ? 0.0 : f * (wd + dlt * sd);
    sd *= f;
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    sd += __shfl_xor_sync(FULL, sd, off);
    wd += __shfl_xor_sync(FULL, wd, off);
    cnt += __shfl_xor_sync(FULL, cnt, off);
  }
  if (lane == 0) {
    sh_s[warp] = sd;
    sh_w[warp] = wd;
    sh_cnt[warp] = cnt;
  }
  __syncthreads();
  if (tid == 0) {
    sd = wd = 0.0;
    cnt = 0;
    for (int k = 0; k < NW; ++k) {
      sd += sh_s[k];
      wd += sh_w[k];
      cnt += sh_cnt[k];
    }
    const bool dead = m == -INFINITY && sd == 0.0;
    const double c = p.c;
    const double mean_t = wd / sd;
    // log of the sum relative to the maximum: every result is a difference to
    // the maximum plus this, which holds even where lse itself is near the
    // type's lowest value
    const double log_s = dead ? 0.0 : log(sd) + (p.inv_t - c * LN2) * (mean_t / c);
    const double ent = dead ? 0.0 : log(sd) - mean_t * LN2;
    sh_log = log_s;
    if (p.lse != nullptr) p.lse[row] = static_cast<float>(dead ? -INFINITY : m * p.inv_t + log_s);
    if (p.entropy != nullptr) p.entropy[row] = static_cast<float>(ent);
    if (p.logp != nullptr) {
      const double v = dead ? -INFINITY : (static_cast<double>(zt) - m) * p.inv_t - log_s;
      p.logp[row] = bad_token ? __int_as_float(0x7fc00000) : static_cast<float>(v);
    }
    if (p.rank != nullptr) p.rank[row] = bad_token ? 0 : cnt + 1;
  }
  __syncthreads();
  if (p.K > 0) {
    // each warp entry's place among all of them
    const uint64_t mine = sh_top[tid];
    if (mine != 0) {
      int place = 0;
      for (int k = 0; k < NT; ++k) place += sh_top[k] > mine ? 1 : 0;
      if (place < p.K) {
        const size_t o = static_cast<size_t>(row) * p.K + place;
        const double v = m == -INFINITY ? value_of(mine) + sh_log : (static_cast<double>(value_of(mine)) - m) * p.inv_t - sh_log;
        p.top_logp[o] = static_cast<float>(v);
        p.top_idx[o] = index_of(mine);
      }
    }
  }
}

static int launch(Args& a, int z_bf16, int rows, float temperature, cudaStream_t st) {
  if (!a.z || (z_bf16 & ~1) || a.V < 1 || a.V > MAX_V || a.ld < a.V || a.K < 0 || a.K > MAX_K || a.K > a.V)
    return DFLASH_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || !(temperature < INFINITY)) return DFLASH_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(a.z) & (z_bf16 ? 1 : 3)) return DFLASH_ERR_INVALID_ARG;
  if ((a.top_logp == nullptr) != (a.top_idx == nullptr) || (a.top_logp != nullptr && a.K == 0))
    return DFLASH_ERR_INVALID_ARG;
  if (a.top_logp == nullptr) a.K = 0;
  a.inv_t = 1.0 / static_cast<double>(temperature);
  a.c = static_cast<float>(1.4426950408889634 / static_cast<double>(temperature));
  if (!(a.c > 0.f) || !(a.c < INFINITY)) return DFLASH_ERR_INVALID_ARG;
  const dim3 grid(static_cast<unsigned>(rows)), block(NT);
  const cudaError_t e = z_bf16 ? launch_kernel(logprobs_kernel<__nv_bfloat16>, grid, block, 0, st, a)
                               : launch_kernel(logprobs_kernel<float>, grid, block, 0, st, a);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // namespace lp
}  // namespace dflash

extern "C" int dflash_token_logprobs(const void* logits, int z_bf16, long long ld, int M, int V, const int32_t* tokens,
                                     float temperature, int K, float* logp, int32_t* rank, float* entropy, float* lse,
                                     float* top_logp, int32_t* top_idx, int* dev_status, void* stream) {
  if (M < 1 || (!tokens && (logp || rank))) return DFLASH_ERR_INVALID_ARG;
  dflash::lp::Args a = {};
  a.z = logits;
  a.ld = ld;
  a.V = V;
  a.K = K;
  a.tokens = tokens;
  a.logp = logp;
  a.rank = rank;
  a.entropy = entropy;
  a.lse = lse;
  a.top_logp = top_logp;
  a.top_idx = top_idx;
  a.status = dev_status;
  return dflash::lp::launch(a, z_bf16, M, temperature, static_cast<cudaStream_t>(stream));
}

extern "C" int dflash_emitted_logprobs(const void* target_logits, int z_bf16, long long ld, int B, int L, int V,
                                       const int32_t* draft, const int32_t* accept_len, const int32_t* next_token,
                                       float temperature, int K, float* logp, int32_t* rank, float* entropy,
                                       float* lse, float* top_logp, int32_t* top_idx, int* dev_status, void* stream) {
  if (!draft || !accept_len || !next_token || B < 1 || L < 1 || L > 32 || B > 0x7fffffff / (L + 1))
    return DFLASH_ERR_INVALID_ARG;
  dflash::lp::Args a = {};
  a.z = target_logits;
  a.ld = ld;
  a.V = V;
  a.K = K;
  a.draft = draft;
  a.accept_len = accept_len;
  a.next_token = next_token;
  a.L = L;
  a.logp = logp;
  a.rank = rank;
  a.entropy = entropy;
  a.lse = lse;
  a.top_logp = top_logp;
  a.top_idx = top_idx;
  a.status = dev_status;
  return dflash::lp::launch(a, z_bf16, B * (L + 1), temperature, static_cast<cudaStream_t>(stream));
}
