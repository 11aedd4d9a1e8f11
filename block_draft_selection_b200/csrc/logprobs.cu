// Log-probabilities of given tokens, with entropy, rank and top alternatives.
//
//   lse = log sum exp(z/T),  logp = z_t/T - lse,  rank = 1 + #{z > z_t},
//   entropy = -sum p log p,  the K largest z (value desc, index asc)
//
// One pass over a row, which a cluster of Q CTAs shares (Q chosen so that few
// rows still fill the GPU).  Each thread keeps a reference value `ref` (a
// value near the largest it has seen), s = sum exp2(t) and w = sum t exp2(t)
// with t = (z - ref) c, c = log2(e) / T, and the count of values above z_t.
// The difference z - ref is taken first (exact near ref, where the terms that
// matter are), so values as large as the type's range need no care, and equal
// values give t = 0 exactly.  ref moves only when a value exceeds it by more
// than LAG / c: terms up to 2^LAG cost no precision, and rescaling is rare.
//
// c is rounded to fp32, i.e. the sums are those of a temperature off by a
// relative 2^-24; the log of the sum is corrected for that to first order with
// the mean of t, which the entropy needs anyway.
//
// Alternatives: K threads whose maxima are at least tau prove that the K-th
// largest value is at least tau.  Each warp's ceil(K / 16)-th largest thread
// maximum, and of those the least, is such a tau; it is found after rounds 1,
// 2, 4, 8, ... of the loop from the running maxima, and a value below it costs
// no more than the comparison of its round's maximum.  The few others (about
// 70 a doubling on unsorted rows) go into their warp's list, sorted over the
// lanes.  At the end the lists' entries above the last tau are ranked by
// counting, first in each CTA, then in the cluster's first CTA, to which the
// others write theirs through distributed shared memory.
#include <cuda_bf16.h>

#include "common.cuh"

namespace dflash {
namespace lp {

constexpr unsigned FULL = 0xffffffffu;
constexpr int NT = 512;
constexpr int NW = NT / 32;
constexpr int MAX_K = 32;
constexpr int MAX_V = 1 << 24;
constexpr int MAX_Q = 16;           // CTAs that share a row: a cluster
constexpr int ELEMS = 16;           // logits per thread and round
constexpr float LAG = 64.f;
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
  int Q;
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

// 16-byte vectors of logits.
template <typename Z>
struct Vec;

template <>
struct Vec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float* x) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ float load(const float* p) { return __ldg(p); }
  static __device__ __forceinline__ uint32_t bits(const float* p) { return __float_as_uint(__ldg(p)); }
};

template <>
struct Vec<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }
};

// Elements [e0, e0 + E) of a row of V, -inf for those outside it: one 16-byte
// load, or single ones for the vectors that reach over an end of the row.
template <typename Z>
__device__ __forceinline__ uint4 load_vec(const Z* z, int e0, int V) {
  constexpr int E = Vec<Z>::E;
  if (e0 >= 0 && e0 + E <= V) return __ldg(reinterpret_cast<const uint4*>(z + e0));
  uint32_t w[4];
  if constexpr (E == 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = e0 + k;
      w[k] = e >= 0 && e < V ? Vec<Z>::bits(z + e) : 0xff800000u;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = e0 + 2 * k;
      const uint32_t lo = e >= 0 && e < V ? __bfloat16_as_ushort(__ldg(z + e)) : 0xff80u;
      const uint32_t hi = e + 1 >= 0 && e + 1 < V ? __bfloat16_as_ushort(__ldg(z + e + 1)) : 0xff80u;
      w[k] = lo | (hi << 16);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The larger one; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t key_of(float z) { return static_cast<uint32_t>(entry_of(z, 0) >> 32); }

__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// Sums relative to a reference: s = sum 2^t, w = sum t 2^t, t = (z - m) c.
struct Sums {
  float m;
  int cnt;
  double s, w;

  // Over the warp: relative to the largest reference, then added in fp64.
  __device__ __forceinline__ void reduce(float c) {
    float big = m;
#pragma unroll
    for (int off = 16; off; off >>= 1) big = fmaxf(big, __shfl_xor_sync(FULL, big, off));
    if (m != -INFINITY && m != big) {   // with m = -inf the sums are 0 (or NaN)
      const float d = (m - big) * c;
      const double f = ex2(d);
      w = f > 0.0 ? f * (w + d * s) : s * 0.0;
      s *= f;
    }
    m = big;
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      s += __shfl_xor_sync(FULL, s, off);
      w += __shfl_xor_sync(FULL, w, off);
      cnt += __shfl_xor_sync(FULL, cnt, off);
    }
  }
};

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

// Shared memory of a CTA; `all` and `sums` of the cluster's first CTA take
// every CTA's list and sums.
struct Shared {
  uint64_t list[NW * 32];           // entries to be ranked
  uint64_t all[MAX_Q * MAX_K];      // [CTA][K], sorted downwards, 0 past the end
  Sums sums[MAX_Q];
  Sums part[NW];
  uint32_t tau[2][NW];
  int n;
  int n_all;
  double log_s;
};

// Rank the n entries of `list` by counting and hand each with its rank to put.
template <typename F>
__device__ __forceinline__ void rank_entries(const uint64_t* list, int n, int K, F put) {
  for (int i = threadIdx.x; i < n; i += NT) {
    const uint64_t mine = list[i];
    int rank = 0;
    for (int k = 0; k < n; ++k) rank += list[k] > mine ? 1 : 0;
    if (rank < K) put(rank, mine);
  }
}

template <typename Z>
__global__ void __launch_bounds__(NT, 2) logprobs_kernel(const Args p) {
  constexpr int E = Vec<Z>::E;
  constexpr int U = ELEMS / E;      // vectors per thread and round
  __shared__ Shared sh;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Q = p.Q, row = blockIdx.x / Q, q = blockIdx.x - row * Q;
  int token;
  if (!row_token(p, row, token)) return;   // the same for every CTA of the cluster
  // remote stores wait until every CTA of the cluster has started
  if (Q > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const Z* z = static_cast<const Z*>(p.z) + static_cast<size_t>(row) * p.ld;
  const bool bad_token = token >= p.V;
  if (bad_token && tid == 0 && q == 0) set_status(p.status, DFLASH_ERR_BAD_INDEX);

  // the row as 16-byte vectors from the boundary at or before its start
  const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(Z));
  const int n_vec = (p.V + lead + E - 1) / E;
  const int v_begin = static_cast<int>(static_cast<long long>(q) * n_vec / Q);
  const int v_end = static_cast<int>(static_cast<long long>(q + 1) * n_vec / Q);
  const int rounds = (v_end - v_begin + U * NT - 1) / (U * NT);
  const uint32_t fill = E == 4 ? 0xff800000u : 0xff80ff80u;
  uint4 nxt[U];
  auto fetch = [&](int r) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = v_begin + (r * U + u) * NT + tid;
      nxt[u] = v < v_end ? load_vec(z, v * E - lead, p.V) : make_uint4(fill, fill, fill, fill);
    }
  };
  fetch(0);
  const float zt = token >= 0 && !bad_token ? Vec<Z>::load(z + token) : 0.f;
  if (tid == 0) sh.n = sh.n_all = 0;

  float ref = -INFINITY, s = 0.f, w = 0.f, top_seen = -INFINITY, tau = -INFINITY;
  int cnt = 0;
  WarpTop top{0, 0};
  int refreshed = 0;
  auto refresh = [&]() {
    const uint32_t key = key_of(top_seen);
    uint32_t k = __reduce_max_sync(FULL, key);
    if (p.K > NW) {   // the second largest
      const bool first = lane == __ffs(__ballot_sync(FULL, key == k)) - 1;
      k = __reduce_max_sync(FULL, first ? 0u : key);
    }
    uint32_t* t = sh.tau[refreshed++ & 1];
    if (lane == 0) t[warp] = k;
    __syncthreads();
    k = __reduce_min_sync(FULL, t[lane & (NW - 1)]);
    tau = value_of(static_cast<uint64_t>(k) << 32);
  };

  for (int r = 0; r < rounds; ++r) {
    float x[ELEMS];
#pragma unroll
    for (int u = 0; u < U; ++u) Vec<Z>::unpack(nxt[u], x + u * E);
    if (r + 1 < rounds) fetch(r + 1);
    float gm[4];   // maxima of groups of four vectors' worth of a quarter of the round
#pragma unroll
    for (int g = 0; g < 4; ++g)
      gm[g] = max_nan(max_nan(x[4 * g], x[4 * g + 1]), max_nan(x[4 * g + 2], x[4 * g + 3]));
    const float m = max_nan(max_nan(gm[0], gm[1]), max_nan(gm[2], gm[3]));
    top_seen = fmaxf(top_seen, m);
    if (m > ref) {
      if (ref == -INFINITY) {
        ref = m;
      } else if ((m - ref) * p.c > LAG) {
        const float d = (ref - m) * p.c;
        const float f = ex2(d);
        w = f > 0.f ? f * (w + d * s) : s * 0.f;
        s *= f;
        ref = m;
      }
    }
    const float base = ref == -INFINITY ? 0.f : ref;
    float es[4], ws[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      es[g] = ws[g] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // a masked value's t = -inf would make 0 * t a NaN; 2^-200 is 0
        const float t = max_nan((x[4 * g + j] - base) * p.c, -200.f);
        const float e = ex2(t);
        es[g] += e;
        ws[g] = fmaf(e, t, ws[g]);
        cnt += x[4 * g + j] > zt ? 1 : 0;
      }
    }
    s += (es[0] + es[1]) + (es[2] + es[3]);
    w += (ws[0] + ws[1]) + (ws[2] + ws[3]);
    if (p.K > 0) {
      if ((r & (r + 1)) == 0) refresh();
      if (__any_sync(FULL, !(m < tau))) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (__any_sync(FULL, !(gm[g] < tau))) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int el = 4 * g + j;
              const int v = v_begin + (r * U + el / E) * NT + tid;
              const int idx = v * E - lead + el % E;
              const bool real = v < v_end && idx >= 0 && idx < p.V;
              top.offer(real && !(x[el] < tau) ? entry_of(x[el], idx) : 0, p.K, lane);
            }
          }
        }
      }
    }
  }

  // sums of the warp, then of the CTA
  Sums sum{ref, cnt, s, w};
  sum.reduce(p.c);
  if (lane == 0) sh.part[warp] = sum;
  if (p.K > 0) {
    refresh();
    if (top.ent != 0 && static_cast<uint32_t>(top.ent >> 32) >= key_of(tau)) sh.list[atomicAdd(&sh.n, 1)] = top.ent;
  }
  __syncthreads();
  if (Q > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const uint32_t lead_all = Q > 1 ? mapa_shared(smem_addr(sh.all + q * MAX_K), 0) : smem_addr(sh.all);
  if (warp == 0) {
    sum = lane < NW ? sh.part[lane] : Sums{-INFINITY, 0, 0.0, 0.0};
    sum.reduce(p.c);
    if (lane == 0) {
      if (Q > 1) {
        const uint32_t to = mapa_shared(smem_addr(sh.sums + q), 0);
        const uint64_t* from = reinterpret_cast<const uint64_t*>(&sum);
#pragma unroll
        for (int k = 0; k < static_cast<int>(sizeof(Sums) / 8); ++k) st_cluster_u64(to + 8 * k, from[k]);
      } else {
        sh.sums[0] = sum;
      }
    }
  }
  if (p.K > 0) {
    const int n = sh.n;
    auto put = [&](int rank, uint64_t e) {
      if (Q > 1)
        st_cluster_u64(lead_all + 8 * rank, e);
      else
        sh.all[rank] = e;
    };
    rank_entries(sh.list, n, p.K, put);
    if (tid >= n && tid < p.K) put(tid, 0);
  }
  if (Q > 1) {
    cluster_sync_all();
    if (q != 0) return;
  } else {
    __syncthreads();
  }

  // the row: sums of its CTAs by warp 0, alternatives by the others
  if (warp == 0) {
    sum = lane < Q ? sh.sums[lane] : Sums{-INFINITY, 0, 0.0, 0.0};
    sum.reduce(p.c);
    if (lane == 0) {
      const double c = p.c;
      const bool dead = sum.m == -INFINITY && sum.s == 0.0;
      const double mean_t = sum.w / sum.s;
      const double log_sum = log(sum.s);
      // log of the sum relative to the maximum: every result is a difference
      // to the reference plus this, which holds even where lse itself is near
      // the type's lowest value
      const double log_s = dead ? 0.0 : log_sum + (p.inv_t - c * LN2) * (mean_t / c);
      sh.log_s = log_s;
      sh.part[0].m = sum.m;
      if (p.lse != nullptr) p.lse[row] = static_cast<float>(dead ? -INFINITY : sum.m * p.inv_t + log_s);
      if (p.entropy != nullptr) p.entropy[row] = static_cast<float>(dead ? 0.0 : log_sum - mean_t * LN2);
      if (p.logp != nullptr) {
        const double v = dead ? -INFINITY : (static_cast<double>(zt) - sum.m) * p.inv_t - log_s;
        p.logp[row] = bad_token ? __int_as_float(0x7fc00000) : static_cast<float>(v);
      }
      if (p.rank != nullptr) p.rank[row] = bad_token ? 0 : sum.cnt + 1;
    }
  }
  if (p.K == 0) return;
  if (Q > 1) {
    // the largest of the CTAs' K-th entries bounds the row's from below
    uint64_t bound = lane < Q ? sh.all[lane * MAX_K + p.K - 1] : 0;
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      const uint64_t o = __shfl_xor_sync(FULL, bound, off);
      bound = o > bound ? o : bound;
    }
    if (tid < Q * MAX_K && (tid & (MAX_K - 1)) < p.K) {
      const uint64_t e = sh.all[tid];
      if (e != 0 && e >= bound) sh.list[atomicAdd(&sh.n_all, 1)] = e;
    }
  }
  __syncthreads();
  const double log_s = sh.log_s;
  const float m = sh.part[0].m;
  auto out = [&](int rank, uint64_t e) {
    const float v = value_of(e);
    const size_t o = static_cast<size_t>(row) * p.K + rank;
    p.top_logp[o] =
        static_cast<float>(m == -INFINITY ? v + log_s : (static_cast<double>(v) - m) * p.inv_t - log_s);
    p.top_idx[o] = index_of(e);
  };
  if (Q > 1)
    rank_entries(sh.list, sh.n_all, p.K, out);
  else if (tid < p.K)
    out(tid, sh.all[tid]);
}

// CTAs per row: enough to give every SM two, as long as each has a round.
static int ctas_per_row(int rows, int V, int size) {
  int q = 1;
  while (q < MAX_Q && static_cast<long long>(rows) * q < 2 * 148 &&
         static_cast<long long>(V) * size / (2 * q) >= NT * ELEMS * size / 2)
    q *= 2;
  return q;
}

static cudaError_t launch_rows(void (*kernel)(const Args), dim3 grid, dim3 block, const Args& a, cudaStream_t st) {
  if (a.Q > 8) {   // beyond the portable cluster size
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel_cluster(kernel, grid, block, 0, st, a.Q, a);
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
  a.Q = ctas_per_row(rows, a.V, z_bf16 ? 2 : 4);
  if (rows > 0x7fffffff / a.Q) return DFLASH_ERR_INVALID_ARG;
  const dim3 grid(static_cast<unsigned>(rows * a.Q)), block(NT);
  const cudaError_t e = z_bf16 ? launch_rows(logprobs_kernel<__nv_bfloat16>, grid, block, a, st)
                               : launch_rows(logprobs_kernel<float>, grid, block, a, st);
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
