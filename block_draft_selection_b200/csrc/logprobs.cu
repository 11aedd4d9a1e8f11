// Log-probabilities of given tokens, with entropy, rank and top alternatives.
//
//   lse = log sum exp(z/T),  logp = z_t/T - lse,  rank = 1 + #{z > z_t},
//   entropy = -sum p log p,  the K largest z (value desc, index asc)
//
// One pass over a row, which a cluster of Q CTAs shares (Q chosen so that few
// rows still fill the GPU).  Each warp keeps the largest z it has seen and a
// reference `base`, that z times c = log2(e) / T in fp32; each thread
// s = sum exp2(t) and w = sum t exp2(t) with t = z c - base, one fused
// multiply-add, and the count of values above z_t.  base moves with every
// record of the warp, so that no term is above 1 (a reference that lags d
// behind leaves errors of d 2^-24 in t and in w, which then cancel against
// log s: rows with one token far above the others had log-probabilities above
// 0 and entropies below it).  A warp's record is rarer than its threads', and
// the branch is the whole warp's, so this costs less than a lagging reference
// for each thread (513 rows of 151643 bf16 50.6 us, with it 51.9).
//
// The results are relative to base, so its rounding cancels; but the largest
// term is 2 to the power of what the rounding took away, up to half a unit of
// base's last place.  So |base| stops at FAR = 2^28, up to which that is 8.  Below
// -FAR a warp's terms are as good as none beside any row's that has a value
// above it (a finite mask), and a row that holds nothing within +-FAR (masked
// as a whole, or of a very low temperature, or with an infinity) has its sums
// taken again from differences z - max.  Values below -1e30 / c count as that
// value.
//
// c is rounded to fp32, i.e. the sums are those of a temperature off by a
// relative 2^-24; the log of the sum is corrected for that to first order with
// the mean of t, which the entropy needs anyway.
//
// The row streams through shared memory: each thread copies its own 16-byte
// vectors (cp.async) S - 1 rounds ahead and reads them back itself, so the
// loop has no barrier for its data, and the bytes in flight do not cost
// registers.  (Bulk copies of a warp's vectors as one chunk were measured instead: the
// longer way through the copy engine costs more than the load instructions
// saved, 31 against 19 us for 8 rows of 151936 on one CTA each.)
//
// Alternatives: K threads whose maxima are at least tau prove that the K-th
// largest value is at least tau.  The K-th largest of the warps' best thread
// maxima (32 of them) is such a tau; it is found after rounds 1, 4, 16, ... of
// the loop from the running maxima.  A thread whose round holds nothing of at
// least tau is done with one comparison; the others (20 to 60 of them between
// two bounds on unsorted rows for K = 16) note the round's maximum and its
// number.  At the end the rounds with a maximum above the last tau are read
// again and their values above it ranked by counting, first in each CTA, then
// in the cluster's first CTA, to which the others write theirs through
// distributed shared memory.  Rows that overflow these buffers (rising ones,
// or with many values equal to the K-th) are read once more against the last
// tau, into a list per warp that is sorted over its lanes.  Values of -inf are
// never listed; where fewer than K others exist, the first -inf fill up.
#include <cuda_bf16.h>

#include "common.cuh"
#include "host_util.cuh"
#include "pairs.cuh"

namespace dflash {
namespace lp {

constexpr unsigned FULL = 0xffffffffu;
constexpr int MAX_K = 32;
constexpr int MAX_V = 1 << 24;
constexpr int MAX_Q = 8;            // CTAs that share a row: a cluster
constexpr int LIST = 512;           // entries ranked at the end: as many as 16 warps' lists hold
constexpr float FAR = 268435456.f;  // 2^28: |base| stops here, the row is far
constexpr float LOW = -1e30f;       // terms below this z c are none
constexpr uint32_t LOWEST_KEY = 0x00800000u;   // of the lowest finite value
constexpr double LN2 = 0.69314718055994530942;

struct Args {
  const void* z;
  long long ld;
  int V;
  int K;
  float c;           // log2(e) / T in fp32
  float lo;          // LOW / c
  double inv_t;      // 1 / T
  double per_t;      // 1 / (T c): nats per unit of t, ln 2 but for c's rounding
  const int32_t* tokens;      // given tokens (or NULL)
  const int32_t* draft;       // emitted tokens: draft [B, L], accept_len, next_token [B]
  const int32_t* accept_len;
  const int32_t* next_token;
  int L;
  int Q;
  int eager;
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
  static __device__ __forceinline__ float value(float v) { return v; }
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
  static __device__ __forceinline__ float value(__nv_bfloat16 v) { return __bfloat162float(v); }
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

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t key_of(float z) { return static_cast<uint32_t>(entry_of(z, 0) >> 32); }

__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// What a thread does with its N words of a round (fp32: one logit each; bf16:
// two, for which maximum, minimum and count run packed).
template <typename Z, int N>
struct Round;

template <int N>
struct Round<float, N> {
  static constexpr int PAIRS = N / 2;
  float x[N];
  __device__ __forceinline__ void set(int i, uint32_t w) { x[i] = __uint_as_float(w); }
  __device__ __forceinline__ F2 pair(int i) const { return F2(x[2 * i], x[2 * i + 1]); }
  __device__ __forceinline__ float largest() const {   // NaN if there is one
    float m = x[0];
#pragma unroll
    for (int i = 1; i + 1 < N; i += 2) m = max_nan(m, max_nan(x[i], x[i + 1]));
    return max_nan(m, x[N - 1]);
  }
  __device__ __forceinline__ void raise(float lo) {   // NaN stays
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = max_nan(x[i], lo);
  }
  __device__ __forceinline__ int above(float zt) const {
    F2 n(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; i += 2) n = add2(n, F2(one_if_above(x[i], zt), one_if_above(x[i + 1], zt)));
    float a, b;
    n.get(a, b);
    return static_cast<int>(a + b);
  }
  static __device__ __forceinline__ float one_if_above(float a, float b) {
    float r;
    asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
  }
};

template <int N>
struct Round<__nv_bfloat16, N> {
  static constexpr int PAIRS = N;
  __nv_bfloat162 x[N];
  __device__ __forceinline__ void set(int i, uint32_t w) { x[i] = *reinterpret_cast<const __nv_bfloat162*>(&w); }
  __device__ __forceinline__ F2 pair(int i) const {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&x[i]);
    return widen2(w);
  }
  __device__ __forceinline__ float largest() const {
    __nv_bfloat162 m = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = __hmax2_nan(m, x[i]);
    return max_nan(__low2float(m), __high2float(m));
  }
  __device__ __forceinline__ void raise(float lo) {
    const __nv_bfloat162 l = __float2bfloat162_rn(lo);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __hmax2_nan(x[i], l);
  }
  __device__ __forceinline__ int above(float zt) const {   // counts up to N <= 256 are exact
    const __nv_bfloat162 t = __float2bfloat162_rn(zt);
    __nv_bfloat162 n = __hgt2(x[0], t);
#pragma unroll
    for (int i = 1; i < N; ++i) n = __hadd2(n, __hgt2(x[i], t));
    return static_cast<int>(__low2float(n) + __high2float(n));
  }
};

// The reference that goes with a largest value (one rounding, the same
// wherever it is taken).
__device__ __forceinline__ float base_of(float top, float c) { return fminf(fmaxf(__fmul_rn(top, c), -FAR), FAR); }

// Sums of values up to `top` (-inf: none): s = sum 2^t, w = sum t 2^t,
// t = z c - base_of(top, c).
struct Sums {
  float top;
  int cnt;
  double s, w;

  // Over groups of G lanes, relative to their largest value's base.
  template <int G>
  __device__ __forceinline__ void reduce(float c) {
    float big = top;
#pragma unroll
    for (int off = G / 2; off; off >>= 1) big = fmaxf(big, __shfl_xor_sync(FULL, big, off));
    if (top != -INFINITY && top != big) {
      const float d = base_of(top, c) - base_of(big, c);
      const double f = ex2(d);
      w = f > 0.0 ? f * (w + d * s) : s * 0.0;
      s *= f;
    }
    top = big;
#pragma unroll
    for (int off = G / 2; off; off >>= 1) {
      s += __shfl_xor_sync(FULL, s, off);
      w += __shfl_xor_sync(FULL, w, off);
      cnt += __shfl_xor_sync(FULL, cnt, off);
    }
  }
};

// 1 / x and log x of a positive finite fp64 sum, to about 1e-12 and 1e-7 of
// log x's mantissa part: fp32 functions (log1p of mantissa - 1 keeps the
// relative precision of sums just above 1), one Newton step for 1 / x.  A few
// fp64 operations instead of the library's hundreds on a row's critical path.
__device__ __forceinline__ double recip(double x) {
  const double r = 1.f / static_cast<float>(x);
  return r * (2.0 - x * r);
}

__device__ __forceinline__ double log_sum(double x) {
  const int hi = __double2hiint(x);
  int e = (hi >> 20) - 1023;
  double mant = __hiloint2double((hi & 0x000fffff) | 0x3ff00000, __double2loint(x));   // [1, 2)
  if (mant > 1.4142135) {
    mant *= 0.5;
    ++e;
  }
  return e * LN2 + static_cast<double>(log1pf(static_cast<float>(mant - 1.0)));
}

// A log-probability without the sign that rounding could give it; a NaN stays.
__device__ __forceinline__ float not_above_0(double x) { return x > 0.0 ? 0.f : static_cast<float>(x); }

// The token asked for in a row: what it is read from, then what it is and
// whether the row is asked for at all.
struct RowToken {
  int n = 0, next = -1, token = -1;

  __device__ __forceinline__ void load(const Args& p, int row) {
    if (p.accept_len != nullptr) {
      const int b = row / (p.L + 1), i = row - b * (p.L + 1);
      n = p.accept_len[b];
      next = p.next_token[b];
      if (i < p.L) token = p.draft[static_cast<size_t>(b) * p.L + i];
    } else if (p.tokens != nullptr) {
      token = p.tokens[row];
    }
  }
  __device__ __forceinline__ bool asked(const Args& p, int row) {
    if (p.accept_len != nullptr) {
      const int i = row % (p.L + 1);
      if (n < 1 || n > p.L + 1) {
        if (threadIdx.x == 0) set_status(p.status, DFLASH_ERR_BAD_INDEX);
        n = n < 1 ? 1 : p.L + 1;
      }
      if (i >= n) return false;
      if (i == n - 1) token = next;
      if (token < 0) token = 0x7fffffff;   // out of range, not padding
      return true;
    }
    return p.tokens == nullptr || token >= 0;
  }
};

// Shared memory of a CTA beside its ring; `all` and `sums` of the cluster's
// first CTA take every CTA's list and sums.
template <int NOTES>
struct Shared {
  uint64_t note[NOTES];             // (key of the round's maximum, round * 32 + lane), per warp
  uint64_t list[LIST];              // entries to be ranked
  uint64_t all[MAX_Q * MAX_K];      // [CTA][K], sorted downwards, 0 past the end
  Sums sums[MAX_Q];
  Sums part[16];
  alignas(16) uint32_t best[2][32]; // keys of thread maxima, 32 / warps of each warp
  int n_list, n_all;
  double origin, base, log_s;       // z's log-probability: ((z - origin) c - base) per_t - log_s
};

// Rank the n entries of `list` by counting, by all warps but the first, and
// hand each with its rank to put.
template <int NT, typename F>
__device__ __forceinline__ void rank_entries(const uint64_t* list, int n, int K, F put) {
  for (int i = static_cast<int>(threadIdx.x) - 32; i >= 0 && i < n; i += NT - 32) {
    const uint64_t mine = list[i];
    int rank = 0;
#pragma unroll 8
    for (int k = 0; k < n; ++k) rank += list[k] > mine ? 1 : 0;
    if (rank < K) put(rank, mine);
  }
}

// The sums of a row from differences to its maximum m, by one CTA: for rows
// where m c is beyond FAR.  s and w in every thread.
template <typename Z, int NT, typename SharedT>
__device__ __noinline__ void far_sums(const Z* z, int V, float c, float m, SharedT& sh, double& s, double& w) {
  constexpr int E = Vec<Z>::E;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  s = w = 0.0;
  auto add = [&](const uint4& u) {
    float y[E], se = 0.f, we = 0.f;
    Vec<Z>::unpack(u, y);
#pragma unroll
    for (int j = 0; j < E; ++j) {   // outside the row -inf: a term of 0
      const float t = max_nan((y[j] - m) * c, -200.f);
      const float e = ex2(t);
      se += e;
      we = fmaf(e, t, we);
    }
    s += se;   // a vector's terms in fp32, vectors in fp64
    w += we;
  };
  const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(Z));
  const int begin = lead > 0 ? 1 : 0, end = (V + lead) / E;   // vectors inside the row whole
  const uint4* zv = reinterpret_cast<const uint4*>(z - lead);
#pragma unroll 4
  for (int v = begin + static_cast<int>(threadIdx.x); v < end; v += NT) add(__ldg(zv + v));
  if (threadIdx.x == 0 && lead > 0) add(load_vec(z, -lead, V));
  if (threadIdx.x == 0 && end >= begin && end * E - lead < V) add(load_vec(z, end * E - lead, V));
  for (int off = 16; off; off >>= 1) {
    s += __shfl_xor_sync(FULL, s, off);
    w += __shfl_xor_sync(FULL, w, off);
  }
  if (lane == 0) {
    sh.part[warp].s = s;
    sh.part[warp].w = w;
  }
  __syncthreads();
  s = w = 0.0;
  for (int k = 0; k < NT / 32; ++k) {
    s += sh.part[k].s;
    w += sh.part[k].w;
  }
}

// NT threads with U vectors each a round, S rounds in the ring.
template <typename Z, int NT, int U, int S, int CTAS>
__global__ void __launch_bounds__(NT, CTAS) logprobs_kernel(const Args p) {
  constexpr int E = Vec<Z>::E;
  constexpr int NW = NT / 32;
  constexpr int NOTES = NT < 256 ? 4 * NT : 1024;   // rounds a CTA can note
  constexpr int CAP = NOTES / NW;     // a warp's notes
  constexpr int STAGE = U * NT;       // vectors per round
  static_assert(NW * 32 <= LIST && NW > 1 && NW <= 16 && MAX_Q * MAX_K <= LIST, "lists fit");
  constexpr int CHUNK = U * 32;       // vectors per warp and round: U times 32, NT apart
  constexpr int SPAN = STAGE - NT + 32;   // from their first to past their last
  extern __shared__ uint4 ring_all[];   // [NW][S][CHUNK]
  __shared__ Shared<NOTES> sh;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint4* ring = ring_all + warp * S * CHUNK;
  const uint32_t ring_addr = smem_addr(ring + lane);
  const int Q = p.Q, row = blockIdx.x / Q, q = blockIdx.x - row * Q;
  RowToken rt;
  rt.load(p, row);
  if (tid == 0) sh.n_list = sh.n_all = 0;
  const Z* z = static_cast<const Z*>(p.z) + static_cast<size_t>(row) * p.ld;

  // the row as 16-byte vectors from the boundary at or before its start
  const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(Z));
  const int n_vec = (p.V + lead + E - 1) / E;
  const int v_begin = static_cast<int>(static_cast<long long>(q) * n_vec / Q);
  const int v_end = static_cast<int>(static_cast<long long>(q + 1) * n_vec / Q);
  const int rounds = (v_end - v_begin + STAGE - 1) / STAGE;
  const uint32_t fill = E == 4 ? 0xff800000u : 0xff80ff80u;
  // vectors [in_begin, in_end) lie inside the row whole
  const int in_begin = lead > 0 ? 1 : 0, in_end = min(v_end, (p.V + lead) / E);
  const uint4* zv = reinterpret_cast<const uint4*>(z - lead);
  const int w_begin = v_begin + warp * 32;   // this warp's first vector of round 0
  // This lane's copies of round r: its vectors that lie inside the row whole.
  auto fetch = [&](int r) {
    const int v0 = w_begin + r * STAGE;
    const uint32_t to = ring_addr + 16 * ((r % S) * CHUNK);
    if (v0 >= in_begin && v0 + SPAN <= in_end) {
#pragma unroll
      for (int u = 0; u < U; ++u) copy16(to + 16 * u * 32, zv + v0 + u * NT + lane);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * NT + lane;
        if (v >= in_begin && v < in_end) copy16(to + 16 * u * 32, zv + v);
      }
    }
    copies_commit();
  };
  // this lane's vectors of round r
  Round<Z, 4 * U> x;
  auto take = [&](int r) {
    const int v0 = w_begin + r * STAGE;
    const uint4* at = ring + (r % S) * CHUNK + lane;
    const bool whole = v0 >= in_begin && v0 + SPAN <= in_end;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = v0 + u * NT + lane;
      uint4 vec;
      if (whole || (v >= in_begin && v < in_end))
        vec = at[u * 32];
      else
        vec = v < v_end ? load_vec(z, v * E - lead, p.V) : make_uint4(fill, fill, fill, fill);
      x.set(4 * u, vec.x);
      x.set(4 * u + 1, vec.y);
      x.set(4 * u + 2, vec.z);
      x.set(4 * u + 3, vec.w);
    }
  };
  // where every row's CTAs run at once, the first loads do not wait for the
  // row's token (a row that is not asked for costs them in vain then)
  if (p.eager) {
#pragma unroll
    for (int r = 0; r < S - 1; ++r) fetch(r);
  }
  // remote stores wait until every CTA of the cluster has started
  if (Q > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (!rt.asked(p, row)) {
    copies_wait<0>();
    // every CTA of the cluster comes to the same answer, unless the tokens
    // change meanwhile; the barriers are met in that case too
    if (Q > 1) {
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      cluster_sync_all();
    }
    return;
  }
  if (!p.eager) {
#pragma unroll
    for (int r = 0; r < S - 1; ++r) fetch(r);
  }
  const bool bad_token = rt.token >= p.V;
  if (bad_token && tid == 0 && q == 0) set_status(p.status, DFLASH_ERR_BAD_INDEX);
  const float zt = rt.token >= 0 && !bad_token ? Vec<Z>::load(z + rt.token) : INFINITY;

  const F2 c2(p.c, p.c);
  F2 s2[2] = {F2(0.f, 0.f), F2(0.f, 0.f)}, w2[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
  float base = 0.f, top = -INFINITY;   // the warp's
  float seen = -INFINITY, tau = -INFINITY;
  uint32_t tau_key = 0;
  int cnt = 0, bounds = 0, notes = 0, next_bound = 0;
  // s and w relative to another base, d below
  auto rescale = [](float d, float& s, float& w) {
    const float f = ex2(d);
    w = f > 0.f ? f * (w + d * s) : s * 0.f;
    s *= f;
  };
  // Called by all threads: publish this warp's best maxima; after a barrier,
  // the K-th largest of all.
  auto publish = [&]() {
    uint32_t left = key_of(seen);
#pragma unroll
    for (int i = 0; i < 32 / NW; ++i) {
      const uint32_t k = __reduce_max_sync(FULL, left);
      const int at = warp * (32 / NW) + i;
      if (lane == 0) sh.best[bounds & 1][at] = (k & ~31u) | at;
      if (lane == __ffs(__ballot_sync(FULL, left == k)) - 1) left = 0;
    }
  };
  auto bound = [&]() {   // two buffers: a warp is at most one bound ahead of another
    const uint4* best = reinterpret_cast<const uint4*>(sh.best[bounds & 1]);
    const uint32_t mine = sh.best[bounds & 1][lane];
    ++bounds;
    int above = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint4 b = best[k];
      above += (b.x > mine) + (b.y > mine) + (b.z > mine) + (b.w > mine);
    }
    // the low bits, which made the keys distinct, off: a little lower still bounds
    tau_key = __shfl_sync(FULL, mine, __ffs(__ballot_sync(FULL, above == p.K - 1)) - 1) & ~31u;
    tau = tau_key < LOWEST_KEY ? -INFINITY : value_of(static_cast<uint64_t>(tau_key) << 32);
  };

  for (int r = 0; r < rounds; ++r) {
    copies_wait<S - 2>();
    take(r);
    fetch(r + S - 1);
    const float m = x.largest();
    seen = fmaxf(seen, m);   // a NaN is not seen
    if (__any_sync(FULL, m > top)) {
      const float now = warp_max(seen), to = base_of(now, p.c);
      if (top != -INFINITY) {   // else all sums are 0
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float s0, s1, w0, w1;
          s2[k].get(s0, s1);
          w2[k].get(w0, w1);
          rescale(base - to, s0, w0);
          rescale(base - to, s1, w1);
          s2[k] = F2(s0, s1);
          w2[k] = F2(w0, w1);
        }
      }
      base = to;
      top = now;
    }
    const bool bounding = p.K > 0 && r == next_bound;
    if (bounding) publish();
    if (m > zt || m != m) cnt += x.above(zt);
    x.raise(p.lo);   // a masked value's t = -inf would make 0 * t a NaN
    const F2 nb(-base, -base);
#pragma unroll
    for (int i = 0; i < x.PAIRS; ++i) {
      const F2 t2 = fma2(x.pair(i), c2, nb);
      float t0, t1;
      t2.get(t0, t1);
      const F2 e(ex2(t0), ex2(t1));
      s2[i & 1] = add2(s2[i & 1], e);
      w2[i & 1] = fma2(e, t2, w2[i & 1]);
    }
    if (bounding) {
      next_bound = 4 * r + 3;   // after 1, 4, 16, ... rounds
      __syncthreads();
      bound();
    }
    if (p.K > 0) {
      const bool note = !(m < tau) && !(m == -INFINITY);
      const unsigned who = __ballot_sync(FULL, note);
      if (who) {
        const int at = notes + __popc(who & ((1u << lane) - 1));
        if (note && at < CAP)
          sh.note[warp * CAP + at] = (static_cast<uint64_t>(key_of(m)) << 32) | static_cast<uint32_t>(r * 32 + lane);
        notes += __popc(who);
      }
    }
  }

  // Noted rounds that still count have their values listed; the round's
  // vectors are read again (from the ring where the whole part is still in it).
  // Each lane's first one is on its way before the sums and the last bound.
  uint4 again[U];
  auto read_again = [&](uint64_t note) {
    const int r = static_cast<int>(static_cast<uint32_t>(note) / 32), ln = static_cast<int>(note % 32);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = u * 32 + ln, v = w_begin + r * STAGE + u * NT + ln;
      again[u] = make_uint4(fill, fill, fill, fill);
      if (rounds <= S && v >= in_begin && v < in_end)
        again[u] = ring[r * CHUNK + at];
      else if (v < v_end)
        again[u] = load_vec(z, v * E - lead, p.V);
    }
  };
  auto list_values = [&](uint64_t note) {
    const int first = (w_begin + static_cast<int>(static_cast<uint32_t>(note) / 32) * STAGE + static_cast<int>(note % 32)) * E - lead;
    uint64_t bits = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float y[E];
      Vec<Z>::unpack(again[u], y);
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (!(y[j] < tau) && !(y[j] == -INFINITY)) bits |= 1ull << (u * E + j);
    }
    int to = atomicAdd(&sh.n_list, __popcll(bits));
    for (; bits != 0; bits &= bits - 1, ++to) {   // one or two
      const int el = __ffsll(static_cast<long long>(bits)) - 1;
      float v = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float y[E];
        Vec<Z>::unpack(again[u], y);
#pragma unroll
        for (int j = 0; j < E; ++j) v = el == u * E + j ? y[j] : v;
      }
      if (to < LIST) sh.list[to] = entry_of(v, first + el / E * (NT * E) + el % E);
    }
  };
  auto note_at = [&](int i) -> uint64_t {   // 0 if it does not count any more
    const uint64_t e = i < min(notes, CAP) ? sh.note[warp * CAP + i] : 0;
    return static_cast<uint32_t>(e >> 32) >= tau_key ? e : 0;
  };
  uint64_t note = 0;
  const bool fresh = next_bound == 4 * rounds - 1;   // the last round ended with a bound
  if (p.K > 0) {
    __syncwarp();   // the warp's notes are its lanes'
    note = note_at(lane);
    if (note != 0) read_again(note);
    if (!fresh) publish();
  }
  // the warp's sums
  {
    float s, w, s1, w1;
    add2(s2[0], s2[1]).get(s, s1);
    add2(w2[0], w2[1]).get(w, w1);
    s += s1;
    w += w1;
    // five levels in fp32, 2^-24 each; across warps and CTAs fp64
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      s += __shfl_xor_sync(FULL, s, off);
      w += __shfl_xor_sync(FULL, w, off);
    }
    cnt = __reduce_add_sync(FULL, cnt);
    if (lane == 0) sh.part[warp] = Sums{top, cnt, s, w};
  }
  __syncthreads();
  if (p.K > 0) {
    if (!fresh) bound();
    if (note != 0 && static_cast<uint32_t>(note >> 32) >= tau_key) list_values(note);
    for (int i = lane + 32; i < min(notes, CAP); i += 32) {
      note = note_at(i);
      if (note != 0) {
        read_again(note);
        list_values(note);
      }
    }
    if (__syncthreads_or(notes > CAP) || sh.n_list > LIST) {   // the same for all threads
      __syncthreads();
      if (tid == 0) sh.n_list = 0;
      WarpTop top{0, 0};
      for (int v0 = w_begin; v0 < v_begin + rounds * STAGE; v0 += STAGE) {
        for (int u = 0; u < U; ++u) {
          const int v = v0 + u * NT + lane;
          float y[E];
          Vec<Z>::unpack(v < v_end ? load_vec(z, v * E - lead, p.V) : make_uint4(fill, fill, fill, fill), y);
#pragma unroll
          for (int j = 0; j < E; ++j)
            top.offer(!(y[j] < tau) && !(y[j] == -INFINITY) ? entry_of(y[j], v * E - lead + j) : 0, p.K, lane);
        }
      }
      __syncthreads();
      if (top.ent != 0) sh.list[atomicAdd(&sh.n_list, 1)] = top.ent;
      __syncthreads();
    }
  }

  // From here the first warp has the sums, the others rank the alternatives.
  int n = p.K > 0 ? sh.n_list : 0;
  Sums sum;
  if (warp == 0) {
    sum = sh.part[lane & (NW - 1)];
    sum.template reduce<NW>(p.c);
  }
  if (Q > 1) {
    // hand list and sums to the cluster's first CTA
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (tid == 0) {
      const uint32_t to = mapa_shared(smem_addr(sh.sums + q), 0);
      const uint64_t* from = reinterpret_cast<const uint64_t*>(&sum);
#pragma unroll
      for (int k = 0; k < static_cast<int>(sizeof(Sums) / 8); ++k) st_cluster_u64(to + 8 * k, from[k]);
    }
    if (p.K > 0) {
      const uint32_t to = mapa_shared(smem_addr(sh.all + q * MAX_K), 0);
      rank_entries<NT>(sh.list, n, p.K, [&](int rank, uint64_t e) { st_cluster_u64(to + 8 * rank, e); });
      if (tid >= n && tid < p.K) st_cluster_u64(to + 8 * tid, 0);
    }
    cluster_sync_all();
    if (q != 0) return;
    if (warp == 0) {
      const int i = lane & (MAX_Q - 1);
      sum = i < Q ? sh.sums[i] : Sums{-INFINITY, 0, 0.0, 0.0};
      sum.template reduce<MAX_Q>(p.c);
    } else if (p.K > 0) {
      // the largest of the CTAs' K-th entries bounds the row's K-th from below
      uint64_t least = lane < Q ? sh.all[lane * MAX_K + p.K - 1] : 0;
#pragma unroll
      for (int off = MAX_Q / 2; off; off >>= 1) {
        const uint64_t o = __shfl_xor_sync(FULL, least, off);
        least = o > least ? o : least;
      }
      least = __shfl_sync(FULL, least, 0);
      for (int i = tid - 32; i < Q * MAX_K; i += NT - 32) {
        const uint64_t e = (i & (MAX_K - 1)) < p.K ? sh.all[i] : 0;
        if (e != 0 && e >= least) sh.list[atomicAdd(&sh.n_all, 1)] = e;
      }
      named_barrier_sync(1, NT - 32);
      n = sh.n_all;
    }
  }
  if (warp != 0 && p.K > 0)
    rank_entries<NT>(sh.list, n, p.K, [&](int rank, uint64_t e) { sh.all[rank] = e; });

  // the row's results but for the alternatives, by one lane
  auto finish = [&](double origin, float base_all) {
    const bool dead = sum.top == -INFINITY && sum.s == 0.0;
    const double from = dead ? 0.0 : base_all;
    const double mean_t = sum.w * recip(sum.s);
    const double log_s0 = log_sum(sum.s);
    const double log_s = dead ? 0.0 : log_s0 + (p.per_t - LN2) * mean_t;
    sh.origin = origin;
    sh.base = from;
    sh.log_s = log_s;
    if (p.lse != nullptr) p.lse[row] = static_cast<float>(dead ? -INFINITY : origin * p.inv_t + from * p.per_t + log_s);
    if (p.entropy != nullptr) p.entropy[row] = dead ? 0.f : 0.f - not_above_0(mean_t * LN2 - log_s0);
    if (p.logp != nullptr) {
      const double v = ((zt - origin) * p.c - from) * p.per_t - log_s;
      p.logp[row] = bad_token ? __int_as_float(0x7fc00000) : not_above_0(v);
    }
    if (p.rank != nullptr) p.rank[row] = bad_token ? 0 : sum.cnt + 1;
  };
  const float base_all = sum.top == -INFINITY ? -INFINITY : base_of(sum.top, p.c);
  const bool far = tid == 0 && !(fabsf(base_all) < FAR) && sum.top != -INFINITY;
  if (tid == 0) {
    if (far)
      sh.origin = sum.top;
    else
      finish(0.0, base_all);
  }
  if (__syncthreads_or(far)) {
    const double origin = sh.origin;
    double s, w;
    far_sums<Z, NT>(z, p.V, p.c, static_cast<float>(origin), sh, s, w);
    sum.s = s;
    sum.w = w;
    if (tid == 0) finish(origin, 0.f);
    __syncthreads();
  }
  if (p.K == 0) return;
  if (Q > 1) n = sh.n_all;   // the first warp's too
  auto out = [&](int rank, uint64_t e) {
    const size_t o = static_cast<size_t>(row) * p.K + rank;
    p.top_logp[o] = not_above_0(((value_of(e) - sh.origin) * p.c - sh.base) * p.per_t - sh.log_s);
    p.top_idx[o] = index_of(e);
  };
  if (tid < min(n, p.K)) out(tid, sh.all[tid]);
  // fewer than K values that are not -inf: the first of -inf, by one warp
  if (n < p.K && warp == NW - 1) {
    int have = n;
    for (int v0 = 0; have < p.K && v0 < p.V; v0 += 32) {
      const int v = v0 + lane;
      const bool none = v < p.V && Vec<Z>::load(z + v) == -INFINITY;
      const unsigned which = __ballot_sync(FULL, none);
      const int rank = have + __popc(which & ((1u << lane) - 1));
      if (none && rank < p.K) out(rank, entry_of(-INFINITY, v));
      have += __popc(which);
    }
  }
}

template <typename Z, int NT, int U, int S, int CTAS>
static cudaError_t launch_rows(int rows, const Args& a, cudaStream_t st) {
  constexpr size_t bytes = sizeof(uint4) * S * U * NT;
  auto* kernel = logprobs_kernel<Z, NT, U, S, CTAS>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e != cudaSuccess) return e;
  return launch_kernel_cluster(kernel, dim3(static_cast<unsigned>(rows * a.Q)), dim3(NT), bytes, st, a.Q, a);
}

// Up to one row per SM: CTAs of 512 threads, one on an SM and all at once, with
// as many of them to a row as fit (each with 4096 logits at least), and loads
// that do not wait for the tokens.  More rows: three CTAs of 256 threads on an
// SM, two to a row while all of them are resident together.  Rows of 151936
// fp32, us, this rule's choice against the other form's best: 8 rows 9.9 / 11.1,
// 32 rows 12.7 / 14.6, 64 rows 17.0 / 18.6, 148 rows 24.3 / 29.4; 200 rows 32.5
// with two CTAs, 37.6 with one, 43.5 in the first form; 300 rows 47.8 with one,
// 51.4 with two.  Clusters of 16 measured 16 us for 8 rows.
//
// What a row costs beside its values (barriers, bound, ranking) falls with the
// CTA's size, so short rows and many rows go to smaller CTAs, more of them on an
// SM.  us, against the forms above, fp32 with K = 16 (bf16 with K = 20 where it
// says so): 128 threads, 100 rows of 2000 4.8 / 5.7 and of 4000 5.8 / 5.7; 200
// of 8000 7.5 / 7.0; 600 of 8000 11.6 / 13.5 and of 16000 17.5 / 18.7, 500 of
// 64000 bf16 33.2 / 29.2; 1700 of 129280 169 / 173, 4352 of 64000 bf16 152 / 174,
// 4352 of 8000 52 / 73.  64 threads: 4352 of 1000 18.5 / 54.5 (128: 29.4), of
// 4000 34.4 / 56.9 (40.1), of 8000 52.3 / 73.2 (51.0); 600 of 1000 5.8 / 10.6
// (7.1), of 4000 9.3 / 10.5 (9.0); 100 of 1000 5.2 / 5.6 (4.7).
template <typename Z>
static cudaError_t launch_rows(int rows, Args& a, cudaStream_t st) {
  const int sms = num_sms_current();
  const long long n_vec = (static_cast<long long>(a.V) * sizeof(Z) + 15) / 16;
  a.Q = 1;
  if (n_vec <= (rows > 8 * sms ? 1024 : 256) && rows > 2 * sms) {
    a.eager = rows <= 12 * sms;
    return launch_rows<Z, 64, 4, 2, 12>(rows, a, st);
  }
  if (n_vec <= 512 || (n_vec <= 4096 && rows > 2 * sms) || rows > 6 * sms) {
    a.eager = rows <= 6 * sms;
    return launch_rows<Z, 128, 4, 3, 6>(rows, a, st);
  }
  a.eager = rows <= sms;
  if (a.eager) {
    while (a.Q < MAX_Q && 2 * a.Q * rows <= sms && a.V / (2 * a.Q) >= 4096) a.Q *= 2;
    return launch_rows<Z, 512, 4, 3, 1>(rows, a, st);
  }
  if (2 * rows <= 3 * sms && a.V >= 2 * 4096) a.Q = 2;
  a.eager = a.Q * rows <= 3 * sms;
  return launch_rows<Z, 256, 4, 3, 3>(rows, a, st);
}

static int launch(Args& a, int z_bf16, int rows, float temperature, cudaStream_t st) {
  if (!a.z || (z_bf16 & ~1) || a.V < 1 || a.V > MAX_V || a.ld < a.V || a.K < 0 || a.K > MAX_K || a.K > a.V)
    return DFLASH_ERR_INVALID_ARG;
  if (!(temperature >= 1e-6f) || !(temperature <= 1e6f)) return DFLASH_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(a.z) & (z_bf16 ? 1 : 3)) return DFLASH_ERR_INVALID_ARG;
  if ((a.top_logp == nullptr) != (a.top_idx == nullptr) || (a.top_logp != nullptr && a.K == 0))
    return DFLASH_ERR_INVALID_ARG;
  if (a.top_logp == nullptr) a.K = 0;
  a.inv_t = 1.0 / static_cast<double>(temperature);
  a.c = static_cast<float>(1.4426950408889634 / static_cast<double>(temperature));
  a.lo = LOW / a.c;
  a.per_t = a.inv_t / a.c;
  if (rows > 0x7fffffff / 2) return DFLASH_ERR_INVALID_ARG;
  const cudaError_t e = z_bf16 ? launch_rows<__nv_bfloat16>(rows, a, st) : launch_rows<float>(rows, a, st);
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
