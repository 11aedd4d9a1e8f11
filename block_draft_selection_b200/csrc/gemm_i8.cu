// Matrix product in 8-bit integers with a scale per token and per channel:
//   C[m,n] = float(sum_k A[m,k] B[n,k]) * sa[m] * sb[n]
//
// A persistent, warp-specialised tcgen05 kernel (kind::i8: int8 x int8 into
// int32 accumulators in TMEM, exact):
//   warp 0      TMA producer: 128-byte-swizzled K-major tiles of B and A into
//               a ring of shared-memory stages of 128 bytes of K
//   warp 1      MMA issuer into a double-buffered TMEM accumulator; owns the
//               TMEM allocation
//   warps 2..9  epilogue: TMEM -> registers -> C
// The channels (rows of B) are on the MMA's M side and the tokens (rows of A)
// on its N side.  A TMEM lane is then a channel and a register a token, so a
// warp's store of one register is 32 consecutive elements of a row of C: full
// 128-byte lines from any alignment of C, without a transpose.  And the tokens'
// side has steps of 16 (32 in a pair) instead of 128: 448 tokens are two tiles
// of 224.
//   STREAM (M <= 128, bound by the bytes of B): one token tile of M rounded
//          up to 16; each CTA owns one contiguous range of channels, balanced
//          at 16 rows, cut into tiles of nearly equal height <= 128, so that
//          no byte of B is read twice and all CTAs end together.
//   LARGE  (M > 128): tiles of 256 channels x up to 256 tokens on a cluster
//          of two CTAs that share one tcgen05.mma.cta_group::2 (each CTA
//          stages half of either operand and receives its 128 channels), dealt
//          out with the token tiles running fastest, so that the tiles in
//          flight share few rows of B through L2.  DFLASH_PAIR=0: single CTAs
//          with 128 channels.
// No load uses cluster multicast.  Every wait is bounded; a CTA that gives up
// drains its copies as the LM-head kernel does (in a pair the leader, on whose
// barriers both CTAs' copies complete, settles the stages that only one of
// them filled).
#include <cuda_bf16.h>

#include <atomic>

#include "common.cuh"
#include "host_util.cuh"

namespace dflash {
namespace gi8 {

constexpr int BK = 128;                 // bytes of K per stage: one swizzle row
constexpr int UMMA_K = 32;              // K per tcgen05.mma kind::i8
constexpr int CH = 128;                 // channels per CTA: the MMA's M side
constexpr int MAX_T = 256;              // tokens per tile: the MMA's N side
constexpr int EPI_WARPS = 8;
constexpr int EPI_THREADS = 32 * EPI_WARPS;
constexpr int NUM_THREADS = 64 + EPI_THREADS;
constexpr int SMEM_BUDGET = 226 * 1024;
constexpr int MAX_STAGES = 12;
constexpr int MAX_K = 131071;           // 128 * 128 * K stays below 2^31
constexpr int MAX_ROWS = 0x7fffff00;    // tile arithmetic stays in int

struct Params {
  int M, N;
  int num_kc;         // K stages per tile
  int stages;
  int tt;             // tokens per tile (MMA N)
  int t_rows;         // token rows this CTA loads (half of tt in a pair)
  int t_stage_bytes;  // stage bytes of the tokens
  int tmem_cols;      // two accumulators of half as many columns each
  int stream;
  int units;          // STREAM: 16-row units of channels
  int m_tiles;        // LARGE
  int tiles;
  int heights[4];     // STREAM: the tile heights, one tensor map each
  int w_prefetch;     // K stages of B prefetched into L2 before the dependency wait
  const float* sa;
  const float* sb;
  void* C;
  int* status;
  unsigned long long timeout_ns;
};

struct Tile {
  int c0;      // this CTA's first channel
  int c_rows;  // channels it loads (and the TMEM lanes that hold any)
  int m0;      // first token of the tile
};

// A CTA's range of n units is cut into this many tiles, the first n % tiles
// of them one unit higher than the rest.
__host__ __device__ inline int stream_tiles(int n) { return (n + CH / 16 - 1) / (CH / 16); }

template <bool PAIR>
__device__ __forceinline__ bool get_tile(const Params& p, int k, uint32_t rank, Tile& t) {
  if (!PAIR && p.stream) {
    const long long G = gridDim.x, c = blockIdx.x;
    const int u0 = static_cast<int>(c * p.units / G);
    const int n = static_cast<int>((c + 1) * p.units / G) - u0;
    const int kt = stream_tiles(n);
    if (k >= kt) return false;
    const int h = n / kt, r = n - h * kt;
    t.c0 = 16 * (u0 + k * h + min(k, r));
    t.c_rows = 16 * (h + (k < r ? 1 : 0));
    t.m0 = 0;
    return true;
  }
  const int unit = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
  const int count = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);
  const long long i = unit + static_cast<long long>(k) * count;
  if (i >= p.tiles) return false;
  const int ct = static_cast<int>(i) / p.m_tiles;
  t.m0 = (static_cast<int>(i) - ct * p.m_tiles) * p.tt;
  t.c0 = ct * (PAIR ? 2 * CH : CH) + static_cast<int>(rank) * CH;
  t.c_rows = CH;
  return true;
}

// Instruction descriptor of kind::i8: [4,6) D format (2 = s32); [7,10) and
// [10,13) A and B format (1 = signed 8-bit); K-major; [17,23) N >> 3;
// [24,29) M >> 4.
__device__ __forceinline__ uint32_t umma_idesc_s8(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

template <bool PAIR>
__device__ __forceinline__ void umma_s8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void put(float* c, float v) { *c = v; }
__device__ __forceinline__ void put(__nv_bfloat16* c, float v) { *c = __float2bfloat16_rn(v); }

template <bool PAIR, typename OUT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    gemm_i8_kernel(const __grid_constant__ CUtensorMap tm_t, const __grid_constant__ CUtensorMap tm_c0,
                   const __grid_constant__ CUtensorMap tm_c1, const __grid_constant__ CUtensorMap tm_c2,
                   const __grid_constant__ CUtensorMap tm_c3, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  constexpr int C_STAGE = CH * BK;
  const uint32_t s_c = smem_addr(smem);                                   // channels' stages
  const uint32_t s_t = s_c + static_cast<uint32_t>(p.stages) * C_STAGE;   // tokens' stages
  uint8_t* tail = smem + static_cast<size_t>(p.stages) * (C_STAGE + p.t_stage_bytes);
  const uint32_t bar0 = smem_addr(tail);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (p.stages + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * p.stages + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * p.stages + 2 + b); };
  const uint32_t drain_bar = bar0 + 8u * (2 * p.stages + 4);
  const uint32_t handover_bar = bar0 + 8u * (2 * p.stages + 5);   // pair: the other CTA's count of loads
  uint8_t* misc = tail + 8 * (2 * p.stages + 6);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  volatile int* peer_issued = reinterpret_cast<volatile int*>(misc + 8);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const uint32_t peer_abort = PAIR ? mapa_shared(smem_addr(const_cast<int*>(abort_flag)), rank ^ 1u) : 0u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), PAIR ? 2 * EPI_THREADS : EPI_THREADS);
    }
    mbar_init(drain_bar, 1);
    mbar_init(handover_bar, 1);
    *abort_flag = 0;
    *peer_issued = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_t);
    prefetch_tmap(&tm_c0);
  }
  if (warp == 1) {
    if (PAIR)
      tmem_alloc_pair(smem_addr(tmem_slot), p.tmem_cols);
    else
      tmem_alloc(smem_addr(tmem_slot), p.tmem_cols);
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  if (PAIR) cluster_sync_all();   // both CTAs' barriers exist before any remote signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int tmem_stride = p.tmem_cols >> 1;
  auto channel_map = [&](int rows) {
    return rows == p.heights[1] ? &tm_c1 : rows == p.heights[2] ? &tm_c2 : rows == p.heights[3] ? &tm_c3 : &tm_c0;
  };
  if (warp == 0 && lane == 0) {
    // B is a weight: its first stages may come into L2 while the kernel before
    // this one ends (L2 is the point of coherence, so nothing stale is seen
    // should that kernel write it after all)
    Tile t;
    if (get_tile<PAIR>(p, 0, rank, t)) {
      const CUtensorMap* mc = channel_map(t.c_rows);
      for (int kc = 0; kc < p.w_prefetch && kc < p.num_kc; ++kc) tma_prefetch_l2_2d(mc, kc * BK, t.c0);
    }
  }
  pdl_wait();
  const uint64_t deadline = globaltimer_ns() + p.timeout_ns;

  int issued = 0;   // producer: stage loads issued, in ring order
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol_c = p.stream ? l2_policy_evict_first() : l2_policy_evict_normal();
      const uint64_t pol_t = l2_policy_evict_last();
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      auto load = [&](uint32_t dst, const CUtensorMap* m, uint32_t fb, int x, int y, uint64_t pol) {
        if (PAIR)
          tma_load_2d_pair(dst, m, mapa_shared(fb, 0), x, y, pol);
        else
          tma_load_2d_hint(dst, m, fb, x, y, pol);
      };
      Tile t;
      for (int k = 0; ok && get_tile<PAIR>(p, k, rank, t); ++k) {
        const CUtensorMap* mc = channel_map(t.c_rows);
        const int t0 = t.m0 + static_cast<int>(rank) * p.t_rows;
        const uint32_t tx = static_cast<uint32_t>((PAIR ? 2 : 1) * (t.c_rows + p.t_rows) * BK);
        for (int kc = 0; kc < p.num_kc; ++kc) {
          if (!mbar_wait(empty_bar(s), ph ^ 1u, deadline, abort_flag, p.status, peer_abort)) {
            ok = false;
            break;
          }
          const uint32_t fb = full_bar(s);
          if (leader) mbar_arrive_expect_tx(fb, tx);
          load(s_c + s * C_STAGE, mc, fb, kc * BK, t.c0, pol_c);
          load(s_t + s * p.t_stage_bytes, &tm_t, fb, kc * BK, t0, pol_t);
          ++issued;
          if (++s == p.stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (PAIR && !leader) {
        st_shared_cluster_u32(mapa_shared(smem_addr(const_cast<int*>(peer_issued)), 0), static_cast<uint32_t>(issued));
        mbar_arrive_cluster(mapa_shared(handover_bar, 0));   // release: the count is visible first
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      const uint32_t idesc = umma_idesc_s8(PAIR ? 2 * CH : CH, p.tt);
      int s = 0, tb = 0;
      uint32_t ph = 0, tph = 0;
      bool ok = true;
      auto commit = [&](uint32_t bar) {
        if (PAIR)
          umma_commit_pair_multicast(bar, 0x3);
        else
          umma_commit(bar);
      };
      Tile t;
      for (int k = 0; ok && get_tile<PAIR>(p, k, rank, t); ++k) {
        if (!mbar_wait(tempty_bar(tb), tph ^ 1u, deadline, abort_flag, p.status, peer_abort)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(tb * tmem_stride);
        for (int kc = 0; kc < p.num_kc; ++kc) {
          if (!mbar_wait(full_bar(s), ph, deadline, abort_flag, p.status, peer_abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t cdesc = umma_desc_sw128(s_c + s * C_STAGE);
          const uint64_t tdesc = umma_desc_sw128(s_t + s * p.t_stage_bytes);
#pragma unroll
          for (int kk = 0; kk < BK / UMMA_K; ++kk)   // 32 bytes of K on: the address field counts 16
            umma_s8<PAIR>(d_tmem, cdesc + 2ull * kk, tdesc + 2ull * kk, idesc, (kc | kk) != 0 ? 1u : 0u);
          commit(empty_bar(s));
          if (++s == p.stages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        commit(tfull_bar(tb));
        if (++tb == 2) {
          tb = 0;
          tph ^= 1u;
        }
      }
      // every MMA issued has completed before TMEM is released
      if (PAIR)
        umma_commit_pair(drain_bar);
      else
        umma_commit(drain_bar);
      const uint64_t dl = globaltimer_ns() + 50000000ull;
      while (!mbar_try_wait(drain_bar, 0) && globaltimer_ns() < dl) {
      }
    }
  } else {
    const int quarter = warp & 3;             // the TMEM lanes this warp may access
    const int half = (warp - 2) >> 2;         // which half of the tile's tokens
    const int nch = p.tt / 16, split = (nch + 1) >> 1;
    int tb = 0;
    uint32_t tph = 0;
    Tile t;
    for (int k = 0; get_tile<PAIR>(p, k, rank, t); ++k) {
      int ok = 0;
      if (lane == 0) ok = mbar_wait(tfull_bar(tb), tph, deadline, abort_flag, p.status, peer_abort) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const int n = t.c0 + quarter * 32 + lane;
      const bool mine = quarter * 32 + lane < t.c_rows && n < p.N;
      const float sbn = mine ? __ldg(p.sb + n) : 0.f;
      const uint32_t taddr =
          tmem_base + static_cast<uint32_t>(tb * tmem_stride) + (static_cast<uint32_t>(quarter * 32) << 16);
      const int ch_end = __any_sync(0xffffffffu, mine) ? (half ? nch : split) : 0;
      for (int ch = half ? split : 0; ch < ch_end; ++ch) {
        const int m = t.m0 + ch * 16;
        if (m >= p.M) break;
        float x[16];
        tmem_ld16(taddr + ch * 16, x);
        tmem_ld_wait();
        OUT* c = static_cast<OUT*>(p.C) + static_cast<size_t>(m) * p.N + n;
        const int rows = min(16, p.M - m);
        if (mine) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (j < rows)
              put(c + static_cast<size_t>(j) * p.N, __int2float_rn(__float_as_int(x[j])) * __ldg(p.sa + m + j) * sbn);
        }
      }
      tc_fence_before();
      if (PAIR && !leader)
        mbar_arrive_cluster(mapa_shared(tempty_bar(tb), 0));
      else
        mbar_arrive(tempty_bar(tb));
      if (++tb == 2) {
        tb = 0;
        tph ^= 1u;
      }
    }
  }

  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  if (PAIR) cluster_sync_all();   // every role of both CTAs is done: abort flags and counts are final
  if (warp == 0 && lane == 0 && leader && *abort_flag != 0) {
    // Loads issued but never consumed must land before the CTA (and the other
    // CTA of a pair) may exit.  A stage load that only the leader issued has
    // the other CTA's bytes counted as arrived; one that only the other CTA
    // issued gets the leader's arrival with that CTA's bytes alone.
    const uint64_t dl = globaltimer_ns() + 50000000ull;
    int n_all = issued;
    if (PAIR && mbar_try_wait_acq_cluster(handover_bar, 0)) {
      const int n_peer = *peer_issued;
      const uint32_t peer_tx = static_cast<uint32_t>((CH + p.t_rows) * BK);
      for (int k = min(issued, n_peer); k < max(issued, n_peer); ++k) {
        if (issued > n_peer)
          mbar_complete_tx(full_bar(k % p.stages), peer_tx);
        else
          mbar_arrive_expect_tx(full_bar(k % p.stages), peer_tx);
      }
      n_all = max(issued, n_peer);
    }
    for (int q = 0; q < p.stages && q < n_all; ++q) {
      const int k_last = q + ((n_all - 1 - q) / p.stages) * p.stages;
      const uint32_t par = static_cast<uint32_t>(k_last / p.stages) & 1u;
      while (!mbar_try_wait(full_bar(q), par) && globaltimer_ns() < dl) {
      }
    }
  }
  if (PAIR) {
    __syncwarp();
    cluster_sync_all();   // the other CTA stays until the leader's drain is done
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem_base, p.tmem_cols);
    else
      tmem_dealloc(tmem_base, p.tmem_cols);
  }
}

// ------------------------------------------------------------ host side ----

// 2-D int8 tensor [rows, cols] row-major, box [box_rows, 128], 128-byte swizzle.
static bool make_map(CUtensorMap* m, const void* base, int rows, int cols, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(BK), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static size_t smem_bytes(const Params& p) {
  return 1024 + static_cast<size_t>(p.stages) * (CH * BK + p.t_stage_bytes) + 8 * (2 * p.stages + 6) + 16;
}

// At every launch: the attribute belongs to the current device and context.
template <bool PAIR, typename OUT>
static cudaError_t allow_smem() {
  return cudaFuncSetAttribute(gemm_i8_kernel<PAIR, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BUDGET);
}

// Clusters of two that can be resident at once on the current device (0:
// pairs cannot run), asked once per device.
static int max_pairs() {
  constexpr int MAX_DEVICES = 64;
  static std::atomic<int> known[MAX_DEVICES];   // the count plus one; 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < MAX_DEVICES) {
    const int k = known[dev].load(std::memory_order_relaxed);
    if (k > 0) return k - 1;
  }
  if (allow_smem<true, float>() != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = SMEM_BUDGET;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int c = 0;
  if (cudaOccupancyMaxActiveClusters(&c, gemm_i8_kernel<true, float>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev < MAX_DEVICES) known[dev].store(c + 1, std::memory_order_relaxed);
  return c;
}

struct Plan {
  Params p;
  bool pair;
  int grid;
};

static bool make_plan(int M, int N, int K, int sms, Plan& pl) {
  Params& p = pl.p;
  p = Params{};
  p.M = M;
  p.N = N;
  p.num_kc = (K + BK - 1) / BK;
  pl.pair = false;
  if (M <= CH) {
    p.stream = 1;
    p.tt = (M + 15) & ~15;
    p.t_rows = p.tt;
    p.units = (N + 15) / 16;
    pl.grid = p.units < sms ? p.units : sms;
    // a range has u or u + 1 units and tiles of two heights: at most four
    const int u = p.units / pl.grid;
    int k = 0;
    for (int n = u; n <= u + 1; ++n) {
      const int kt = stream_tiles(n);
      for (int h : {n / kt, n / kt + (n % kt ? 1 : 0)}) {
        bool have = false;
        for (int j = 0; j < k; ++j) have = have || p.heights[j] == 16 * h;
        if (!have) p.heights[k++] = 16 * h;
      }
    }
  } else {
    const int pairs = pair_allowed() ? max_pairs() : 0;
    pl.pair = pairs >= 1;
    const int units = pl.pair ? (pairs < sms / 2 ? pairs : sms / 2) : sms;
    const int ch = pl.pair ? 2 * CH : CH;
    const long long c_tiles = (static_cast<long long>(N) + ch - 1) / ch;
    // tokens per tile: the fewest rounds of tiles, a tile's time being that
    // of its operands' bytes (channels plus tokens)
    long long best = -1;
    for (int tt = MAX_T; tt >= 32; tt -= 32) {
      const long long tiles = c_tiles * ((M + tt - 1) / tt);
      const long long cost = (tiles + units - 1) / units * (ch + tt);
      if (best < 0 || cost < best) {
        best = cost;
        p.tt = tt;
      }
    }
    p.m_tiles = (M + p.tt - 1) / p.tt;
    const long long tiles = c_tiles * p.m_tiles;
    if (tiles > 0x7fffffffLL) return false;
    p.tiles = static_cast<int>(tiles);
    p.t_rows = pl.pair ? p.tt / 2 : p.tt;
    p.heights[0] = CH;
    const int used = tiles < units ? static_cast<int>(tiles) : units;
    pl.grid = pl.pair ? 2 * used : used;
  }
  p.t_stage_bytes = p.t_rows * BK;
  p.tmem_cols = 32;
  while (p.tmem_cols < 2 * p.tt) p.tmem_cols *= 2;
  for (p.stages = MAX_STAGES; p.stages > 2 && smem_bytes(p) > SMEM_BUDGET;) --p.stages;
  return smem_bytes(p) <= SMEM_BUDGET;
}

template <bool PAIR, typename OUT>
static cudaError_t launch_as(const Plan& pl, const CUtensorMap& tt, const CUtensorMap* tc, cudaStream_t st) {
  const cudaError_t e = allow_smem<PAIR, OUT>();
  if (e != cudaSuccess) return e;
  return launch_kernel_cluster(gemm_i8_kernel<PAIR, OUT>, dim3(pl.grid), dim3(NUM_THREADS), smem_bytes(pl.p), st,
                               PAIR ? 2 : 1, tt, tc[0], tc[1], tc[2], tc[3], pl.p);
}

}  // namespace gi8
}  // namespace dflash

extern "C" int dflash_gemm_i8(const int8_t* A, const float* sa, const int8_t* B, const float* sb, void* C, int c_bf16,
                              int M, int N, int K, int* dev_status, void* stream) {
  using namespace dflash;
  using namespace dflash::gi8;
  if (!A || !sa || !B || !sb || !C || M < 1 || N < 1 || M > MAX_ROWS || N > MAX_ROWS || K < 16 || K > MAX_K ||
      K % 16 != 0 || (c_bf16 & ~1))
    return DFLASH_ERR_INVALID_ARG;
  auto mis = [](const void* q, unsigned n) { return (reinterpret_cast<uintptr_t>(q) & (n - 1)) != 0; };
  if (mis(A, 16) || mis(B, 16) || mis(sa, 4) || mis(sb, 4) || mis(C, c_bf16 ? 2 : 4)) return DFLASH_ERR_INVALID_ARG;
  const int sms = num_sms_current();
  if (sms < 1) return DFLASH_ERR_CUDA;
  Plan pl;
  if (!make_plan(M, N, K, sms, pl)) return DFLASH_ERR_UNSUPPORTED;
  Params& p = pl.p;
  p.w_prefetch = p.stream ? 8 : 0;
  p.sa = sa;
  p.sb = sb;
  p.C = C;
  p.status = dev_status;
  p.timeout_ns = timeout_ns_from_env();
  CUtensorMap tt, tc[4];
  bool ok = gi8::make_map(&tt, A, M, K, p.t_rows);
  for (int j = 0; j < 4; ++j) {
    if (p.heights[j] > 0)
      ok = ok && gi8::make_map(&tc[j], B, N, K, p.heights[j]);
    else
      tc[j] = tc[0];
  }
  if (!ok) return DFLASH_ERR_CUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (pl.pair)
    e = c_bf16 ? launch_as<true, __nv_bfloat16>(pl, tt, tc, st) : launch_as<true, float>(pl, tt, tc, st);
  else
    e = c_bf16 ? launch_as<false, __nv_bfloat16>(pl, tt, tc, st) : launch_as<false, float>(pl, tt, tc, st);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
