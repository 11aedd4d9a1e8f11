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
// A stage costs the lanes that issue for it 350 to 450 clocks whatever it
// holds, and an SM's share of the memory bandwidth is about 23 bytes a clock, so
// stages are kept full, with the operand whose bytes bound the call on the side
// of the MMA that takes more of it:
//   STREAM (M <= 128, bound by the bytes of B): channels (rows of B) on the N
//          side, up to 256 a tile, the tokens (rows of A), rounded up to 16, on
//          the M side: a stage holds up to 32 KB of B (with the channels on the
//          M side 16 KB; [96 x 151936 x 5120] took 159 us, so it took 147).  The
//          tiles are dealt out as CTAs come to need them, since SMs do not get
//          equal shares of the bandwidth: the grid has a CTA per tile, the
//          first ones run, and each asks the hardware to cancel a CTA that has
//          not started yet and takes its tile (cluster launch control).
//          The accumulator's rows are tokens; the epilogue turns blocks of
//          32 x 32 through shared memory and stores whole rows of them, from
//          any alignment of C.  With N <= 128 < M the operands change places:
//          few channels on the M side, the tokens as the long operand
//          ([4352 x 5 x 5120] took 70 us on LARGE's tiles, mostly empty).
//   SPLIT  the same with few tiles: a cluster of up to 8 CTAs to a tile, each
//          with a part of K.  Each leaves its int32 sums in its shared memory
//          and adds up its share of the tile over the cluster's: integers, so
//          the result is the same.  No more clusters than run at once.
//          Both also take a few hundred tokens in tiles of up to 128 where
//          there would be few tiles of pairs with a long K (plan_few).
//   LARGE  (else): channels on the M side, tokens on the N side, in steps of
//          32 instead of 128 (448 tokens are two tiles of 224).  Tiles of 256
//          channels x up to 256 tokens on a cluster of two CTAs that share one
//          tcgen05.mma.cta_group::2 (each CTA stages half of either operand and
//          receives its 128 channels), dealt out with the token tiles running
//          fastest, so that the tiles in flight share few rows of B through
//          L2.  A TMEM lane is a channel and a register a token, so a warp's
//          store of one register is 32 consecutive elements of a row of C
//          without a transpose.  DFLASH_PAIR=0: single CTAs with 128 channels.
// No load uses cluster multicast.  Every wait is bounded; a CTA that gives up
// drains its copies as the LM-head kernel does (in a pair the leader, on whose
// barriers both CTAs' copies complete, settles the stages that only one of
// them filled).
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "host_util.cuh"

namespace dflash {
namespace gi8 {

constexpr int BK = 128;                 // bytes of K per stage: one swizzle row
constexpr int UMMA_K = 32;              // K per tcgen05.mma kind::i8
constexpr int CH = 128;                 // the MMA's M side in one CTA: channels (LARGE), tokens (STREAM)
constexpr int MAX_N = 256;              // its N side: tokens (LARGE), channels (STREAM)
constexpr int BLOCK = 32 * 33;          // STREAM: a 32 x 32 block of C on its way, rows padded by one
constexpr int EPI_WARPS = 8;
constexpr int EPI_THREADS = 32 * EPI_WARPS;
constexpr int NUM_THREADS = 64 + EPI_THREADS;
constexpr int SMEM_BUDGET = 226 * 1024;
constexpr int MAX_STAGES = 24;
constexpr int MAX_SPLIT = 8;            // SPLIT: a portable cluster
constexpr int MAX_K = 131071;           // 128 * 128 * K stays below 2^31
constexpr int MAX_ROWS = 0x7fffff00;    // tile arithmetic stays in int

enum { STREAM, SPLIT, LARGE, LARGE_PAIR };

struct Params {
  int M, N;           // STREAM, SPLIT with `swapped`: of the exchanged operands
  int swapped;        // what is called tokens here are rows of B, the channels rows of A
  int split;          // SPLIT: CTAs that share a tile's K
  int num_kc;         // K stages per tile
  int stages;
  int tt;             // tokens per tile (MMA N)
  int t_rows;         // token rows this CTA loads (half of tt in a pair)
  int t_stage_bytes;  // stage bytes of the tokens
  int pitch;          // SPLIT: of the sums in shared memory, elements a row of C
  int tmem_cols;      // two accumulators of half as many columns each
  int height;         // channels of a tile that this CTA loads (LARGE: 128)
  int c_stage_bytes;  // stage bytes of the channels
  int m_tiles;        // tiles of tokens, which run fastest
  int tiles;
  int w_prefetch;     // K stages of B prefetched into L2 before the dependency wait
  const float* sa;
  const float* sb;
  void* C;
  int* status;
  unsigned long long timeout_ns;
};

struct Tile {
  int c0;      // this CTA's first channel
  int m0;      // first token of the tile
};

// Tile i.
template <bool PAIR>
__device__ __forceinline__ Tile tile_at(const Params& p, int i, uint32_t rank) {
  Tile t;
  const int ct = i / p.m_tiles;
  t.m0 = (i - ct * p.m_tiles) * p.tt;
  t.c0 = (PAIR ? 2 * ct + static_cast<int>(rank) : ct) * p.height;
  return t;
}

// Ask for the tile of a CTA of this grid that has not started; 16 bytes of
// answer arrive at `answer`, counted on `bar`.
__device__ __forceinline__ void ask_tile(uint32_t answer, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
               "r"(bar)
               : "memory");
}

// The tile in an answer that has arrived, -1 if there was none left.
__device__ __forceinline__ int answered_tile(uint32_t answer) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, h;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(answer)
      : "memory");
  // the answer's bytes may be written again by the asynchronous proxy
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  return got ? static_cast<int>(x) : -1;
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

// Whether the phase is complete, at once (mbarrier.try_wait may wait a while).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// True in one lane of a converged warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void load32(uint32_t taddr, int (&v)[32]) {
  float f[2][16];
  tmem_ld16(taddr, f[0]);
  tmem_ld16(taddr + 16, f[1]);
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = __float_as_int(f[j / 16][j % 16]);
}

__device__ __forceinline__ void put(float* c, float v) { *c = v; }
__device__ __forceinline__ void put(__nv_bfloat16* c, float v) { *c = __float2bfloat16_rn(v); }

__device__ __forceinline__ int4 ld_cluster_v4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <int MODE, typename OUT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    gemm_i8_kernel(const __grid_constant__ CUtensorMap tm_t, const __grid_constant__ CUtensorMap tm_c, const Params p) {
  constexpr bool PAIR = MODE == LARGE_PAIR;
  constexpr bool FEW = MODE == STREAM || MODE == SPLIT;   // one tile of tokens, on the M side
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t s_t = smem_addr(smem);                                           // tokens' stages
  const uint32_t s_c = s_t + static_cast<uint32_t>(p.stages) * p.t_stage_bytes;   // channels' stages
  uint8_t* tail = smem + static_cast<size_t>(p.stages) * (p.c_stage_bytes + p.t_stage_bytes);
  const uint32_t bar0 = smem_addr(tail);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (p.stages + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * p.stages + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * p.stages + 2 + b); };
  const uint32_t drain_bar = bar0 + 8u * (2 * p.stages + 4);
  const uint32_t handover_bar = bar0 + 8u * (2 * p.stages + 5);   // pair: the other CTA's count of loads
  // STREAM: two answers in turn, one barrier each for "arrived" and "read by all"
  auto asked_bar = [&](int b) { return bar0 + 8u * (2 * p.stages + 6 + b); };
  auto read_bar = [&](int b) { return bar0 + 8u * (2 * p.stages + 8 + b); };
  __shared__ alignas(16) uint4 answers[2];
  uint8_t* misc = tail + 8 * (2 * p.stages + 10);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  volatile int* peer_issued = reinterpret_cast<volatile int*>(misc + 8);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR || MODE == SPLIT ? cluster_ctarank() : 0u;
  const bool leader = !PAIR || rank == 0;
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
    for (int b = 0; b < 2; ++b) {
      mbar_init(asked_bar(b), 1);
      mbar_init(read_bar(b), 1 + EPI_WARPS);   // the issuer and the epilogue's warps
    }
    *abort_flag = 0;
    *peer_issued = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_t);
    prefetch_tmap(&tm_c);
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
  const int first_tile = PAIR            ? static_cast<int>(blockIdx.x >> 1)
                         : MODE == SPLIT ? static_cast<int>(blockIdx.x) / p.split
                                         : static_cast<int>(blockIdx.x);
  // this CTA's part of K
  const int k_begin = MODE == SPLIT ? static_cast<int>(rank) * p.num_kc / p.split : 0;
  const int k_end = MODE == SPLIT ? (static_cast<int>(rank) + 1) * p.num_kc / p.split : p.num_kc;
  if (warp == 0 && lane == 0) {
    // B is a weight: its first stages may come into L2 while the kernel before
    // this one ends (L2 is the point of coherence, so nothing stale is seen
    // should that kernel write it after all)
    const Tile t = tile_at<PAIR>(p, first_tile, rank);
    for (int kc = k_begin; kc < k_begin + p.w_prefetch && kc < k_end; ++kc) tma_prefetch_l2_2d(&tm_c, kc * BK, t.c0);
  }
  pdl_wait();

  // The producer's and the issuer's loops are run by their whole warps, and one
  // lane issues: addresses, coordinates and descriptors then are in uniform
  // registers, where these instructions take them from, and each looks at the
  // next stage's barrier before it issues for this one (a barrier that is
  // complete still takes 160 clocks to be seen).  With the loops inside a branch
  // for one lane a stage took its producer 500 clocks and its issuer 710, which
  // bound every size.
  const bool elected = elect_one();
  auto wait = [&](uint32_t bar, uint32_t parity) {
    bool ok = true;
    uint64_t deadline = 0;   // of this wait, from the first look that was in vain
    while (ok && !mbar_try_wait(bar, parity)) {
      const uint64_t now = globaltimer_ns();
      if (deadline == 0) deadline = now + p.timeout_ns;
      if (*abort_flag) {
        ok = false;
      } else if (now > deadline) {   // both CTAs of a pair stop together
        ok = false;
        set_status(p.status, DFLASH_ERR_TIMEOUT);
        *abort_flag = 1;
        if (PAIR) st_shared_cluster_u32(peer_abort, 1u);
      }
    }
    return __all_sync(0xffffffffu, ok) != 0;
  };
  // The tile after `i`, the it-th of this CTA, in all lanes of a warp; -1 at
  // the end, or when a wait gives up.
  auto next_tile = [&](int i, int it, bool counted) {
    if (MODE == SPLIT) return -1;
    if (MODE != STREAM) {
      const int step = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);
      return i < p.tiles - step ? i + step : -1;
    }
    if (!wait(asked_bar(it & 1), (it >> 1) & 1)) return -1;
    const int n = __reduce_max_sync(0xffffffffu, answered_tile(smem_addr(answers + (it & 1))));
    if (counted && elected) mbar_arrive(read_bar(it & 1));
    return n;
  };

  int issued = 0;   // producer: stage loads issued, in ring order
  int asked = 0;    // producer: tiles asked for
  if (warp == 0) {
    const uint64_t pol_c = FEW ? l2_policy_evict_first() : l2_policy_evict_normal();
    const uint64_t pol_t = l2_policy_evict_last();
    int s = 0;
    uint32_t ph = 0;
    bool ok = true, ready = true;   // ready: the stage's barrier has been seen to be complete
    auto load = [&](uint32_t dst, const CUtensorMap* m, uint32_t fb, int x, int y, uint64_t pol) {
      if (PAIR)
        tma_load_2d_pair(dst, m, mapa_shared(fb, 0), x, y, pol);
      else
        tma_load_2d_hint(dst, m, fb, x, y, pol);
    };
    const uint32_t tx = static_cast<uint32_t>((PAIR ? 2 : 1) * (p.height + p.t_rows) * BK);
    for (int i = first_tile, it = 0; ok && i >= 0; i = ok ? next_tile(i, it, false) : -1, ++it) {
      if (MODE == STREAM) {   // the tile after this one, while this one loads
        if (it >= 2 && !wait(read_bar(it & 1), ((it >> 1) - 1) & 1)) break;
        if (elected) {
          mbar_arrive_expect_tx(asked_bar(it & 1), 16);
          ask_tile(smem_addr(answers + (it & 1)), asked_bar(it & 1));
        }
        ++asked;
      }
      const Tile t = tile_at<PAIR>(p, i, rank);
      const int t0 = t.m0 + (PAIR ? static_cast<int>(rank) * p.t_rows : 0);
      for (int kc = k_begin; kc < k_end; ++kc) {
        if (!ready && !wait(empty_bar(s), ph ^ 1u)) {
          ok = false;
          break;
        }
        const int s1 = s + 1 == p.stages ? 0 : s + 1;
        const uint32_t ph1 = s1 == 0 ? ph ^ 1u : ph;
        const bool peek = mbar_test(empty_bar(s1), ph1 ^ 1u);
        const uint32_t fb = full_bar(s), to_c = s_c + s * p.c_stage_bytes, to_t = s_t + s * p.t_stage_bytes;
        if (elected) {
          if (leader) mbar_arrive_expect_tx(fb, tx);
          load(to_c, &tm_c, fb, kc * BK, t.c0, pol_c);
          load(to_t, &tm_t, fb, kc * BK, t0, pol_t);
        }
        ++issued;
        ready = __all_sync(0xffffffffu, peek) != 0;
        s = s1;
        ph = ph1;
      }
    }
    if (PAIR && !leader && elected) {
      st_shared_cluster_u32(mapa_shared(smem_addr(const_cast<int*>(peer_issued)), 0), static_cast<uint32_t>(issued));
      mbar_arrive_cluster(mapa_shared(handover_bar, 0));   // release: the count is visible first
    }
  } else if (warp == 1) {
    if (leader) {
      const uint32_t idesc = umma_idesc_s8(PAIR ? 2 * CH : CH, FEW ? p.height : p.tt);
      int s = 0, tb = 0;
      uint32_t ph = 0, tph = 0;
      bool ok = true, ready = false;
      auto commit = [&](uint32_t bar) {
        if (PAIR)
          umma_commit_pair_multicast(bar, 0x3);
        else
          umma_commit(bar);
      };
      for (int i = first_tile, it = 0; ok && i >= 0; i = ok ? next_tile(i, it, true) : -1, ++it) {
        if (!wait(tempty_bar(tb), tph ^ 1u)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(tb * tmem_stride);
        for (int kc = k_begin; kc < k_end; ++kc) {
          if (!ready && !wait(full_bar(s), ph)) {
            ok = false;
            break;
          }
          const int s1 = s + 1 == p.stages ? 0 : s + 1;
          const uint32_t ph1 = s1 == 0 ? ph ^ 1u : ph;
          const bool peek = mbar_test(full_bar(s1), ph1);
          tc_fence_after();
          const uint64_t cdesc = umma_desc_sw128(s_c + s * p.c_stage_bytes);
          const uint64_t tdesc = umma_desc_sw128(s_t + s * p.t_stage_bytes);
          const uint64_t mdesc = FEW ? tdesc : cdesc, ndesc = FEW ? cdesc : tdesc;
          const uint32_t eb = empty_bar(s);
          if (elected) {
#pragma unroll
            for (int kk = 0; kk < BK / UMMA_K; ++kk)   // 32 bytes of K on: the address field counts 16
              umma_s8<PAIR>(d_tmem, mdesc + 2ull * kk, ndesc + 2ull * kk, idesc, ((kc - k_begin) | kk) != 0 ? 1u : 0u);
            commit(eb);
          }
          ready = __all_sync(0xffffffffu, peek) != 0;
          s = s1;
          ph = ph1;
        }
        if (!ok) break;
        if (elected) commit(tfull_bar(tb));
        if (++tb == 2) {
          tb = 0;
          tph ^= 1u;
        }
      }
      // every MMA issued has completed before TMEM is released
      if (elected) {
        if (PAIR)
          umma_commit_pair(drain_bar);
        else
          umma_commit(drain_bar);
      }
      const uint64_t dl = globaltimer_ns() + 50000000ull;
      while (!mbar_try_wait(drain_bar, 0) && globaltimer_ns() < dl) {
      }
    }
  } else {
    const int quarter = warp & 3;             // the TMEM lanes this warp may access
    const int half = (warp - 2) >> 2;         // which half of the tile's tokens
    const int nch = p.tt / 16, split = (nch + 1) >> 1;
    float* block = reinterpret_cast<float*>(tail + 8 * (2 * p.stages + 10) + 16) + (quarter * 2 + half) * BLOCK;
    int tb = 0;
    uint32_t tph = 0;
    for (int i = first_tile, it = 0; i >= 0; ++it) {
      const Tile t = tile_at<PAIR>(p, i, rank);
      if (!wait(tfull_bar(tb), tph)) break;
      tc_fence_after();
      const uint32_t taddr =
          tmem_base + static_cast<uint32_t>(tb * tmem_stride) + (static_cast<uint32_t>(quarter * 32) << 16);
      // FEW: this warp's tokens of the tile, a lane each
      const int m0 = t.m0 + quarter * 32, rows = min(min(32, p.tt - quarter * 32), p.M - m0);
      const float sa_row = MODE == STREAM && lane < rows ? __ldg(p.sa + m0 + lane) : 0.f;
      if constexpr (MODE == SPLIT) {
        // the sums over this CTA's part of K into the ring, which every load
        // and MMA is done with
        int* part = reinterpret_cast<int*>(smem);
        const int r = quarter * 32 + lane;
        for (int b = half; rows > 0 && b * 32 < p.height; b += 2) {
          int x[32];
          load32(taddr + b * 32, x);
          if (lane < rows) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              if (b * 32 + j >= p.height) break;   // a multiple of 16
              if (p.swapped) {
#pragma unroll
                for (int k = 0; k < 4; ++k) part[(b * 32 + j + k) * p.pitch + r] = x[j + k];
              } else {
                *reinterpret_cast<int4*>(part + r * p.pitch + b * 32 + j) = make_int4(x[j], x[j + 1], x[j + 2], x[j + 3]);
              }
            }
          }
        }
      } else if (MODE == STREAM && p.swapped) {
        // lanes are columns of C, registers its rows
        for (int b = half; rows > 0 && b * 32 < p.height && t.c0 + b * 32 < p.N; b += 2) {
          const int m = t.c0 + b * 32, tokens = min(min(32, p.height - b * 32), p.N - m);
          const float scale = lane < tokens ? __ldg(p.sb + m + lane) : 0.f;
          int x[32];
          load32(taddr + b * 32, x);
          OUT* c = static_cast<OUT*>(p.C) + static_cast<size_t>(m) * p.M + m0 + lane;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float v = __int2float_rn(x[j]) * __shfl_sync(0xffffffffu, scale, j) * sa_row;
            if (j < tokens && lane < rows) put(c, v);
            c += p.M;
          }
        }
      } else if constexpr (MODE == STREAM) {
        // blocks of 32 tokens (this warp's lanes) x 32 channels; the two warps
        // of a quarter take every other block
        for (int b = half; rows > 0 && b * 32 < p.height && t.c0 + b * 32 < p.N; b += 2) {
          int x[32];
          load32(taddr + b * 32, x);
#pragma unroll
          for (int j = 0; j < 32; ++j) block[lane * 33 + j] = __int2float_rn(x[j]) * sa_row;
          __syncwarp();
          const int n = t.c0 + b * 32 + lane;
          if (b * 32 + lane < p.height && n < p.N) {
            const float sbn = __ldg(p.sb + n);
            OUT* c = static_cast<OUT*>(p.C) + static_cast<size_t>(m0) * p.N + n;
#pragma unroll 8
            for (int r = 0; r < rows; ++r) put(c + static_cast<size_t>(r) * p.N, block[r * 33 + lane] * sbn);
          }
          __syncwarp();
        }
      } else {
        const int n = t.c0 + quarter * 32 + lane;
        const bool mine = quarter * 32 + lane < p.height && n < p.N;
        const float sbn = mine ? __ldg(p.sb + n) : 0.f;
        const int ch_end = __any_sync(0xffffffffu, mine) ? (half ? nch : split) : 0;
        for (int ch = half ? split : 0; ch < ch_end; ch += 2) {
          const int m = t.m0 + ch * 16;
          if (m >= p.M) break;
          // two chunks of 16 tokens (one at the end), their scales a lane each
          const int rows = min(p.M - m, 16 * min(2, ch_end - ch));
          const float sam = lane < rows ? __ldg(p.sa + m + lane) : 0.f;
          int x[32];
          load32(taddr + ch * 16, x);
          OUT* c = static_cast<OUT*>(p.C) + static_cast<size_t>(m) * p.N + n;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float v = __int2float_rn(x[j]) * __shfl_sync(0xffffffffu, sam, j) * sbn;
            if (j < rows && mine) put(c, v);
            c += p.N;
          }
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
      i = next_tile(i, it, true);
    }
  }

  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  if (MODE == SPLIT) {
    // every CTA adds up its share of the tile's elements over the cluster
    cluster_sync_all();
    const Tile t = tile_at<false>(p, first_tile, 0);
    const int across = min(p.height, p.N - t.c0), down = min(p.tt, p.M - t.m0);
    const int rows = p.swapped ? across : down, cols = p.swapped ? down : across;   // of C
    const int m0 = p.swapped ? t.c0 : t.m0, n0 = p.swapped ? t.m0 : t.c0;
    const float* sa = (p.swapped ? p.sb : p.sa) + m0;
    const float* sb = (p.swapped ? p.sa : p.sb) + n0;
    const size_t ld = p.swapped ? p.M : p.N;
    OUT* c = static_cast<OUT*>(p.C) + m0 * ld + n0;
    const int fours = (cols + 3) / 4, total = rows * fours;   // four elements a thread
    const int end = static_cast<int>((rank + 1) * total / p.split);
    uint32_t from[MAX_SPLIT];
#pragma unroll
    for (int q = 0; q < MAX_SPLIT; ++q) from[q] = mapa_shared(s_t, q < p.split ? q : 0);
    for (int e = static_cast<int>(rank * total / p.split) + static_cast<int>(threadIdx.x); e < end; e += NUM_THREADS) {
      const int m = e / fours, n = 4 * (e - m * fours);
      const float sam = __ldg(sa + m);
      float sbn[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) sbn[k] = n + k < cols ? __ldg(sb + n + k) : 0.f;
      const uint32_t off = 4u * (m * p.pitch + n);
      int x[4] = {0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < MAX_SPLIT; ++q) {
        if (q >= p.split) break;
        const int4 v = ld_cluster_v4(from[q] + off);
        x[0] += v.x;
        x[1] += v.y;
        x[2] += v.z;
        x[3] += v.w;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (n + k < cols) put(c + m * ld + n + k, __int2float_rn(x[k]) * sam * sbn[k]);
    }
    __syncwarp();
    cluster_sync_all();   // nobody's part is read any more
  }
  if (PAIR) cluster_sync_all();   // every role of both CTAs is done: abort flags and counts are final
  if (warp == 0 && elected && leader && *abort_flag != 0) {
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
    for (int it = max(asked - 2, 0); it < asked; ++it)
      while (!mbar_try_wait(asked_bar(it & 1), (it >> 1) & 1) && globaltimer_ns() < dl) {
      }
  }
  if (PAIR && *abort_flag != 0) {   // set in both CTAs or in neither
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
  // Rows that start inside a line cost two lines a stage, and fetching wider ones
  // then costs more than it gives: us with 256 bytes / without, [333 x 4099 x
  // 2576] 12.0 / 11.1, [96 x 100000 x 2576] 72.8 / 69.7, [2000 x 40000 x 2576] 250 /
  // 235; [96 x 151936 x 5120] 149 / 154.
  const bool whole = ((reinterpret_cast<uintptr_t>(base) | static_cast<uintptr_t>(cols)) & 127) == 0;
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            whole ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// At every launch: the attribute belongs to the current device and context.
template <int MODE, typename OUT>
static cudaError_t allow_smem() {
  return cudaFuncSetAttribute(gemm_i8_kernel<MODE, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BUDGET);
}

// Clusters of 2, 4 or 8 CTAs with all of the shared memory that can be resident
// at once on the current device (0: they cannot run), asked once per device.
template <int MODE>
static int max_clusters(int size) {
  constexpr int MAX_DEVICES = 64;
  static std::atomic<int> known[MAX_DEVICES][4];   // the count plus one; 0: not asked yet
  const int which = size == 2 ? 1 : size == 4 ? 2 : 3;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < MAX_DEVICES) {
    const int k = known[dev][which].load(std::memory_order_relaxed);
    if (k > 0) return k - 1;
  }
  if (allow_smem<MODE, float>() != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size);
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = SMEM_BUDGET;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int c = 0;
  if (cudaOccupancyMaxActiveClusters(&c, gemm_i8_kernel<MODE, float>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev < MAX_DEVICES) known[dev][which].store(c + 1, std::memory_order_relaxed);
  return c;
}

struct Plan {
  Params p;
  int mode;
  int grid;
};

// STREAM: an MMA reads 128 rows from its token stage's start.  What lies past
// the stage is never read back, but has to be shared memory of the CTA: the
// span of the last stage ends inside the ring or what follows it.
static size_t smem_bytes(const Plan& pl) {
  const Params& p = pl.p;
  const size_t ring = static_cast<size_t>(p.stages) * (p.c_stage_bytes + p.t_stage_bytes);
  const size_t span = static_cast<size_t>(p.stages - 1) * p.t_stage_bytes + CH * BK;
  const size_t blocks = pl.mode == STREAM ? sizeof(float) * BLOCK * 2 * ((p.tt + 31) / 32) : 0;
  return 1024 + std::max(ring + 8 * (2 * p.stages + 10) + 16 + blocks, span);
}

// Tiles of up to 128 tokens x up to 256 channels: STREAM or SPLIT.  Returns
// the estimated time in tenths of a clock, -1 if such a tile would not do.
//
// Few tiles: K over clusters of 2, 4 or 8 CTAs, higher tiles for it.  The
// estimate is a fit of what was measured, in clocks: a stage 380, or 2.2 a row
// of either operand, or 170 and 4.2 a channel where no other CTA reads the same
// channels; an element of the tile 0.32 on its way to C; the cluster's barriers
// and the other CTAs' sums 1400; more than one tile of tokens 1000 to 1400.  us
// with 1, 2, 4 and 8 CTAs to a tile, the choice starred: [8 x 64 x 5120] 11.2,
// 7.0, 5.3, 4.6*; [8 x 2560 x 2560] 7.3, 6.2, 6.1*, 6.5; [128 x 2560 x 2560] 8.0,
// 7.3*, 7.4, 10.0; [128 x 5120 x 5120] 12.9, 10.6*, 11.4; [8 x 5120 x 640] 4.3*,
// 5.1, 5.8; [8 x 10000 x 5120] 13.9, 12.4*; [4352 x 5 x 5120] 12.1, 9.3*, 9.1.
static long long plan_few(int sms, Plan& pl) {
  Params& p = pl.p;
  p.m_tiles = (p.M + CH - 1) / CH;
  p.tt = ((p.M + p.m_tiles - 1) / p.m_tiles + 15) & ~15;
  p.t_rows = p.tt;
  const int units = (p.N + 15) / 16;
  long long best = -1;
  for (int split = 1; split <= MAX_SPLIT && split <= p.num_kc; split *= 2) {
    const int at_once = (split == 1 ? sms : max_clusters<SPLIT>(split)) / p.m_tiles;
    if (at_once < 1) continue;
    // the highest tiles of which every SM gets the same number: fewer tiles
    // are fewer MMAs, and less is read of the tokens for each ([8 x 151936 x
    // 2560]: 13 units high 66 us, 16 units, four for each SM and two left over,
    // 70; 8 units 77)
    const int most = MAX_N / 16 * at_once;
    const int rounds = split == 1 && p.m_tiles == 1 ? (units + most - 1) / most : 1;
    const int h = (units + rounds * at_once - 1) / (rounds * at_once);
    if (h * 16 > MAX_N) continue;
    const long long stage =
        std::max({3800, 22 * (16 * h + p.tt), p.m_tiles == 1 ? 1700 + 42 * 16 * h : 0});
    const long long cost = rounds * ((p.num_kc + split - 1) / split * stage + 51LL * p.tt * h) +
                           (p.m_tiles == 1 ? (split > 1 ? 14000 : 0) : (split > 1 ? 28000 : 10000));
    if (best < 0 || cost < best) {
      best = cost;
      p.split = split;
      p.height = 16 * h;
    }
  }
  if (best < 0) return -1;
  pl.mode = p.split > 1 ? SPLIT : STREAM;
  p.pitch = p.swapped ? (p.tt + 3) & ~3 : p.height + 4;
  p.tiles = (p.N + p.height - 1) / p.height * p.m_tiles;
  pl.grid = p.tiles * p.split;
  return best;
}

static bool make_plan(int M, int N, int K, int sms, Plan& pl) {
  Params& p = pl.p;
  p = Params{};
  p.M = M;
  p.N = N;
  p.num_kc = (K + BK - 1) / BK;
  if (M <= CH || N <= CH) {
    p.swapped = M > CH;
    if (p.swapped) std::swap(p.M, p.N);
    if (plan_few(sms, pl) < 0) return false;
  } else {
    const int pairs = pair_allowed() ? max_clusters<LARGE_PAIR>(2) : 0;
    const bool pair = pairs >= 1;
    const int units = pair ? (pairs < sms / 2 ? pairs : sms / 2) : sms;
    const int ch = pair ? 2 * CH : CH;
    const long long c_tiles = (static_cast<long long>(N) + ch - 1) / ch;
    // tokens per tile: the fewest rounds of tiles, a tile's time being that
    // of its operands' bytes, which come at 57 B/ns to an SM (channels plus
    // tokens; [448 x 151936 x 2560]: 6.8, 8.3, 9.5 and 11.6 us a tile of 64,
    // 128, 192 and 256)
    long long best = -1;
    int tt = 0;
    for (int t = MAX_N; t >= 32; t -= 32) {
      const long long tiles = c_tiles * ((M + t - 1) / t);
      const long long cost = (tiles + units - 1) / units * (ch + t);
      if (best < 0 || cost < best) {
        best = cost;
        tt = t;
      }
    }
    const long long m_tiles = (M + tt - 1) / tt, tiles = c_tiles * m_tiles;
    if (tiles > 0x7fffffffLL) return false;
    // Few tiles of pairs, a long K: the other tiles with K split, if they are
    // estimated to take less.  A stage of a pair 380 clocks, or 3.3 a token,
    // a token's accumulators 27 on their way to C, 500 for the pair's barriers.
    // us, pairs / the others: [130 x 300 x 5120] 10.6 / 6.7*, [192 x 1024 x 5120]
    // 10.7 / 8.1*, [600 x 600 x 5120] 11.7 / 9.7*, [2000 x 300 x 5120] 13.3 / 10.5*,
    // [200 x 5120 x 2560] 8.5* / 10.1, [448 x 5120 x 5120] 15.8* / 18.4.
    const long long cost = (tiles + units - 1) / units * p.num_kc * std::max(3800, 33 * tt) + 270LL * tt + 5000;
    bool few = false;
    if (pair && M <= CH * sms) {
      const long long other = plan_few(sms, pl);
      few = other >= 0 && other < cost;
    }
    if (!few) {
      pl.mode = pair ? LARGE_PAIR : LARGE;
      p.split = 1;
      p.tt = tt;
      p.m_tiles = static_cast<int>(m_tiles);
      p.tiles = static_cast<int>(tiles);
      p.t_rows = pair ? tt / 2 : tt;
      p.height = CH;
      const int used = tiles < units ? static_cast<int>(tiles) : units;
      pl.grid = pair ? 2 * used : used;
    }
  }
  p.t_stage_bytes = p.t_rows * BK;
  p.c_stage_bytes = p.height * BK;
  p.tmem_cols = 32;
  const int columns = ((pl.mode == STREAM || pl.mode == SPLIT ? p.height : p.tt) + 31) & ~31;   // read in blocks of 32
  while (p.tmem_cols < 2 * columns) p.tmem_cols *= 2;
  for (p.stages = MAX_STAGES; p.stages > 2 && smem_bytes(pl) > SMEM_BUDGET;) --p.stages;
  return smem_bytes(pl) <= SMEM_BUDGET;
}

template <int MODE, typename OUT>
static cudaError_t launch_as(const Plan& pl, const CUtensorMap& tt, const CUtensorMap& tc, cudaStream_t st) {
  const cudaError_t e = allow_smem<MODE, OUT>();
  if (e != cudaSuccess) return e;
  return launch_kernel_cluster(gemm_i8_kernel<MODE, OUT>, dim3(pl.grid), dim3(NUM_THREADS), smem_bytes(pl), st,
                               MODE == LARGE_PAIR ? 2 : MODE == SPLIT ? pl.p.split : 1, tt, tc, pl.p);
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
  p.w_prefetch = (pl.mode == STREAM || pl.mode == SPLIT) && !p.swapped ? 8 : 0;
  p.sa = p.swapped ? sb : sa;
  p.sb = p.swapped ? sa : sb;
  p.C = C;
  p.status = dev_status;
  p.timeout_ns = timeout_ns_from_env();
  CUtensorMap tt, tc;
  const bool ok = gi8::make_map(&tt, p.swapped ? B : A, p.swapped ? N : M, K, p.t_rows) &&
                  gi8::make_map(&tc, p.swapped ? A : B, p.swapped ? M : N, K, p.height);
  if (!ok) return DFLASH_ERR_CUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (pl.mode == STREAM)
    e = c_bf16 ? launch_as<STREAM, __nv_bfloat16>(pl, tt, tc, st) : launch_as<STREAM, float>(pl, tt, tc, st);
  else if (pl.mode == SPLIT)
    e = c_bf16 ? launch_as<SPLIT, __nv_bfloat16>(pl, tt, tc, st) : launch_as<SPLIT, float>(pl, tt, tc, st);
  else if (pl.mode == LARGE_PAIR)
    e = c_bf16 ? launch_as<LARGE_PAIR, __nv_bfloat16>(pl, tt, tc, st) : launch_as<LARGE_PAIR, float>(pl, tt, tc, st);
  else
    e = c_bf16 ? launch_as<LARGE, __nv_bfloat16>(pl, tt, tc, st) : launch_as<LARGE, float>(pl, tt, tc, st);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
