// Matrix product of e4m3 codes with block scales for many rows, sm_100a:
//
//   Y[m, n] = sum_g sx[g][m] sw[n / 128][g] P_g[m, n]  (+ bias[n])
//   P_g[m, n] = sum_{k in g} X[m, k] W[n, k]
//
// P_g comes from the tensor cores (tcgen05.mma kind::f8f6f4, fp32 sums).  Its
// factor changes with every group of 128 columns of K and is any fp32 number,
// so the sum over g cannot stay in the tensor cores' accumulator: P_g of each
// group is read from TMEM and added to fp32 registers with its factor.
//
// Structure: clusters of two CTAs on neighbouring SMs (a CTA pair), one CTA
// per SM, persistent over 256 x BN tiles.  Each CTA loads its own 128 rows of
// X and BN / 2 rows of W per group (TMA, 128-byte swizzle, completing on the
// leader's barrier), keeps its 128 rows of P_g in its own TMEM, sums and
// writes them.  No multicast.
//   warps 0, 3  TMA producers, every second group each
//   warps 1, 2  in the leader, issue the MMAs of every second group each (4 of
//               256 x 128 x 32 per unit), round-robin over the TMEM buffers
//   warps 4-11  two per TMEM lane quarter, one row per thread and half of the
//               tile's columns: they add P_g times sx sw to BN / 2 registers
//               and write Y at the tile's end, while the next tile's first
//               two groups already run
//
// A group of a 256-wide tile is computed in two units of 128 columns (64 of
// each CTA's rows of W), so that four TMEM buffers are in turn: from a
// buffer's MMAs to its next pass the commit, a read, the arrivals of both
// CTAs at the leader and an issue, each of them a poll or two of barriers,
// which take 100 to 200 cycles while the MMAs read shared memory.  For the
// same reason the loads and the MMAs are issued by two warps each, a waiting
// warp polls its barriers together or ahead of need, and the scales come in
// boxes of 16 groups.
//
// What bounds it: no unit alone.  Time over groups of the fullest pair, tile
// ends included, at 2048 x 12288 x 49152, and with parts left out in scratch
// builds (ns; alone, at 128 and 256 columns):
//   all                                261   518
//   without the multiply-adds          221   422
//   nor the reads of the sums          218   404
//   nor the MMAs: loads and barriers   179   252
// The tensor cores' own time is 130 and 260, the multiply-adds' (128 x 128 and
// 128 x 256 by eight warps) 67 and 133.  At 128 columns the loads, 24 KB per SM
// and group from L2 (20 TB/s over all SMs), are most of it, and MMAs and loads
// together, which meet in shared memory, nearly all the rest; at 256 columns
// the loads are lighter per column, and the chain of a group (MMAs, poll, read,
// hand-back, adds) is what does not overlap.  Per column the two are equal.
// 2048 x 12288 x 49152 takes 1030 to 1073 us alone over several machines, 0.71
// to 0.74 of twice the measured bf16 rate; 2048 x 8192 x 8192 115 us at 128
// columns and 132 at 256.  Back to back the power cap takes the clock to 1.43
// GHz, and 2048 x 12288 x 49152 to 1230 to 1265 us.
//
// BN: 256 or 128, by the pairs' rounds (block_pair_width).  Widths of 160 and
// 192, whose halves straddle blocks of the weight scales, took 5% and 18% more
// per column.
//
// Every wait is bounded; a timeout sets the status word and the CTA drains
// and exits.
#include "block8.cuh"
#include "block8_gemm.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

#include <algorithm>

namespace i8mm {
namespace {

constexpr int TILE_M = 256;
constexpr int BM = 128;  // rows per CTA
constexpr int EPI_WARPS = 8;
// Three warpgroups, so that registers can move between them: launched with
// 168 each (384 x 168 = 64512), the first (two producers, two MMA
// issuers) goes down to 40 and the two epilogue groups up to 232
// (128 x 40 + 256 x 232 = 64512).
constexpr int THREADS = 128 + 32 * EPI_WARPS;
constexpr int REGS_LAUNCH = 168, REGS_FRONT = 40, REGS_EPI = 232;
static_assert(128 * REGS_FRONT + 32 * EPI_WARPS * REGS_EPI <= THREADS * REGS_LAUNCH, "registers within the launch's");

// Scales of a CTA's rows come up to SX_CHUNK groups of one tile at a time, two
// chunks in turn.
constexpr int SX_CHUNK = kSxChunk;

template <int BN>
struct PCfg {
  static constexpr int A_BYTES = BM * kGroup;
  static constexpr int B_BYTES = BN / 2 * kGroup;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = 212992 / STAGE;
  static constexpr int HALF = BN / 2;  // columns per epilogue warp
  // A group of a wide tile is computed in two units of half its columns (half
  // from each CTA's rows of W), each with a TMEM buffer of its own.
  static constexpr int UNITS = BN / 128;
  static constexpr int UNIT = 128;
  static constexpr int BUFS = 4;
  static constexpr int ISSUERS = 2;       // warps that issue MMAs, every second group each
  static constexpr int CW = HALF / UNITS;  // an epilogue warp's columns of a unit
  static constexpr int NBARS = 2 * STAGES + 2 * BUFS + ISSUERS + 4;
  static constexpr int SX_OFF = STAGES * STAGE;
  static constexpr int BAR_OFF = SX_OFF + 2 * SX_CHUNK * BM * 4;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
  static constexpr int SMEM = MISC_OFF + 16 + 1024;  // + slack to align the base to 1024
  static constexpr uint32_t IDESC = idesc_f16_f32(TILE_M, UNIT);  // e4m3 and fp16 operands share the encoding 0
  static_assert((BN == 128 || BN == 256) && STAGE % 1024 == 0 && SMEM <= 232448, "tile shape");
};

// D[tmem of both CTAs] (+)= A * B^T over the pair's shared memory, e4m3 to fp32.
__device__ __forceinline__ void mma_e4m3_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 1 in one lane of the (converged) warp, 0 in the others.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint64_t make_desc(uint32_t lo, uint32_t hi) {
  return (static_cast<uint64_t>(hi) << 32) | lo;
}

__device__ __forceinline__ void gfail(const BlockGemmArgs& a, volatile int* abort_flag) {
  *abort_flag = 1;
  atomicOr(a.status, kStatusTimeout);
}

// Arrive on a barrier of either CTA of the pair without ordering this
// thread's memory accesses: what it hands over is a TMEM buffer, whose reads
// tcgen05.wait::ld has completed.  A release at cluster scope instead waits
// for every outstanding load of the thread, here the scales fetched ahead,
// once per group: 2048 x 12288 x 49152 took 2666 us with it.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// acc (two fp32) += p (two fp32) * s (two fp32), each rounded once.
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t p0, uint32_t p1, uint64_t s) {
  asm("{\n\t.reg .b64 p;\n\tmov.b64 p, {%1, %2};\n\tfma.rn.f32x2 %0, p, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(p0), "r"(p1), "l"(s));
}
__device__ __forceinline__ uint64_t twice(float s) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(s));
  return r;
}
__device__ __forceinline__ float2 halves(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}

__device__ __forceinline__ float lds_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// W columns of this thread's TMEM lane, and the wait for them.  The
// registers go through the wait, so that no use of them can move above it.
template <int W>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[W]) {
#pragma unroll
  for (int c = 0; c + 32 <= W; c += 32) tmem_ld_32x32b_x32(taddr + c, *reinterpret_cast<uint32_t(*)[32]>(&r[c]));
  if constexpr (W % 32 != 0) tmem_ld_32x32b_x16(taddr + W / 32 * 32, &r[W / 32 * 32]);
}
template <int W>
__device__ __forceinline__ void tmem_wait_cols(uint32_t (&r)[W]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < W; i += 16)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                 "+r"(r[i + 6]), "+r"(r[i + 7]), "+r"(r[i + 8]), "+r"(r[i + 9]), "+r"(r[i + 10]), "+r"(r[i + 11]),
                 "+r"(r[i + 12]), "+r"(r[i + 13]), "+r"(r[i + 14]), "+r"(r[i + 15])::"memory");
}

// Polls a barrier without suspending, the whole warp together (see
// mbar_wait2_warp).
__device__ __forceinline__ bool mbar_wait_poll(uint32_t bar, uint32_t parity, unsigned long long tmo,
                                               volatile int* abort_flag) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    if ((i & 4095u) == 0) {
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (__any_sync(0xffffffffu, *abort_flag != 0 || now - t0 > tmo)) return false;
    }
  }
}

template <int BN, typename TY>
__global__ void __launch_bounds__(THREADS, 1)
    block_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                           const __grid_constant__ CUtensorMap tmS, const BlockGemmArgs a) {
  using C = PCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + C::BUFS;
  uint64_t* drain = tempty + C::BUFS;
  uint64_t* sfull = drain + C::ISSUERS;
  uint64_t* sempty = sfull + 2;
  float* sx_s = reinterpret_cast<float*>(smem + C::SX_OFF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int M = a.M, N = a.N;
  const uint32_t rank = cluster_ctarank();
  const int tile0 = static_cast<int>(blockIdx.x) / 2;
  const int tstride = static_cast<int>(gridDim.x) / 2;
  const int num_m = (M - 1) / TILE_M + 1;  // M + TILE_M may pass 2^31
  const int num_tiles = num_m * ((N - 1) / BN + 1);
  const int G = (a.K + kGroup - 1) / kGroup;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::BUFS; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], EPI_WARPS * 2);
    }
    for (int s = 0; s < C::ISSUERS; ++s) mbar_init(&drain[s], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sempty[s], EPI_WARPS);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmS);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();  // the peer's barriers are initialised before any remote arrive
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const unsigned long long tmo = a.timeout_ns;
  if (warp == 0 && tile0 < num_tiles && elect_one()) {
    // the first tiles of W into L2 while the stream's previous kernel ends: a
    // hint that needs no order with it (a tile lies within N_pad)
    const int row = tile0 / num_m * BN + static_cast<int>(rank) * (BN / 2);
    for (int g = 0; g < min(G, C::STAGES); ++g)
      bulk_prefetch_l2(a.Wb + (static_cast<size_t>(g) * a.N_pad + row) * kGroup, C::B_BYTES);
  }
  __syncwarp();
  dependency_wait();

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_FRONT));
    if (warp == 0 || warp == 3) {
      // ----------------------------------------------------- TMA producers
      // Every second group each: its wait and loads take one warp longer than
      // its MMAs take the tensor cores.  Both CTAs' loads complete on the
      // leader's barrier; its producer announces the pair's bytes.
      const int mine = warp == 0 ? 0 : 1;
      const uint32_t issuer = elect_one();
      const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0);
      int stage = mine, g = mine, t = tile0;
      uint32_t phase = 1, chunk0 = 0;  // chunk0: scale chunks of the tiles before t
      const uint32_t chunks = static_cast<uint32_t>((G + SX_CHUNK - 1) / SX_CHUNK);
      bool ok = true;
      const uint64_t pol_x = l2_policy_evict_last();  // every column tile of its rows reads X again
      while (ok) {
        while (g >= G && t < num_tiles) {
          g -= G;
          t += tstride;
          chunk0 += chunks;
        }
        if (t >= num_tiles) break;
        const int m0 = (t % num_m) * TILE_M + static_cast<int>(rank) * BM;
        const int w0 = (t / num_m) * BN + static_cast<int>(rank) * (BN / 2);
#pragma unroll 1
        for (; g < G && ok; g += 2) {
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], phase, tmo, abort_flag));
          if (ok && g % SX_CHUNK == 0) {
            // the scales of up to 16 groups of this CTA's rows, one box
            const uint32_t chunk = chunk0 + static_cast<uint32_t>(g / SX_CHUNK);
            ok = __all_sync(0xffffffffu, mbar_wait(&sempty[chunk & 1u], ((chunk >> 1) & 1u) ^ 1u, tmo, abort_flag));
            if (ok && issuer) {
              mbar_arrive_expect_tx(&sfull[chunk & 1u], SX_CHUNK * BM * 4);
              tma_load_2d(sx_s + (chunk & 1u) * (SX_CHUNK * BM), &tmS, &sfull[chunk & 1u], m0, g);
            }
          }
          if (ok && issuer) {
            uint8_t* st = smem + stage * C::STAGE;
            const uint32_t bar = full0 + static_cast<uint32_t>(stage) * 8u;
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * C::STAGE);
            tma_load_2d_pair_hint(st, &tmX, bar, g * kGroup, m0, pol_x);
            tma_load_2d_pair(st + C::A_BYTES, &tmW, bar, 0, g * a.N_pad + w0);
          }
          __syncwarp();
          stage += 2;
          if (stage >= C::STAGES) {
            stage -= C::STAGES;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        // the loads already issued land, microseconds later, before the CTA exits
        if (issuer) gfail(a, abort_flag);
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 200000ull) {
        }
      }
    } else if (warp <= C::ISSUERS) {
      if (rank == 0) {
        // ------------------------------------------------------- MMA issuers
        // Every ISSUERS-th group: a group's waits and issue take one warp longer
        // than its MMAs take the tensor cores.  The whole warp walks the loop
        // and one elected lane issues: the descriptors then stay in uniform
        // registers.
        const uint32_t issuer = elect_one();
        const uint32_t desc_hi = static_cast<uint32_t>(smem_desc_k_sw128(0) >> 32);
        const uint32_t desc_lo = static_cast<uint32_t>(smem_desc_k_sw128(smem_u32(smem)));
        int stage = warp - 1, buf = C::UNITS * (warp - 1);
        uint32_t phase = 0, bphase = 1;
        bool ok = true;
        const int my_tiles = tile0 < num_tiles ? (num_tiles - tile0 + tstride - 1) / tstride : 0;
        for (long long it = warp - 1; it < static_cast<long long>(my_tiles) * G && ok; it += C::ISSUERS) {
#pragma unroll
          for (int u = 0; u < C::UNITS; ++u) {
            ok = ok && mbar_wait2_warp(&full[stage], phase, &tempty[buf + u], bphase, tmo, abort_flag);
            if (ok) {
              tc_fence_after();
              if (issuer) {
                const uint32_t ad = desc_lo + static_cast<uint32_t>(stage * (C::STAGE >> 4));
                const uint32_t bd = ad + static_cast<uint32_t>((C::A_BYTES + u * C::CW * kGroup) >> 4);
                const uint32_t d = tmem_base + static_cast<uint32_t>((buf + u) * C::UNIT);
#pragma unroll
                for (int kk = 0; kk < kGroup / 32; ++kk)  // 32 bytes along K inside the 128-byte swizzled row
                  mma_e4m3_pair(d, make_desc(ad + kk * 2, desc_hi), make_desc(bd + kk * 2, desc_hi), C::IDESC, kk != 0);
                mma_commit_pair(&tfull[buf + u], 0x3);
                if (u == C::UNITS - 1) mma_commit_pair(&empty[stage], 0x3);  // frees the stage in both CTAs
              }
              __syncwarp();
            }
          }
          buf += C::UNITS * C::ISSUERS;
          if (buf >= C::BUFS) {
            buf -= C::BUFS;
            bphase ^= 1u;
          }
          stage += C::ISSUERS;
          if (stage >= C::STAGES) {
            stage -= C::STAGES;
            phase ^= 1u;
          }
        }
        if (!ok && issuer) {
          gfail(a, abort_flag);
          mma_commit_pair(&drain[warp - 1], 0x1);
          mbar_wait(&drain[warp - 1], 0, tmo, nullptr);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPI));
    // ----------------------------------------------------- sums and epilogue
    const int q = warp & 3;             // TMEM lane quarter this warp may read
    const int h = (warp - 4) >> 2;      // half of the tile's columns
    const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(h * C::CW);
    const uint32_t tempty0 = mapa_shared(smem_u32(&tempty[0]), 0);
    uint32_t chunk = 0, buf = 0, ph = 0;
    bool alive = true;
    const uint32_t tfull0 = smem_u32(&tfull[0]);
    const uint32_t sx0 = smem_u32(sx_s) + static_cast<uint32_t>(q * 32 + lane) * 4u;
    for (int t = tile0; t < num_tiles && alive; t += tstride) {
      const int m = (t % num_m) * TILE_M + static_cast<int>(rank) * BM + q * 32 + lane;
      const int nh = (t / num_m) * BN + h * C::HALF;
      const bool row_ok = m < M;
      // the weight scales of the half-tile's block (past N: the last block's,
      // the sums are dropped), one group per lane, a chunk ahead
      const float* swp = a.sw + static_cast<size_t>(min(nh / kGroup, (N - 1) / kGroup)) * G;
      auto weight_scale = [&](int g) { return __ldg(swp + min(g + lane, G - 1)); };
      float wn = weight_scale(0);
      uint64_t acc[C::HALF / 2];
#pragma unroll
      for (int i = 0; i < C::HALF / 2; ++i) acc[i] = 0ull;
      // (the row's scales come through shared memory: with the next ones on
      // their way from global memory, tcgen05.wait::ld waited for them too)
      bool ready = false;  // the next group was complete when polled during the last one
#pragma unroll 1
      for (int g0 = 0; g0 < G && alive; g0 += SX_CHUNK, ++chunk) {
        const float w = wn;
        wn = weight_scale(g0 + SX_CHUNK);
        alive = __all_sync(0xffffffffu, mbar_wait(&sfull[chunk & 1u], (chunk >> 1) & 1u, tmo, abort_flag));
        uint32_t sx = sx0 + (chunk & 1u) * (SX_CHUNK * BM * 4);
        const int n = min(SX_CHUNK, G - g0);
#pragma unroll 1
        for (int j = 0; j < n && alive; ++j, sx += BM * 4) {
          const float x = lds_f32(sx);
          const uint64_t sc = twice(__fmul_rn(x, __shfl_sync(0xffffffffu, w, j)));
#pragma unroll
          for (int u = 0; u < C::UNITS; ++u) {
            if (alive && !__all_sync(0xffffffffu, ready))
              alive = mbar_wait_poll(tfull0 + buf * 8u, ph, tmo, abort_flag);
            tc_fence_after();
            uint32_t r[C::CW];
            tmem_ld_cols<C::CW>(t_row + buf * C::UNIT, r);
            tmem_wait_cols<C::CW>(r);
            tc_fence_before();  // the buffer is read: hand it back to the leader
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(tempty0 + buf * 8u);
            if (++buf == C::BUFS) {
              buf = 0;
              ph ^= 1u;
            }
            ready = mbar_test_wait(tfull0 + buf * 8u, ph);
#pragma unroll
            for (int i = 0; i < C::CW / 2; ++i)
              fma2(acc[u * C::CW / 2 + i], r[2 * i], r[2 * i + 1], sc);
          }
        }
        __syncwarp();
        if (lane == 0 && !(a.skip_scales && warp == 4 && rank == 1)) mbar_arrive(&sempty[chunk & 1u]);
      }
      if (!alive) {
        if (lane == 0) gfail(a, abort_flag);
        break;
      }
      if (row_ok) {
        TY* yp = static_cast<TY*>(a.Y) + static_cast<size_t>(m) * N + nh;
        const TY* bp = static_cast<const TY*>(a.bias) + nh;
        const bool y32 = (reinterpret_cast<uintptr_t>(a.Y) & 31u) == 0;
#pragma unroll
        for (int c = 0; c < C::HALF / 16; ++c) {  // 16 columns at a time; N is a multiple of 16
          if (nh + c * 16 < N) {
            uint4 o[2];
            uint32_t* ow = reinterpret_cast<uint32_t*>(o);
            uint4 b[2] = {};
            if (a.bias != nullptr) {
              b[0] = __ldg(reinterpret_cast<const uint4*>(bp + c * 16));
              b[1] = __ldg(reinterpret_cast<const uint4*>(bp + c * 16) + 1);
            }
            const uint32_t* bw = reinterpret_cast<const uint32_t*>(b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float2 v = halves(acc[c * 8 + i]);
              if (a.bias != nullptr) {
                const float2 bb = pair_to_float<TY>(bw[i]);
                v.x = __fadd_rn(v.x, bb.x);
                v.y = __fadd_rn(v.y, bb.y);
              }
              ow[i] = float_to_pair<TY>(v.x, v.y);
            }
            uint4* d = reinterpret_cast<uint4*>(yp + c * 16);
            if (y32) {
              st_global_256(d, o[0], o[1]);
            } else {
              d[0] = o[0];
              d[1] = o[1];
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

template <int BN, typename TY>
cudaError_t launch_pair(const CUtensorMap& tmX, const CUtensorMap& tmW, const CUtensorMap& tmS,
                        const BlockGemmArgs& a, int num_sms, cudaStream_t stream) {
  auto kern = block_gemm_pair_kernel<BN, TY>;
  static std::atomic<unsigned long long> ready{0};  // one bit per device
  const cudaError_t e = smem_attribute_once(kern, PCfg<BN>::SMEM, ready);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((a.M - 1) / TILE_M + 1) * ((a.N - 1) / BN + 1);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(tiles, num_sms / 2) * 2));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = PCfg<BN>::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1 + overlap_attribute(&attr[1]);
  return cudaLaunchKernelEx(&cfg, kern, tmX, tmW, tmS, a);
}

}  // namespace

// The width whose fullest pair is done first, by a model whose weights (ns a
// group, ns a tile's end) are chosen so that it names the faster width at the
// ten shapes timed with both, M 128 to 4096, K 1024 to 20480; its times are
// within 25% of theirs.  256 and 128: 2048 x 1024 x 4096 takes 18.4 and 20.5
// us, 1024 x 8192 x 8192 71.7 and 67.6, 2048 x 20480 x 5120 229 and 188; 2048 x
// 12288 x 49152 takes 1030 either way.
int block_pair_width(int64_t M, int64_t N, int64_t K, int num_sms) {
  const int64_t pairs = std::max(1, num_sms / 2), num_m = (M + TILE_M - 1) / TILE_M, G = block_groups(K);
  const int64_t wide = (num_m * ((N + 255) / 256) + pairs - 1) / pairs * (505 * G + 4000);
  const int64_t narrow = (num_m * ((N + 127) / 128) + pairs - 1) / pairs * (240 * G + 2500);
  return wide <= narrow ? 256 : 128;
}

cudaError_t launch_block_gemm_pair(const CUtensorMap& tmX, const CUtensorMap& tmW, const CUtensorMap& tmS,
                                   const BlockGemmArgs& a, int width, int num_sms, cudaStream_t stream) {
#define PAIR(W)                                                                    \
  if (width == W)                                                                  \
    return a.bf16 ? launch_pair<W, __nv_bfloat16>(tmX, tmW, tmS, a, num_sms, stream)    \
                  : launch_pair<W, __half>(tmX, tmW, tmS, a, num_sms, stream)
  PAIR(256);
  PAIR(128);
#undef PAIR
  return cudaErrorInvalidValue;
}

}  // namespace i8mm
