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
//   warp 0      TMA producer
//   warp 1      allocates TMEM; in the leader one lane issues the MMAs of a
//               group (4 of 256 x BN x 32), alternating between two buffers
//   warps 4-11  two per TMEM lane quarter, one row per thread and half of the
//               tile's columns: they add P_g times sx sw to BN / 2 registers
//               and write Y at the tile's end, while the next tile's first
//               two groups already run
// A group takes the tensor cores 2 BN cycles (BN = 256: 512).  Reading 128 x
// 256 values from TMEM takes the eight warps 142 cycles, adding them 262 (two
// per packed instruction), both measured alone, so the sums fit beside the
// tensor cores; what bounds the kernel is the way of a buffer: its MMAs, the
// commit, the reads, the arrivals at the leader, the next issue.  A barrier
// poll takes 200 cycles and more while the MMAs read shared memory, so waits
// are polled ahead or two at a time, and the reads of the next 32 columns run
// under the multiply-adds of the last.
// Units of half a group (N = 128, four buffers) would have more slack, but
// read the X tile twice from shared memory: 1393 us for 2048 x 12288 x 49152.
//
// BN: the tile width is chosen from 256, 192 and 128 so that the tiles fill
// the pairs' rounds (block_pair_width).  A 192-wide tile does not start on a
// 128-column block of the weight scales, but its chunks of 32 columns never
// cross one: a half-tile meets at most two blocks.
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
// 168 each (384 x 168 = 64512), the first (producer, MMA issuer, two idle
// warps) goes down to 40 and the two epilogue groups up to 232
// (128 x 40 + 256 x 232 = 64512).
constexpr int THREADS = 128 + 32 * EPI_WARPS;
constexpr int REGS_LAUNCH = 168, REGS_FRONT = 40, REGS_EPI = 232;
static_assert(128 * REGS_FRONT + 32 * EPI_WARPS * REGS_EPI <= THREADS * REGS_LAUNCH, "registers within the launch's");

// TMEM: two buffers of 256 columns.
constexpr int SLOTS = 2, SLOT_COLS = 256;

// Scales of a CTA's rows come up to SX_CHUNK groups of one tile at a time, two
// chunks in turn.
constexpr int SX_CHUNK = 16;

template <int BN>
struct PCfg {
  static constexpr int A_BYTES = BM * kGroup;
  static constexpr int B_BYTES = BN / 2 * kGroup;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = 204800 / STAGE;
  static constexpr int HALF = BN / 2;  // columns per epilogue warp
  static constexpr int NBARS = 2 * STAGES + 2 * SLOTS + 1 + 4;
  static constexpr int SX_OFF = STAGES * STAGE;
  static constexpr int BAR_OFF = SX_OFF + 2 * SX_CHUNK * BM * 4;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
  static constexpr int SMEM = MISC_OFF + 16 + 1024;  // + slack to align the base to 1024
  static constexpr uint32_t IDESC = idesc_f16_f32(TILE_M, BN);  // e4m3 and fp16 operands share the encoding 0
  static_assert(HALF % 32 == 0 && BN <= SLOT_COLS && STAGE % 1024 == 0 && SMEM <= 232448, "tile shape");
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
// Untiled copy of `bytes` (a multiple of 16) to shared memory, counted on
// this CTA's barrier.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
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

// Waits for this thread's TMEM reads.  The registers they fill go through the
// statement, so that no use of them can move above it.
__device__ __forceinline__ void tmem_wait_cols(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

template <int BN, typename TY>
__global__ void __launch_bounds__(THREADS, 1)
    block_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                           const BlockGemmArgs a) {
  using C = PCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + SLOTS;
  uint64_t* drain = tempty + SLOTS;
  uint64_t* sfull = drain + 1;
  uint64_t* sempty = sfull + 2;
  float* sx_s = reinterpret_cast<float*>(smem + C::SX_OFF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int M = a.M, N = a.N;
  const uint32_t rank = cluster_ctarank();
  const int tile0 = static_cast<int>(blockIdx.x) / 2;
  const int tstride = static_cast<int>(gridDim.x) / 2;
  const int num_m = (M + TILE_M - 1) / TILE_M;
  const int num_tiles = num_m * ((N + BN - 1) / BN);
  const int G = (a.K + kGroup - 1) / kGroup;
  const int G2 = (G + 1) & ~1;  // groups are taken in pairs, one per TMEM buffer

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < SLOTS; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], EPI_WARPS * 2);
    }
    mbar_init(drain, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sempty[s], EPI_WARPS);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
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

  if (warp < 4) {
   asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_FRONT));
   if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------ TMA producer
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_phase = 0, chunk = 0;
      bool ok = true;
      const uint64_t pol_x = l2_policy_evict_last();  // every column tile of its rows reads X again
      for (int t = tile0; t < num_tiles && ok; t += tstride) {
        const int m0 = (t % num_m) * TILE_M + static_cast<int>(rank) * BM;
        const int n0 = (t / num_m) * BN + static_cast<int>(rank) * (BN / 2);
        // rows of scales: up to lds, a multiple of 4 (16 bytes)
        const uint32_t sx_bytes = static_cast<uint32_t>(max(0, min(BM, (M - m0 + 3) & ~3))) * 4u;
        for (int g = 0; g < G; ++g) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, tmo, abort_flag) ||
              (g % SX_CHUNK == 0 && !mbar_wait(&sempty[chunk & 1u], ((chunk >> 1) & 1u) ^ 1u, tmo, abort_flag))) {
            ok = false;
            break;
          }
          // both CTAs' loads complete on the leader's barrier; the leader
          // announces the pair's bytes
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * C::STAGE);
          const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
          uint8_t* st = smem + stage * C::STAGE;
          tma_load_2d_pair_hint(st, &tmX, bar, g * kGroup, m0, pol_x);
          tma_load_2d_pair(st + C::A_BYTES, &tmW, bar, 0, g * a.N_pad + n0);
          if (g % SX_CHUNK == 0) {
            uint64_t* sb = &sfull[chunk & 1u];
            float* dst = sx_s + (chunk & 1u) * (SX_CHUNK * BM);
            const int n = min(SX_CHUNK, G - g);
            if (sx_bytes != 0u) {
              mbar_arrive_expect_tx(sb, sx_bytes * static_cast<uint32_t>(n));
              for (int j = 0; j < n; ++j)
                bulk_load(dst + j * BM, a.sx + static_cast<size_t>(g + j) * a.lds + m0, sx_bytes, sb);
            } else {
              mbar_arrive(sb);
            }
            ++chunk;
          }
          issued_mask |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        gfail(a, abort_flag);
        for (uint32_t j = chunk > 2 ? chunk - 2 : 0; j < chunk; ++j)
          mbar_wait(&sfull[j & 1u], (j >> 1) & 1u, tmo, nullptr);
        // every load already issued lands before the CTA can exit (the peer
        // cannot watch the leader's barriers: it waits a while)
        if (rank == 0) {
          for (int s = 0; s < C::STAGES; ++s)
            if (issued_mask & (1u << s)) mbar_wait(&full[s], (issued_phase >> s) & 1u, tmo, nullptr);
        } else {
          const uint64_t t0 = global_timer_ns();
          while (global_timer_ns() - t0 < 200000ull) {
          }
        }
      }
    }
   } else if (warp == 1) {
    if (rank == 0) {
      // -------------------------------------------------------- MMA issuer
      // The whole warp walks the loop and one elected lane issues: the
      // descriptors then stay in uniform registers.
      const uint32_t issuer = elect_one();
      const uint32_t desc_hi = static_cast<uint32_t>(smem_desc_k_sw128(0) >> 32);
      const uint32_t desc_lo = static_cast<uint32_t>(smem_desc_k_sw128(smem_u32(smem)));
      int stage = 0;
      uint32_t phase = 0, it = 0;
      bool ok = true;
      for (int t = tile0; t < num_tiles && ok; t += tstride) {
        for (int g = 0; g < G2 && ok; ++g, ++it) {
          const uint32_t buf = it & 1u;
          if (g == G) {  // an odd tile's last group is empty: no MMAs, only the commit
            ok = mbar_wait2_warp(&tempty[buf], ((it >> 1) & 1u) ^ 1u, &tempty[buf], ((it >> 1) & 1u) ^ 1u, tmo,
                                 abort_flag);
            if (ok && issuer) mma_commit_pair(&tfull[buf], 0x3);
            __syncwarp();
            continue;
          }
          ok = mbar_wait2_warp(&full[stage], phase, &tempty[buf], ((it >> 1) & 1u) ^ 1u, tmo, abort_flag);
          if (ok) {
            tc_fence_after();
            if (issuer) {
              const uint32_t ad = desc_lo + static_cast<uint32_t>(stage * (C::STAGE >> 4));
              const uint32_t bd = ad + (C::A_BYTES >> 4);
              const uint32_t d = tmem_base + buf * SLOT_COLS;
#pragma unroll
              for (int kk = 0; kk < kGroup / 32; ++kk)  // 32 bytes along K inside the 128-byte swizzled row
                mma_e4m3_pair(d, make_desc(ad + kk * 2, desc_hi), make_desc(bd + kk * 2, desc_hi), C::IDESC, kk != 0);
              mma_commit_pair(&tfull[buf], 0x3);
              mma_commit_pair(&empty[stage], 0x3);  // frees the stage in both CTAs
            }
            __syncwarp();
          }
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && issuer) {
        gfail(a, abort_flag);
        mma_commit_pair(drain, 0x1);
        mbar_wait(drain, 0, tmo, nullptr);
      }
    }
   }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPI));
    // ----------------------------------------------------- sums and epilogue
    const int q = warp & 3;             // TMEM lane quarter this warp may read
    const int h = (warp - 4) >> 2;      // half of the tile's columns
    const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(h * C::HALF);
    const uint32_t tempty0 = mapa_shared(smem_u32(&tempty[0]), 0);
    constexpr int CH = C::HALF / 32;
    const int NB = (N + kGroup - 1) / kGroup;
    uint32_t chunk = 0, ph = 0;
    bool alive = true;
    const uint32_t tfull0 = smem_u32(&tfull[0]);
    const uint32_t sx0 = smem_u32(sx_s) + static_cast<uint32_t>(q * 32 + lane) * 4u;
    for (int t = tile0; t < num_tiles && alive; t += tstride) {
      const int m = (t % num_m) * TILE_M + static_cast<int>(rank) * BM + q * 32 + lane;
      const int nh = (t / num_m) * BN + h * C::HALF;
      const bool row_ok = m < M;
      // the weight scales of the one or two blocks that the half-tile meets
      // (past N: any block's, the sums are dropped), one group per lane, a
      // chunk ahead
      const int b0 = min(nh / kGroup, NB - 1), b1 = min((nh + C::HALF - 1) / kGroup, NB - 1);
      const float* sw0 = a.sw + static_cast<size_t>(b0) * G;
      const float* sw1 = a.sw + static_cast<size_t>(b1) * G;
      auto weight_scale = [&](const float* p, int g) { return __ldg(p + min(g + lane, G - 1)); };
      float w0n = weight_scale(sw0, 0), w1n = BN % 256 != 0 ? weight_scale(sw1, 0) : 0.0f;
      const int cross = (b0 + 1) * kGroup - nh;  // first column of the second block
      uint64_t acc[C::HALF / 2];
#pragma unroll
      for (int i = 0; i < C::HALF / 2; ++i) acc[i] = 0ull;
      // columns [32 c, 32 c + 32) of the warp's half-tile += r times the scale
      auto add = [&](const uint32_t (&r)[32], int c, uint64_t s0, uint64_t s1) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          fma2(acc[c * 16 + i], r[2 * i], r[2 * i + 1], (BN % 256 != 0 && c * 32 >= cross) ? s1 : s0);
      };
      // (the row's scales come through shared memory: with the next ones on
      // their way from global memory, tcgen05.wait::ld waited for them too)
      bool ready = false;  // the next group was complete when polled during the last one
#pragma unroll 1
      for (int g0 = 0; g0 < G && alive; g0 += SX_CHUNK, ++chunk) {
        const float w0 = w0n, w1 = w1n;
        w0n = weight_scale(sw0, g0 + SX_CHUNK);
        if constexpr (BN % 256 != 0) w1n = weight_scale(sw1, g0 + SX_CHUNK);
        alive = __all_sync(0xffffffffu, mbar_wait(&sfull[chunk & 1u], (chunk >> 1) & 1u, tmo, abort_flag));
        uint32_t sx = sx0 + (chunk & 1u) * (SX_CHUNK * BM * 4);
        const int n = min(SX_CHUNK, G - g0);
#pragma unroll 1
        for (int j = 0; j < n && alive; j += 2, sx += 2 * BM * 4, ph ^= 1u) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (!__all_sync(0xffffffffu, ready))
              alive = alive && mbar_wait2_warp(&tfull[u], ph, &tfull[u], ph, tmo, abort_flag);
            tc_fence_after();
            if (u == 0 || j + 1 < n) {
              const uint32_t t = t_row + u * SLOT_COLS;
              uint32_t ra[32], rb[32];
              tmem_ld_32x32b_x32(t, ra);
              const float x = lds_f32(sx + u * (BM * 4));
              const uint64_t s0 = twice(__fmul_rn(x, __shfl_sync(0xffffffffu, w0, j + u)));
              const uint64_t s1 = BN % 256 != 0 ? twice(__fmul_rn(x, __shfl_sync(0xffffffffu, w1, j + u))) : s0;
#pragma unroll
              for (int c = 0; c < CH; ++c) {
                uint32_t(&r)[32] = (c & 1) ? rb : ra;
                uint32_t(&nx)[32] = (c & 1) ? ra : rb;
                tmem_wait_cols(r);
                if (c + 1 < CH) {
                  tmem_ld_32x32b_x32(t + static_cast<uint32_t>((c + 1) * 32), nx);
                } else {  // the buffer is read: hand it back to the leader
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) mbar_arrive_cluster_relaxed(tempty0 + u * 8u);
                }
                if (c == CH - 2) ready = mbar_test_wait(tfull0 + (u ^ 1) * 8u, u == 0 ? ph : ph ^ 1u);
                add(r, c, s0, s1);
              }
            } else {  // the empty group of an odd tile
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster_relaxed(tempty0 + u * 8u);
              ready = false;
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[chunk & 1u]);
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
cudaError_t launch_pair(const CUtensorMap& tmX, const CUtensorMap& tmW, const BlockGemmArgs& a, int num_sms,
                        cudaStream_t stream) {
  auto kern = block_gemm_pair_kernel<BN, TY>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PCfg<BN>::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((a.M + TILE_M - 1) / TILE_M) * ((a.N + BN - 1) / BN);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(tiles, num_sms / 2) * 2));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = PCfg<BN>::SMEM;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tmX, tmW, a);
}

}  // namespace

// Time of the fullest pair in columns of 256 rows: rounds of tiles x (width
// + a fixed cost per tile).
int block_pair_width(int64_t M, int64_t N, int num_sms) {
  const int64_t pairs = std::max(1, num_sms / 2), num_m = (M + TILE_M - 1) / TILE_M;
  int best = 0;
  int64_t best_cost = 0;
  for (int w : kPairWidths) {
    const int64_t rounds = (num_m * ((N + w - 1) / w) + pairs - 1) / pairs;
    const int64_t cost = rounds * (w + 8);
    if (best == 0 || cost < best_cost) {
      best = w;
      best_cost = cost;
    }
  }
  return best;
}

cudaError_t launch_block_gemm_pair(const CUtensorMap& tmX, const CUtensorMap& tmW, const BlockGemmArgs& a, int width,
                                   int num_sms, cudaStream_t stream) {
#define PAIR(W)                                                                    \
  if (width == W)                                                                  \
    return a.bf16 ? launch_pair<W, __nv_bfloat16>(tmX, tmW, a, num_sms, stream)    \
                  : launch_pair<W, __half>(tmX, tmW, a, num_sms, stream)
  PAIR(256);
  PAIR(192);
  PAIR(128);
#undef PAIR
  return cudaErrorInvalidValue;
}

}  // namespace i8mm
