// Matrix product of e4m3 codes with block scales for few rows (tokens), sm_100a:
//
//   Y[m, n] = sum_g sx[g][m] sw[n / 128][g] P_g[m, n]  (+ bias[n])
//   P_g[m, n] = sum_{k in g} X[m, k] W[n, k]
//
// Bound by reading W once.  The operands are swapped: 128 rows of W (columns n
// of Y) take the MMA's M slot and the MP padded tokens its N slot; P_g comes
// from the tensor cores (tcgen05.mma kind::f8f6f4) and is added to fp32
// registers with its factor, as in the kernel for many rows.
//
// Work split: a cluster of S CTAs takes a run of W's rows, in 16s, so that all
// clusters' runs are equal within 16 rows; its CTAs take equal parts of the
// groups of K.  Each tile's S partial sums meet in shared memory of the
// cluster: CTA r finishes the tokens [r MP / S, (r + 1) MP / S), adding the S
// parts in the order of the ranks; the parts travel as one bulk copy per pair
// of CTAs (stored value by value from the registers into the peers' memory,
// 32 tokens at K = N = 8192 took 36.9 us, 14 more than one token).  No
// workspace, no atomics, and the same result every time.  Splitting N alone
// would leave SMs idle at small N and the last round part-filled; splitting K
// alone would need the sum in memory.
//   warp 0      TMA producer (W marked evict-first in L2), GS groups per stage
//   warp 1      TMEM, MMA issuer
//   warps 4..   sums: one row n per thread; with 64 or more tokens two warps
//               share a TMEM lane quarter, half of the tokens each
// Two groups per stage: a step's waits take each of these
// warps some 500 cycles, a group's 16 KB of W some 700 at the SM's share of
// the HBM rate.
//
// Measured in a captured chain, weights in turn: 1 x 12288 x 49152 95.0 us, 97%
// of the measured copy rate (one weight again and again 92.4, of which a part
// is still in L2; back to back over three weights 92 to 98 on several
// machines), 32 x 8192 x 8192 16.8 us, of which the stream of W is 10.4.
//
// Every wait is bounded; a timeout sets the status word, and the CTA drains
// and exits with its cluster.
#include "block8.cuh"
#include "block8_gemm.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

#include <algorithm>

namespace i8mm {
namespace {

constexpr int RM = 128;  // rows of W per tile
constexpr int R_CHUNK = kSxChunk;

template <int MP>
struct RCfg {
  static constexpr int GS = 2;                 // groups per stage
  static constexpr int NH = MP >= 64 ? 2 : 1;  // token halves
  static constexpr int TH = MP / NH;           // tokens per thread
  static constexpr int EPI = 4 * NH;           // epilogue warps
  static constexpr int THREADS = 128 + 32 * EPI;
  static constexpr int W_BYTES = RM * kGroup, X_BYTES = MP * kGroup;
  static constexpr int STAGE = GS * (W_BYTES + X_BYTES);
  static constexpr int STAGES = MP <= 16 ? 5 : (MP <= 32 ? 4 : 3);
  static constexpr int SX_OFF = STAGES * STAGE;             // [2][R_CHUNK][MP] scales
  static constexpr int OUT_OFF = SX_OFF + 2 * R_CHUNK * MP * 4;  // [MP][RM] this CTA's partial sums
  static constexpr int RED_OFF = OUT_OFF + MP * RM * 4;          // [S][MP / S][RM] the others' of my tokens
  static constexpr int BAR_OFF = RED_OFF + MP * RM * 4;
  static constexpr int NBARS = 2 * STAGES + 4 + 4 + 2 + 1;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
  static constexpr int SMEM = MISC_OFF + 16 + 1024;
  static constexpr int TMEM_COLS = 2 * GS * MP < 32 ? 32 : 2 * GS * MP;
  static constexpr uint32_t IDESC = idesc_f16_f32(RM, MP);  // e4m3 and fp16 operands share the encoding 0
  static_assert(STAGE % 1024 == 0 && X_BYTES % 1024 == 0 && SMEM <= 232448, "shared memory");
  static_assert((TMEM_COLS & (TMEM_COLS - 1)) == 0 && TMEM_COLS <= 512, "TMEM allocation");
};

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ uint32_t relect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_nctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_id_x() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_count_x() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%nclusterid.x;" : "=r"(r));
  return r;
}
// Copy of `bytes` (a multiple of 16) from this CTA's shared memory to a
// cluster address, counted on the barrier there.
__device__ __forceinline__ void bulk_to_cluster(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "r"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void epi_sync(int threads) { asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory"); }

// mbar_wait for a phase that other CTAs of the cluster complete, with their
// writes to this CTA's shared memory visible after it.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, uint64_t timeout_ns,
                                                  volatile int* abort) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((it & 15) == 0) {
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (*abort || now - t0 > timeout_ns) return false;
    }
  }
}

__device__ __forceinline__ void rfail(const BlockGemmArgs& a, volatile int* abort_flag) {
  *abort_flag = 1;
  atomicOr(a.status, kStatusTimeout);
}

// N columns of this thread's TMEM lane.
template <int N>
__device__ __forceinline__ void rows_ld(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 16) {
    tmem_ld_32x32b_x16(taddr, r);
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 32) tmem_ld_32x32b_x32(taddr + c, *reinterpret_cast<uint32_t(*)[32]>(&r[c]));
  }
}
// Waits for them; the registers go through it, so that no use moves above it.
template <int N>
__device__ __forceinline__ void rows_wait(uint32_t (&r)[N]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; i += 16)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                 "+r"(r[i + 6]), "+r"(r[i + 7]), "+r"(r[i + 8]), "+r"(r[i + 9]), "+r"(r[i + 10]), "+r"(r[i + 11]),
                 "+r"(r[i + 12]), "+r"(r[i + 13]), "+r"(r[i + 14]), "+r"(r[i + 15])::"memory");
}

// tmW: the weight's rows of 128 bytes with 128-row boxes; tmWl with boxes of
// a.last_rows, the rows of the longest run's last tile (a shorter run's last
// tile reads 16 rows too many, and drops them); tmX: the codes [M, K] with
// MP-row boxes; tmS: the scales [G][M] with 16 x MP boxes.
template <int MP, typename TY>
__global__ void __launch_bounds__(RCfg<MP>::THREADS, 1)
    block_gemm_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmWl,
                           const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmS,
                           const BlockGemmArgs a) {
  using C = RCfg<MP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* sx_s = reinterpret_cast<float*>(smem + C::SX_OFF);
  float* out_s = reinterpret_cast<float*>(smem + C::OUT_OFF);
  float* red_s = reinterpret_cast<float*>(smem + C::RED_OFF);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;  // [2]
  uint64_t* tempty = tfull + 2;         // [2]
  uint64_t* sfull = tempty + 2;         // [2]
  uint64_t* sempty = sfull + 2;         // [2]
  uint64_t* rfull = sempty + 2;         // every CTA of the cluster has sent its part of my tokens
  uint64_t* rempty = rfull + 1;         // the other CTAs have read my parts
  uint64_t* drain = rempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int S = static_cast<int>(cluster_nctas()), rank = static_cast<int>(cluster_ctarank());
  const int G = (a.K + kGroup - 1) / kGroup;
  const int g_begin = G * rank / S, g_end = G * (rank + 1) / S;
  const int steps = (g_end - g_begin + C::GS - 1) / C::GS;
  const long long units = a.N / 16, nclus = cluster_count_x(), clus = cluster_id_x();
  const int row_begin = static_cast<int>(units * clus / nclus) * 16;
  const int row_end = static_cast<int>(units * (clus + 1) / nclus) * 16;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], C::EPI);
      mbar_init(&sfull[b], 1);
      mbar_init(&sempty[b], C::EPI);
    }
    mbar_init(rfull, static_cast<uint32_t>(S));
    mbar_init(rempty, static_cast<uint32_t>(max(1, (S - 1) * C::EPI)));
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmS);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  cluster_sync_all();  // the peers' barriers are initialised before any remote arrive
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const unsigned long long tmo = a.timeout_ns;
  if (warp == 0 && relect_one()) {
    // The first tiles of W into L2 while the stream's previous kernel ends: a
    // hint that needs no order with it.  In a captured chain 16 x 8192 x 8192
    // (four weights in turn) 16.7 -> 15.2 us, 1 x 12288 x 49152 (one weight)
    // 94.8 -> 92.
    const uint32_t bytes = static_cast<uint32_t>(min(RM, row_end - row_begin) * kGroup);
    for (int g = g_begin; g < min(g_end, g_begin + C::STAGES * C::GS); ++g)
      bulk_prefetch_l2(a.Wb + (static_cast<size_t>(g) * a.N_pad + row_begin) * kGroup, bytes);
  }
  __syncwarp();
  dependency_wait();

  if (warp == 0) {
    // ---------------------------------------------------------- TMA producer
    const uint32_t issuer = relect_one();
    const uint64_t pol_w = l2_policy_evict_first();  // W is read once
    int stage = 0;
    uint32_t phase = 1, chunk = 0;
    bool ok = true;
    for (int r0 = row_begin; r0 < row_end && ok; r0 += RM) {
      const bool last = r0 - row_begin >= (a.tiles - 1) * RM;
      const int rows = last ? a.last_rows : RM;
      for (int s = 0; s < steps && ok; ++s) {
        const int g = g_begin + s * C::GS, n = min(C::GS, g_end - g);
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], phase, tmo, abort_flag));
        if (ok && s % (R_CHUNK / C::GS) == 0) {
          // the scales of the next 16 groups, one box
          ok = __all_sync(0xffffffffu, mbar_wait(&sempty[chunk & 1u], ((chunk >> 1) & 1u) ^ 1u, tmo, abort_flag));
          if (ok && issuer) {
            mbar_arrive_expect_tx(&sfull[chunk & 1u], R_CHUNK * MP * 4);
            tma_load_2d(sx_s + (chunk & 1u) * (R_CHUNK * MP), &tmS, &sfull[chunk & 1u], 0, g);
          }
          ++chunk;
        }
        if (ok && issuer) {
          uint8_t* st = smem + stage * C::STAGE;
          mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(n * (rows * kGroup + C::X_BYTES)));
          for (int u = 0; u < n; ++u) {
            uint8_t* w = st + u * C::W_BYTES;
            const int wr = (g + u) * a.N_pad + r0;
            tma_load_2d_hint(w, last ? &tmWl : &tmW, &full[stage], 0, wr, pol_w);
            tma_load_2d(st + C::GS * C::W_BYTES + u * C::X_BYTES, &tmX, &full[stage], (g + u) * kGroup, 0);
          }
        }
        __syncwarp();
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {
      // the loads already issued land, microseconds later, before the CTA exits
      if (issuer) rfail(a, abort_flag);
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 200000ull) {
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t issuer = relect_one();
    const uint32_t desc_hi = static_cast<uint32_t>(smem_desc_k_sw128(0) >> 32);
    const uint32_t desc_lo = static_cast<uint32_t>(smem_desc_k_sw128(smem_u32(smem)));
    int stage = 0;
    uint32_t phase = 0, it = 0;
    bool ok = true;
    for (int r0 = row_begin; r0 < row_end && ok; r0 += RM) {
      for (int s = 0; s < steps && ok; ++s, ++it) {
        const int n = min(C::GS, g_end - g_begin - s * C::GS);
        const uint32_t buf = it & 1u;
        ok = mbar_wait2_warp(&full[stage], phase, &tempty[buf], ((it >> 1) & 1u) ^ 1u, tmo, abort_flag);
        if (ok) {
          tc_fence_after();
          if (issuer) {
            const uint32_t sd = desc_lo + static_cast<uint32_t>(stage * (C::STAGE >> 4));
#pragma unroll
            for (int u = 0; u < C::GS; ++u) {
              if (u < n) {
                const uint32_t ad = sd + u * (C::W_BYTES >> 4);
                const uint32_t bd = sd + ((C::GS * C::W_BYTES + u * C::X_BYTES) >> 4);
                const uint32_t d = tmem_base + (buf * C::GS + u) * MP;
#pragma unroll
                for (int kk = 0; kk < kGroup / 32; ++kk)  // 32 bytes along K inside the 128-byte swizzled row
                  mma_e4m3(d, (static_cast<uint64_t>(desc_hi) << 32) | (ad + kk * 2),
                           (static_cast<uint64_t>(desc_hi) << 32) | (bd + kk * 2), C::IDESC, kk != 0);
              }
            }
            mma_commit(&tfull[buf]);
            mma_commit(&empty[stage]);
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
      rfail(a, abort_flag);
      mma_commit(drain);
      mbar_wait(drain, 0, tmo, nullptr);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------ sums and epilogue
    const int q = warp & 3, h = (warp - 4) >> 2;
    const int row = q * 32 + lane;  // of the tile
    const int m0 = h * C::TH;       // first token
    const int M = a.M, N = a.N;
    const int NB = (N + kGroup - 1) / kGroup;
    const int TS = MP / S;          // tokens that a CTA finishes
    const int mine = max(0, min(TS, M - rank * TS));
    const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(m0);
    uint32_t it = 0, chunk = 0, tile = 0;
    bool alive = true;
    // after a timeout a warp still takes part in the named barriers
    for (int r0 = row_begin; r0 < row_end; r0 += RM, ++tile) {
      const int n = r0 + row;
      const bool n_ok = n < row_end;
      // scales of the one or two blocks that the tile's rows meet, 16 groups
      // at a time: lanes 0-15 the first block's, 16-31 the second's
      const int b0 = r0 / kGroup, b1 = min(b0 + 1, NB - 1);
      const float* swp = a.sw + static_cast<size_t>(lane < 16 ? b0 : b1) * G;
      const int sel = (n / kGroup != b0) ? 16 : 0;
      auto weight_scale = [&](int g) { return __ldg(swp + min(g + (lane & 15), G - 1)); };
      float wn = weight_scale(g_begin);
      float acc[C::TH];
#pragma unroll
      for (int t = 0; t < C::TH; ++t) acc[t] = 0.0f;
#pragma unroll 1
      for (int g0 = g_begin; g0 < g_end && alive; g0 += R_CHUNK, ++chunk) {
        const float w = wn;
        wn = weight_scale(g0 + R_CHUNK);
        alive = __all_sync(0xffffffffu, mbar_wait(&sfull[chunk & 1u], (chunk >> 1) & 1u, tmo, abort_flag));
        const float* sx = sx_s + (chunk & 1u) * (R_CHUNK * MP) + m0;
        const int ng = min(R_CHUNK, g_end - g0);
#pragma unroll 1
        for (int j = 0; j < ng && alive; j += C::GS, ++it) {
          const uint32_t buf = it & 1u;
          alive = mbar_wait2_warp(&tfull[buf], (it >> 1) & 1u, &tfull[buf], (it >> 1) & 1u, tmo, abort_flag);
          if (!alive) break;
          tc_fence_after();
#pragma unroll
          for (int u = 0; u < C::GS; ++u) {
            uint32_t r[C::TH];
            rows_ld<C::TH>(t_row + (buf * C::GS + u) * MP, r);  // of no use past ng, and not used
            const float ws = __shfl_sync(0xffffffffu, w, sel + ((j + u) & 15));
            rows_wait<C::TH>(r);
            if (u == C::GS - 1) {  // the buffer is read: hand it back
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&tempty[buf]);
            }
            if (j + u < ng) {
              const float4* s4 = reinterpret_cast<const float4*>(sx + (j + u) * MP);
#pragma unroll
              for (int t = 0; t < C::TH; t += 4) {
                const float4 s = s4[t / 4];
                acc[t + 0] = __fmaf_rn(__uint_as_float(r[t + 0]), __fmul_rn(s.x, ws), acc[t + 0]);
                acc[t + 1] = __fmaf_rn(__uint_as_float(r[t + 1]), __fmul_rn(s.y, ws), acc[t + 1]);
                acc[t + 2] = __fmaf_rn(__uint_as_float(r[t + 2]), __fmul_rn(s.z, ws), acc[t + 2]);
                acc[t + 3] = __fmaf_rn(__uint_as_float(r[t + 3]), __fmul_rn(s.w, ws), acc[t + 3]);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0 && !(a.skip_scales && warp == 4 && rank == 0)) mbar_arrive(&sempty[chunk & 1u]);
      }
      const float bias = (n_ok && a.bias != nullptr) ? static_cast<float>(static_cast<const TY*>(a.bias)[n]) : 0.0f;
      TY* y = static_cast<TY*>(a.Y) + n;
      if (S == 1) {
        if (alive && n_ok) {
#pragma unroll
          for (int t = 0; t < C::TH; ++t)
            if (m0 + t < M) y[static_cast<size_t>(m0 + t) * N] = TY(__fadd_rn(acc[t], bias));
        }
      } else {
        // the tile's parts meet.  The last tile's have been read everywhere:
        // by the other CTAs (which then also have my copies), and by this one.
        if (tile > 0 && alive)
          alive = __all_sync(0xffffffffu, mbar_wait_cluster(rempty, (tile - 1) & 1u, tmo, abort_flag));
        epi_sync(C::EPI * 32);
#pragma unroll
        for (int t = 0; t < C::TH; ++t)
          if (m0 + t < M) out_s[(m0 + t) * RM + row] = acc[t];
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        epi_sync(C::EPI * 32);
        if (warp == 4 && lane == 0 && alive && *abort_flag == 0) {
          if (mine > 0) mbar_arrive_expect_tx(rfull, static_cast<uint32_t>((S - 1) * mine * RM * 4));
          else mbar_arrive(rfull);
          for (int c = 0; c < S; ++c) {
            if (c == rank) continue;
            const uint32_t bar = mapa_shared(smem_u32(rfull), static_cast<uint32_t>(c));
            const int theirs = min(TS, M - c * TS);
            if (theirs > 0)
              bulk_to_cluster(mapa_shared(smem_u32(red_s + rank * TS * RM), static_cast<uint32_t>(c)),
                              smem_u32(out_s + c * TS * RM), static_cast<uint32_t>(theirs * RM * 4), bar);
            // also where no token is theirs: a CTA that waited for nobody could
            // finish a tile before this one has noticed the end of the last,
            // and rempty would pass two phases unseen
            if (!(a.skip_meeting && rank == 0)) mbar_arrive_cluster(bar);
          }
        }
        if (alive) alive = __all_sync(0xffffffffu, mbar_wait_cluster(rfull, tile & 1u, tmo, abort_flag));
        if (alive) {
          // eight tokens at a time: their loads from shared memory, slow while
          // the next tile's MMAs read it, overlap
          constexpr int U = C::TH < 8 ? C::TH : 8;
          for (int k0 = h; k0 < mine; k0 += C::NH * U) {
            float v[U];
#pragma unroll
            for (int i = 0; i < U; ++i) v[i] = 0.0f;
            for (int c = 0; c < S; ++c) {
              const float* part = (c == rank ? out_s + rank * TS * RM : red_s + c * TS * RM) + row;
#pragma unroll
              for (int i = 0; i < U; ++i) {
                const int k = k0 + i * C::NH;
                if (k < mine) v[i] = __fadd_rn(v[i], part[k * RM]);
              }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
              const int k = k0 + i * C::NH;
              if (n_ok && k < mine) y[static_cast<size_t>(rank * TS + k) * N] = TY(__fadd_rn(v[i], bias));
            }
          }
          __syncwarp();
          if (lane == 0)
            for (int c = 0; c < S; ++c)
              if (c != rank) mbar_arrive_cluster(mapa_shared(smem_u32(rempty), static_cast<uint32_t>(c)));
        }
      }
      if (!alive && lane == 0) rfail(a, abort_flag);
    }
    if (!alive) {  // copies already issued land before the cluster exits
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 200000ull) {
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its peers may still write to it or signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <int MP, typename TY>
cudaError_t configure_rows(int S, cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr) {
  auto kern = block_gemm_rows_kernel<MP, TY>;
  static std::atomic<unsigned long long> ready{0};  // one bit per device
  const cudaError_t e = smem_attribute_once(kern, RCfg<MP>::SMEM, ready);
  if (e != cudaSuccess) return e;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = static_cast<unsigned>(S);
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(S));
  cfg.blockDim = dim3(RCfg<MP>::THREADS);
  cfg.dynamicSmemBytes = RCfg<MP>::SMEM;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaSuccess;
}

template <int MP, typename TY>
cudaError_t launch_rows(const CUtensorMap& tmW, const CUtensorMap& tmWl, const CUtensorMap& tmX,
                        const CUtensorMap& tmS, const BlockGemmArgs& a, const RowsPlan& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  const cudaError_t e = configure_rows<MP, TY>(p.split, cfg, attr);
  if (e != cudaSuccess) return e;
  cfg.numAttrs += overlap_attribute(&attr[cfg.numAttrs]);
  cfg.gridDim = dim3(static_cast<unsigned>(p.split * p.clusters));
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, block_gemm_rows_kernel<MP, TY>, tmW, tmWl, tmX, tmS, a);
}

}  // namespace

int rows_padded_tokens(int64_t M) { return M <= 16 ? 16 : (M <= 32 ? 32 : 64); }

// Clusters of S CTAs that fit the device at once, one CTA per SM.
cudaError_t rows_max_clusters(int S, int* clusters) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  cudaError_t e = configure_rows<64, __half>(S, cfg, &attr);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(clusters, block_gemm_rows_kernel<64, __half>, &cfg);
  return e;
}

// Split of K and number of clusters for M tokens: the least time of the
// fullest CTA, in rows x groups (2.8 ns each at an SM's share of the HBM
// rate).  A tile of fewer than 48 rows takes the time of 48.  The meeting of a
// tile's sums takes MEET, and where another tile follows, whose MMAs then wait
// for it, MEET_M per token more.  The constants were fitted before the first
// tiles were prefetched; the choice still holds where splits of 1, 2 and 4 were
// timed after it (captured, us): N = K = 8192 16 tokens 16.2, 13.7, 20.3, 32
// tokens 19.6, 16.3, 21.7, 64 tokens 22.1, 18.0, 23.7; K = 5120, N = 20480, 32
// tokens 27.2, 34.2, 42.9; K = 12288, N = 49152 (unsplit three tiles) 1 token
// 92.5, 105, 127, 32 tokens 93.1, 118, 145.
RowsPlan rows_plan(int64_t M, int64_t N, int64_t K, const int (&max_clusters)[4]) {
  constexpr int64_t MEET = 700, MEET_M = 40, UNSPLIT = 200;
  const int64_t units = N / 16, G = block_groups(K);
  RowsPlan best{1, 1, 1, 16};
  int64_t best_cost = -1;
  for (int i = 0; i < 4; ++i) {
    const int S = 1 << i;
    if (S > G || max_clusters[i] < 1) continue;
    const int64_t c = std::min<int64_t>(units, max_clusters[i]);
    const int64_t rows = (units + c - 1) / c * 16, groups = (G + S - 1) / S;
    const int64_t tiles = (rows + RM - 1) / RM, last = rows - (tiles - 1) * RM;
    const int64_t cost = ((tiles - 1) * RM + std::max<int64_t>(last, 48)) * groups +
                         (S > 1 ? tiles * MEET + (tiles - 1) * MEET_M * M : tiles * UNSPLIT);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = RowsPlan{S, static_cast<int>(c), static_cast<int>(tiles), static_cast<int>(last)};
    }
  }
  return best;
}

cudaError_t launch_block_gemm_rows(const CUtensorMap& tmW, const CUtensorMap& tmWl, const CUtensorMap& tmX,
                                   const CUtensorMap& tmS, const BlockGemmArgs& a, const RowsPlan& p,
                                   cudaStream_t stream) {
#define ROWS(MP)                                                                              \
  case MP:                                                                                    \
    return a.bf16 ? launch_rows<MP, __nv_bfloat16>(tmW, tmWl, tmX, tmS, a, p, stream)        \
                  : launch_rows<MP, __half>(tmW, tmWl, tmX, tmS, a, p, stream)
  switch (rows_padded_tokens(a.M)) {
    ROWS(16);
    ROWS(32);
    ROWS(64);
  }
#undef ROWS
  return cudaErrorInvalidValue;
}

}  // namespace i8mm
