// gemm_m64_w8.cuh -- the few-row GEMM (gemm_m64.cuh) over e4m3 weights read as
// they are stored, for mla_tree_decode on sm_100a.
//
// mla_decode first writes a bf16 copy of W_kvb and W_o: the 134 MB of codes of
// 128 heads are read, 268 MB written and read again, 89 us before the products
// begin. Here each CTA's share of the codes goes from HBM to shared memory by
// TMA and sixteen warps turn it into the bf16 operand there, so that a weight
// costs one byte of HBM traffic. W_o of 128 heads and 128 rows: 48 us, shared
// memory busy for three quarters of it (codes and A written by TMA, codes read,
// the operand written, both operands read by the tensor core: 80 KB for 8 KB of
// codes). Tiles of 256 columns halve A's part, but leave two buffers of operand
// for four: 1.5 us slower at 128 rows, 3.5 faster at 256.
// Scales (one per 128 x 128 block):
//   absorb  (q_nope . W_UK, K = 128): one scale per output tile, applied to the
//           fp32 accumulator; the codes are exact in bf16
//   unabsorb (o_lat . W_UV^T, K = 512): one scale per 128 of K, which the
//           attention has multiplied into o_lat before rounding it
//   W_o     (stream-K): bf16(code * scale), rounded once, as the copy would be
//
// Roles (736 threads, one CTA per SM): warp 0 asks for codes, warp 22 for A; warp
// 1 tensor memory and UMMA issuer; warps 2..5 epilogue; warps 6..21 converters,
// four teams that take tiles in turn. Codes ([64 x 128], 8 KB), A ([BM x 64]) and
// converted operands (16 KB) have rings of their own: with a common stage, five
// to seven of which fit, only 40 to 56 KB of codes were in flight per SM, and W_o's
// 117 MB took 53 us. Work (segments, stream-K shares, batches) as in
// gemm_m64.cuh.
#pragma once

#include <cuda_fp8.h>

#include "gemm_m64.cuh"

namespace mla {

// B_MN_MAJOR_: weights stored [K, N]; else [N, K]. BATCH_: one product per head
// with bf16 C; else stream-K with fp32 partial tiles and scaled conversion.
template <int BM_, bool B_MN_MAJOR_, bool BATCH_>
struct GemmM64W8Cfg {
  static constexpr int BM = BM_, BN = 128, BK = 64;
  static constexpr bool B_MN_MAJOR = B_MN_MAJOR_, BATCH = BATCH_;
  static constexpr int A_STAGES = BM_ == 64 ? 6 : 5, W_STAGES = BM_ == 64 ? 14 : 10, BUFS = 4;
  static constexpr int A_BYTES = BM * BK * 2, W_BYTES = BK * BN, BUF_BYTES = BK * BN * 2;
  static constexpr int CONVERTERS = 16, TEAMS = 4, TEAM = CONVERTERS / TEAMS;
  static constexpr int THREADS = 192 + 32 * CONVERTERS + 32;
  static constexpr int NUM_BARS = 2 * (A_STAGES + W_STAGES + BUFS) + 4;
  static constexpr int A0 = 0, BUF0 = A0 + A_STAGES * A_BYTES, W0 = BUF0 + BUFS * BUF_BYTES;
  static constexpr int BARS = W0 + W_STAGES * W_BYTES;
  static constexpr int SMEM_BYTES = 1024 + BARS + NUM_BARS * 8 + 16;
  static constexpr uint32_t TMEM_COLS = 256;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(BUFS % TEAMS == 0 && W_STAGES >= BUFS, "a team has buffers of its own; see its first wait");
};

// Two e4m3 codes to two bf16, times s if SCALED (fp32 product, one rounding;
// without it exact).
template <bool SCALED>
__device__ __forceinline__ uint32_t e4m3x2_bf16x2(uint32_t codes, float s) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3);
  float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  if (SCALED) fma2_scalar(f.x, f.y, s, -0.f);  // one packed product; + -0 changes nothing
  return pack_bf16x2(f.x, f.y);
}

// scale: BATCH and B_MN_MAJOR (absorb): [2 * count][4], entry (2 z) * 4 + nt for
// the accumulator of item z, column tile nt; stream-K: [K / 128][N / 128];
// BATCH and K-major: unused.
template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
gemm_m64_w8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW, int M, int N, int K,
                   const M64Batch bt, const float* __restrict__ scale, float* __restrict__ part,
                   __nv_bfloat16* __restrict__ out, int* err) {
  constexpr int BK = Cfg::BK, SA = Cfg::A_STAGES, SW = Cfg::W_STAGES, NB = Cfg::BUFS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::BARS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Cfg::NUM_BARS);
  int* abort_word = reinterpret_cast<int*>(tmem_slot + 1);
  const uint32_t afull0 = smem_u32(bars), aempty0 = afull0 + 8 * SA;
  const uint32_t wfull0 = aempty0 + 8 * SA, wempty0 = wfull0 + 8 * SW;
  const uint32_t bfull0 = wempty0 + 8 * SW, bempty0 = bfull0 + 8 * NB;
  const uint32_t accf0 = bempty0 + 8 * NB, acce0 = accf0 + 16;
  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < SA; ++s) {
      mbar_init(afull0 + 8 * s, 1);
      mbar_init(aempty0 + 8 * s, 1);
    }
    for (int s = 0; s < SW; ++s) {
      mbar_init(wfull0 + 8 * s, 1);
      mbar_init(wempty0 + 8 * s, Cfg::TEAM);
    }
    for (int b = 0; b < NB; ++b) {
      mbar_init(bfull0 + 8 * b, Cfg::TEAM);
      mbar_init(bempty0 + 8 * b, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(accf0 + 8 * a, 1);
      mbar_init(acce0 + 8 * a, 4);  // the four epilogue warps
    }
    *abort_word = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmW);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), Cfg::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const Abort ab{abort_word, err};
  griddep_launch();

  M64Work work(M, N, K, bt.count, Cfg::BM, Cfg::BATCH);
  M64Seg sg;

  if (warp == 0 || warp == Cfg::THREADS / 32 - 1) {
    if (lane == 0) {
      // ---------------- TMA producers. The weights do not come from the kernels
      // of this chain: their codes are asked for at once, A after the kernel before.
      const bool codes = warp == 0;
      if (!codes) griddep_wait();
      const uint32_t full0 = codes ? wfull0 : afull0, empty0 = codes ? wempty0 : aempty0;
      const uint32_t base = smem_u32(smem) + (codes ? Cfg::W0 : Cfg::A0), bytes = codes ? Cfg::W_BYTES : Cfg::A_BYTES;
      const int stages = codes ? SW : SA;
      int s = 0, left = codes ? 0x7fffffff : bt.most_tiles;
      uint32_t parity = 1;
      bool ok = true, waited = !codes;
      while (ok && work.next(sg)) {
        const int wrow = bt.b_row0 + sg.z * bt.b_step;
        for (int kb = sg.kb0; kb < sg.kb1; ++kb) {
          if (--left < 0 || !mbar_wait_short(empty0 + 8 * s, parity, ab, kErrWaitConsumer)) {
            ok = false;
            break;
          }
          const uint32_t fb = full0 + 8 * s, dst = base + s * bytes;
          const int k = kb * BK;
          mbar_arrive_expect_tx(fb, bytes);
          if (!codes)
            tma_load_2d(dst, &tmA, fb, sg.z * bt.a_step + k, sg.mt * Cfg::BM);  // rows past M read as zero
          else if constexpr (Cfg::B_MN_MAJOR)
            tma_load_2d(dst, &tmW, fb, sg.nt * Cfg::BN, wrow + k);
          else
            tma_load_2d(dst, &tmW, fb, k, wrow + sg.nt * Cfg::BN);
          if (++s == stages) {
            s = 0, parity ^= 1;
            if (!waited) griddep_wait();  // the next lap's stages come free behind A's first tiles
            waited = true;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- UMMA issuer, the whole warp (see umma_ss_pair_x4)
    constexpr uint32_t idesc = idesc_bf16_f32(Cfg::BM, Cfg::BN, 0, Cfg::B_MN_MAJOR ? 1 : 0);
    const uint32_t issue = elect_lane();
    const uint64_t da = smem_desc_sw128(smem_u32(smem + Cfg::A0), 16, 1024);
    const uint64_t db = smem_desc_sw128(smem_u32(smem + Cfg::BUF0), Cfg::B_MN_MAJOR ? BK * 128 : 16, 1024);
    uint32_t s = 0, sp = 0, b = 0, bp = 0;
    int t = 0, last = -1;
    bool ok = true;
    griddep_wait();
    for (; ok && work.next(sg); ++t) {
      const int a = t & 1;
      if (!mbar_wait_short(acce0 + 8 * a, ((t >> 1) & 1) ^ 1, ab, kErrWaitEpilogue)) break;
      tc_fence_after();
      const uint32_t d = tmem_base + a * Cfg::BN;
#pragma unroll 1
      for (int kb = sg.kb0; kb < sg.kb1; ++kb) {
        if (!mbar_wait_short(afull0 + 8 * s, sp, ab, kErrWaitTma) || !mbar_wait_short(bfull0 + 8 * b, bp, ab, kErrWaitSoftmax)) {
          ok = false;
          break;
        }
        tc_fence_after();
        umma_ss_x4<2, Cfg::B_MN_MAJOR ? 128 : 2>(d, da + s * (Cfg::A_BYTES >> 4), db + b * (Cfg::BUF_BYTES >> 4), idesc,
                                                 kb != sg.kb0 ? 1u : 0u, issue);
        umma_commit_warp(aempty0 + 8 * s, issue);
        umma_commit_warp(bempty0 + 8 * b, issue);
        last = static_cast<int>(2 * s + sp);
        if (++s == SA) s = 0, sp ^= 1;
        if (++b == NB) b = 0, bp ^= 1;
      }
      if (!ok) break;
      umma_commit_warp(accf0 + 8 * a, issue);
    }
    if (!ok && last >= 0) mbar_wait_drain(aempty0 + 8 * (last >> 1), last & 1);
  } else if (warp >= 6) {
    // ---------------- converters: 16 codes at a time, 512 such pieces per stage.
    // A row of 64 codes (64 bytes, four pieces) becomes a 128-byte operand row:
    // stored [K, N], code row k holds two, of the 64-column chunks 0 and 1;
    // stored [N, K], one. Eight lanes with neighbouring pieces load 128 bytes, and
    // in the swizzled operand two rows of one parity fill the same four 16-byte
    // columns, so they take an even and an odd row: stored [K, N], chunk 0 of
    // one and chunk 1 of the other. Loads and both stores are then free of bank
    // conflicts (both chunks of one row: stores twice as long, W_o of 128 rows 53 us for 48).
    constexpr int PIECES = 512 / (32 * Cfg::TEAM);
    // Operand row r and chunk c of a piece, and where its codes lie.
    auto place = [](int piece, int& r, int& c) -> int {
      const int u = piece >> 2, q = piece & 3;
      r = Cfg::B_MN_MAJOR ? (u >> 2) << 1 | (u & 1) : u;
      c = Cfg::B_MN_MAJOR ? (u ^ u >> 1) & 1 : 0;
      return Cfg::B_MN_MAJOR ? r * 128 + c * 64 + q * 16 : piece * 16;
    };
    const int me = (static_cast<int>(threadIdx.x) - 192) % (32 * Cfg::TEAM), team = (warp - 6) / Cfg::TEAM;
    int it = 0;
    bool ok = true;
    while (ok && work.next(sg)) {
#pragma unroll 1
      for (int kb = sg.kb0; kb < sg.kb1; ++kb, ++it) {
        if (it % Cfg::TEAMS != team) continue;
        if (it / NB == 1) griddep_wait();  // from here on a buffer comes free behind A's tiles
        const int s = it % SW, b = it % NB;
        float f = 1.f;
        if constexpr (!Cfg::BATCH) f = __ldg(scale + static_cast<int64_t>(kb >> 1) * (N / 128) + sg.nt);
        // The buffer first: once the product four tiles before is done with it, all
        // codes up to that tile have landed, the lap before of this stage among
        // them. A stage is taken by two teams in turn and loads land in any
        // order, so the other way round the parity of two laps before could
        // let a team through to old codes.
        if (!(ok = warp_wait_all(bempty0 + 8 * b, ((it / NB) & 1) ^ 1, ab, kErrWaitMma))) break;
        if (!(ok = warp_wait_all(wfull0 + 8 * s, (it / SW) & 1, ab, kErrWaitTma))) break;
        const uint8_t* src = smem + Cfg::W0 + s * Cfg::W_BYTES;
        uint4 w[PIECES];
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          int r, c;
          w[i] = *reinterpret_cast<const uint4*>(src + place(me + i * 32 * Cfg::TEAM, r, c));
        }
        uint8_t* dst = smem + Cfg::BUF0 + b * Cfg::BUF_BYTES;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          const int piece = me + i * 32 * Cfg::TEAM, q = piece & 3;
          int r, c;
          place(piece, r, c);
          const uint32_t in[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[2 * e] = e4m3x2_bf16x2<!Cfg::BATCH>(in[e], f);
            o[2 * e + 1] = e4m3x2_bf16x2<!Cfg::BATCH>(in[e] >> 16, f);
          }
          uint8_t* d = dst + c * BK * 128 + r * 128;
          *reinterpret_cast<uint4*>(d + (((2 * q) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(d + (((2 * q + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        // For the stores, which the tensor core reads, and the loads of the codes,
        // whose stage TMA writes again: without it before the stage's release,
        // loads came after that write, in a tile or so per call.
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bfull0 + 8 * b);
          mbar_arrive(wempty0 + 8 * s);
        }
      }
    }
  } else {
    // ---------------- epilogue: rows [16q, 16q+16) of the tile in lanes 0..15
    // (M = 64) or [32q, 32q+32) in all lanes (M = 128)
    constexpr int RPW = Cfg::BM / 4;  // rows per warp
    const int q = warp & 3;
    int t = 0;
    griddep_wait();
    for (; work.next(sg); ++t) {
      const int a = t & 1;
      float f = 1.f;
      if constexpr (Cfg::BATCH && Cfg::B_MN_MAJOR) f = __ldg(scale + 8 * sg.z + sg.nt);
      if (!warp_wait(accf0 + 8 * a, (t >> 1) & 1, ab, kErrWaitMma)) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + a * Cfg::BN;
      const int row = sg.mt * Cfg::BM + RPW * q + static_cast<int>(lane);
#pragma unroll 1
      for (int c = 0; c < Cfg::BN; c += 32) {
        uint32_t v[32];
        tmem_ld32(tb + c, v);
        if (static_cast<int>(lane) < RPW && row < M) {
          if constexpr (Cfg::BATCH) {
            uint4* d4 = reinterpret_cast<uint4*>(out + static_cast<size_t>(row) * bt.ldc + sg.z * bt.c_step +
                                                 sg.nt * Cfg::BN + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t o[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                o[e] = pack_bf16x2(__uint_as_float(v[8 * i + 2 * e]) * f, __uint_as_float(v[8 * i + 2 * e + 1]) * f);
              d4[i] = make_uint4(o[0], o[1], o[2], o[3]);
            }
          } else {
            float4* d4 = reinterpret_cast<float4*>(
                part + (static_cast<size_t>(sg.slot) * Cfg::BM + (row - sg.mt * Cfg::BM)) * Cfg::BN + c);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              d4[i] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                  __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acce0 + 8 * a);
    }
  }

  tc_fence_before();
  __syncthreads();
  // After a wait has run out in any warp, what others have asked for must land
  // before the CTA can exit.
  if (ab.raised()) spin_ns(2000000);
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
}

}  // namespace mla
