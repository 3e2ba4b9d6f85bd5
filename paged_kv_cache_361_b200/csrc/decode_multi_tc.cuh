// pa_decode_multi with more than 8 rows (new tokens x query heads) per
// (sequence, kv head), on tcgen05.mma with the accumulators in tensor memory.
// The mathematics, the masks and the division of the work are those of
// decode_multi.cuh.
//
// From 24 rows or so an mma.sync form is bound by its products, not by HBM (40
// rows: 1.15 ms for 1.15 GB). Here the rows of a (sequence, kv head), at most
// 16 x 8 = 128, are the M of one MMA, so every K/V byte is read once whatever the
// row count. The tensor cores have the padding to spare: S and P V of 64 keys
// take about 640 cycles at M 128, the 32 KB of those keys 1400 cycles of the SM's
// share of HBM. What has to be kept short is the chain S -> softmax -> P -> P V:
//   * two softmax warpgroups work on two 64-key halves of a 128-key stage, each
//     with its own running maximum, sum and O in tensor memory;
//   * with 64 rows or fewer the rows are there RF = 2 or 4 times, in other TMEM
//     lanes (a warp reaches 32 lanes): the replicas' warps take a quarter or half
//     of the half's keys each (their weights for the others are zeros) and have
//     their own maximum, sum and O.
// The 2 RF states of a row are folded at a segment's end.
//
// Measured (kernels back to back in a graph, inputs larger than L2): 16 sequences of
// 1000..32768 keys, 5 tokens of 64/8 heads (40 rows): 187 to 193 us, 6.0 to 6.2 TB/s,
// 0.91 to 0.94 of a copy's rate (in runs of seconds the power cap lowers the clock to
// 1.45 GHz and the chain is the longer side: 215 us); 32 of 1024..8192, 8 tokens of 32/8
// heads: 110 us over bf16, 5.6 TB/s, 131 to 137 us over e4m3, 2.3 to 2.4 TB/s, bound by
// the converter and the chain.
//
// Warps: 0-3 and 4-7 softmax of half t (thread = row = TMEM lane), 8 producer
// (K; over an 8-bit cache K and V codes), 9 MMA issuer, 10-13 converter (V bf16
// -> f16 in place, or codes -> f16 K and V; rows outside [kbeg, kend) as zeros),
// 14 V producer (bf16). A kind::f16 MMA takes both operands of one type, and
// the weights are f16 (11 bits): so V is f16. Every role walks the worker's
// segments by itself; the rings and phases run on from one to the next.
#pragma once

#include "decode_multi.cuh"
#include "prefill_tc.cuh"

namespace pa {

template <int D, int CF>
struct MultiTcCfg {
  static constexpr bool F8 = CF != 0;
  static constexpr int kHalf = 64;                          // keys of a warpgroup per stage
  static constexpr int kKeys = 2 * kHalf;                   // keys per stage
  static constexpr int kCols = D / 64;                      // 128-byte box columns of a 16-bit row
  static constexpr int kColBytes = kKeys * 128;             // one box column of K or V in a stage
  static constexpr int kTileBytes = kCols * kColBytes;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kCodeTileBytes = kKeys * D;
  static constexpr int kCodeStageBytes = 2 * kCodeTileBytes;
  static constexpr int kStages = D == 128 ? (F8 ? 2 : 3) : (F8 ? 3 : 4);
  static constexpr int kCodeStages = F8 ? (D == 128 ? 2 : 3) : 0;
  static constexpr int kQColBytes = 128 * 128;
  static constexpr int kQBytes = kCols * kQColBytes;
  static constexpr int kSmemBytes = 1024 + kQBytes + kStages * kStageBytes + kCodeStages * kCodeStageBytes;
  static constexpr int kProducerWarp = 8, kMmaWarp = 9, kConvWarp0 = 10, kConvWarps = 4, kVProducerWarp = 14;
  static constexpr int kThreads = 32 * (F8 ? 14 : 15);
  // TMEM: O of each half, then two buffers of S (keys of half 0, then 1), each
  // half's P in the place of its S
  static constexpr uint32_t kSCol = 2 * D;
  static constexpr int kRowPitch = D + 4;                   // floats of a row in the fold
  static constexpr int kMinChunks = kMultiTcMinKeys / kKeys;
  static_assert(kSmemBytes <= 226 * 1024, "shared memory");
  static_assert(128 * (kRowPitch + 2) * 4 <= kStages * kStageBytes, "merge buffer");
};

template <int D, int CF, int RF>
__global__ void __launch_bounds__(MultiTcCfg<D, CF>::kThreads, 1)
    decode_multi_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                           const MultiArgs a) {
  using Cfg = MultiTcCfg<D, CF>;
  constexpr bool F8 = Cfg::F8;
  constexpr int S = Cfg::kStages, C = Cfg::kHalf, CK = Cfg::kKeys, CS = F8 ? Cfg::kCodeStages : 1;
  constexpr int RC = 128 / RF, CW = C / RF;  // rows, and keys of a softmax thread per chunk

  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t kfull[S], kempty[S];             // 16-bit stages (bf16: their K)
  __shared__ uint64_t vfull[S], vempty[S], vready[S];  // bf16: V of a stage, and V rewritten as f16
  __shared__ uint64_t cfull[CS], cempty[CS];           // 8-bit: code staging ring
  __shared__ uint64_t s_full[2], p_full[2][2], o_bar[2], o_last[2], q_full, drain;
  __shared__ uint64_t seg_done;  // a segment's rows are out: its stages (the fold's memory) may be filled again
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag, stop;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw);
  const uint32_t kv0 = sbase + Cfg::kQBytes;
  const uint32_t cs0 = kv0 + S * Cfg::kStageBytes;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
    mbar_init(&q_full, 8);
    mbar_init(&seg_done, 8);
    mbar_init(&drain, 1);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t][0], 4);
      mbar_init(&p_full[t][1], 4);
      mbar_init(&o_bar[t], 1);
      mbar_init(&o_last[t], 1);
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
      mbar_init(&kfull[i], F8 ? Cfg::kConvWarps : 1);
      mbar_init(&kempty[i], 1);
      mbar_init(&vfull[i], 1);
      mbar_init(&vempty[i], 1);
      mbar_init(&vready[i], Cfg::kConvWarps);
    }
#pragma unroll
    for (int i = 0; i < CS; ++i) {
      mbar_init(&cfull[i], 1);
      mbar_init(&cempty[i], Cfg::kConvWarps);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == Cfg::kMmaWarp) {
    tc::alloc(smem_u32(&tmem_base_sh), 512);
    tc::relinquish();
    tc::fence_before();
  }
  MultiWalk<CK> walk(find_work<CK>(a, blockIdx.x, gridDim.x, Cfg::kMinChunks, warp == 0), blockIdx.x);
  MultiSegment e;
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_base_sh;
  int jg = 0;  // chunks of the segments before, in every role's count

  if (warp == Cfg::kProducerWarp || (!F8 && warp == Cfg::kVProducerWarp)) {
    // ---- producers: every chunk's blocks that hold a key in [kbeg, kend) ----
    const bool is_v = !F8 && warp == Cfg::kVProducerWarp;
    constexpr int R = F8 ? CS : S;
    uint64_t* full = F8 ? cfull : (is_v ? vfull : kfull);
    uint64_t* empty = F8 ? cempty : (is_v ? vempty : kempty);
    const CUtensorMap* map = is_v ? &tmv : &tmk;
    const uint32_t box_bytes = static_cast<uint32_t>(a.bs) * (F8 ? D : 128);  // of one box column
    const uint64_t pol = kv_stream_policy();
    bool ok = true;
    int si = 0;  // segments with keys so far
    while (ok && walk.next(a, e)) {
      if (e.chunks == 0) continue;
      BlocksAhead<CK> ahead;
      ahead.init(a, e, lane);
      if (si > 0 && !warp_wait(&seg_done, (si - 1) & 1, &abort_flag)) break;
      ++si;
      for (int j = 0; j < e.chunks; ++j, ++jg) {
        const int st = jg % R;
        if (jg >= R && !warp_wait(&empty[st], ((jg / R) - 1) & 1, &abort_flag)) {
          ok = false;
          break;
        }
        int32_t blk;
        const bool in = ahead.next(a, e, e.begin + j * CK, lane, !is_v, blk);
        const int cnt = __popc(__ballot_sync(0xffffffffu, in));
        if (lane == 0) mbar_arrive_expect_tx(&full[st], (F8 ? 2u : Cfg::kCols) * cnt * box_bytes);
        __syncwarp();
        if (in) {
          const int32_t y = (blk * a.hkv + e.g) * a.bs;
          if constexpr (F8) {
            const uint32_t dst = cs0 + st * Cfg::kCodeStageBytes + lane * box_bytes;
            tma_load_2d(dst, &tmk, 0, y, &full[st], pol);
            tma_load_2d(dst + Cfg::kCodeTileBytes, &tmv, 0, y, &full[st], pol);
          } else {
            const uint32_t dst = kv0 + st * Cfg::kStageBytes + (is_v ? Cfg::kTileBytes : 0) + lane * box_bytes;
#pragma unroll
            for (int hf = 0; hf < Cfg::kCols; ++hf)
              tma_load_2d(dst + hf * Cfg::kColBytes, map, hf * 64, y, &full[st], pol);
          }
        }
      }
    }
    if (abort_flag && lane == 0)  // copies already started land before exit
      for (int j = (jg > R ? jg - R : 0); j < jg; ++j) mbar_wait(&full[j % R], (j / R) & 1);
  } else if (warp >= Cfg::kConvWarp0 && warp < Cfg::kConvWarp0 + Cfg::kConvWarps) {
    // ---- converter: thread = (row of a half, half of its dims), both halves ----
    const int ct = tid - 32 * Cfg::kConvWarp0;
    const int row = ct >> 1, half = ct & 1;
    bool ok = true;
    while (ok && walk.next(a, e)) {
      for (int j = 0; j < e.chunks; ++j, ++jg) {
        const int st = jg % S;
        uint8_t* stage = sgen + Cfg::kQBytes + st * Cfg::kStageBytes;
        if constexpr (F8) {
          const int cst = jg % CS;
          ok = warp_wait(&cfull[cst], (jg / CS) & 1, &abort_flag) &&
               (jg < S || warp_wait(&kempty[st], ((jg / S) - 1) & 1, &abort_flag));
          if (!ok) break;
          const uint8_t* src = sgen + (cs0 - sbase) + cst * Cfg::kCodeStageBytes;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int rr = u * C + row;
            const int32_t key = e.begin + j * CK + rr;
            const bool live = key >= e.kbeg && key < e.kend;
            widen_row_half<D, CF, Cfg::kColBytes>(src, stage, rr, half, live);
            widen_row_half<D, CF, Cfg::kColBytes>(src + Cfg::kCodeTileBytes, stage + Cfg::kTileBytes, rr, half, live);
          }
          tc::fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&kfull[st]);
            mbar_arrive(&cempty[cst]);
          }
        } else {
          ok = warp_wait(&vfull[st], (jg / S) & 1, &abort_flag);
          if (!ok) break;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int rr = u * C + row;
            const int32_t key = e.begin + j * CK + rr;
            v_to_f16_inplace<D, Cfg::kColBytes>(stage + Cfg::kTileBytes, rr, half, key >= e.kbeg && key < e.kend);
          }
          tc::fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&vready[st]);
        }
      }
    }
  } else if (warp == Cfg::kMmaWarp) {
    // ---- MMA issuer: S(j + 1), then O_t += P_t(j) V_t(j) of each half. S is one
    // product over the stage's 128 keys (64 cycles a step; two of 64 keys, bound by
    // reading q twice, 96) ----
    constexpr uint32_t kIdS = F8 ? tc::idesc_f16(128, CK, false) : tc::idesc_bf16(128, CK, false);
    constexpr uint32_t kIdPV = tc::idesc_f16(128, D, true);
    const uint64_t qdesc0 = tc::smem_desc(sbase, 16, 1024);
    const uint64_t kdesc0 = tc::smem_desc(kv0, 16, 1024);
    const uint64_t vdesc0 = tc::smem_desc(kv0 + Cfg::kTileBytes, Cfg::kCols > 1 ? Cfg::kColBytes : 1024, 1024);
    auto issue_s = [&](int j) {
      const uint64_t kb = kdesc0 + static_cast<uint64_t>(((j % S) * Cfg::kStageBytes) >> 4);
      const uint32_t dst = tmem + Cfg::kSCol + (j & 1) * CK;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t offq = static_cast<uint32_t>((kk >> 2) * Cfg::kQColBytes + (kk & 3) * 32) >> 4;
        const uint32_t offk = static_cast<uint32_t>((kk >> 2) * Cfg::kColBytes + (kk & 3) * 32) >> 4;
        tc::mma_ss(dst, qdesc0 + offq, kb + offk, kIdS, kk > 0);
      }
      tc::commit(smem_u32(&s_full[j & 1]));
    };
    auto issue_pv = [&](int t, int j, bool first, bool last) -> bool {
      const int sb = j & 1;
      if (!warp_wait(&p_full[t][sb], (j >> 1) & 1, &abort_flag)) return false;
      tc::fence_after();
      const uint64_t vb = vdesc0 + static_cast<uint64_t>(((j % S) * Cfg::kStageBytes + t * C * 128) >> 4);
      const uint32_t to = tmem + t * D, tp = tmem + Cfg::kSCol + sb * CK + t * C;
#pragma unroll
      for (int ks = 0; ks < C / 16; ++ks)
        tc::mma_ts(to, tp + ks * 8, vb + static_cast<uint64_t>((ks * 16 * 128) >> 4), kIdPV, !first || ks > 0);
      tc::commit(smem_u32(&o_bar[t]));
      if (last) tc::commit(smem_u32(&o_last[t]));
      return true;
    };
    bool ok = true;
    int qi = 0;
    while (ok && walk.next(a, e)) {
      const int j0 = jg, j1 = jg + e.chunks;
      jg = j1;
      if (j0 == j1) continue;
      // (q of this segment: its O of the one before has been read too)
      ok = warp_wait(&q_full, qi & 1, &abort_flag) && warp_wait(&kfull[j0 % S], (j0 / S) & 1, &abort_flag);
      ++qi;
      tc::fence_after();
      if (ok) {
        issue_s(j0);
        if constexpr (!F8) tc::commit(smem_u32(&kempty[j0 % S]));  // the stage's K is read once these finish
      }
      for (int j = j0; ok && j < j1; ++j) {
        if (j + 1 < j1) {
          if (!(ok = warp_wait(&kfull[(j + 1) % S], ((j + 1) / S) & 1, &abort_flag))) break;
          tc::fence_after();
          issue_s(j + 1);
          if constexpr (!F8) tc::commit(smem_u32(&kempty[(j + 1) % S]));
        }
        if constexpr (!F8) {
          if (!(ok = warp_wait(&vready[j % S], (j / S) & 1, &abort_flag))) break;
          tc::fence_after();
        }
        ok = issue_pv(0, j, j == j0, j + 1 == j1) && issue_pv(1, j, j == j0, j + 1 == j1);
        if (ok) tc::commit(smem_u32(F8 ? &kempty[j % S] : &vempty[j % S]));
      }
    }
    if (jg > 0) {
      tc::commit(smem_u32(&drain));  // every MMA issued has finished before TMEM is released
      mbar_wait(&drain, 0);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ---- softmax of half t: thread = row rho of replica rep ----
    const int t = warp >> 2, r = tid & 127, rho = r % RC, rep = r / RC;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t trow = lanes + t * D, srow = lanes + Cfg::kSCol + t * C;  // O, and S of buffer 0
    float* stage0 = reinterpret_cast<float*>(sgen + Cfg::kQBytes);  // the fold: rows of O, then (m, l) of each half
    float* stg = stage0 + r * Cfg::kRowPitch;
    float* ml = stage0 + 128 * Cfg::kRowPitch;
    const CapPoly poly(a.score.cap_log2);
    int qi = 0;
    while (walk.next(a, e)) {
      if (e.chunks == 0) {  // rows that see no key
        for (int i = tid; i < e.rows * (D / 4); i += 256)
          store_multi<D>(a, e, i / (D / 4), i % (D / 4) * 4, -INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f));
        continue;
      }
      const bool active = rho - lane < e.rows;  // some row of the warp is live (rho - lane: the warp's first)
      const bool valid = rho < e.rows;
      const int32_t pos0 = e.ms.L - e.ms.n;
      const int32_t pos = valid ? pos0 + (rho >> a.gshift) : pos0;
      const int32_t lo = max(e.kbeg, pos - a.window + 1), hi = min(e.kend - 1, pos);  // the keys the row sees here
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      {
        // q: each warpgroup half of the row's 16-byte pieces
        constexpr int NP = D / 16;
        const uint4* src = reinterpret_cast<const uint4*>(a.q + multi_row(a, e, valid ? rho : 0) * D) + t * NP;
        uint4 qv[NP];
#pragma unroll
        for (int u = 0; u < NP; ++u) qv[u] = valid ? __ldg(src + u) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int u = 0; u < NP; ++u) {
          uint4 v = qv[u];
          if constexpr (F8)
            v = make_uint4(pack_f16(bf16lo(v.x), bf16hi(v.x)), pack_f16(bf16lo(v.y), bf16hi(v.y)),
                           pack_f16(bf16lo(v.z), bf16hi(v.z)), pack_f16(bf16lo(v.w), bf16hi(v.w)));
          const int c16 = t * NP + u, hf = c16 >> 3, cc = c16 & 7;
          *reinterpret_cast<uint4*>(sgen + hf * Cfg::kQColBytes + r * 128 + ((cc ^ (r & 7)) << 4)) = v;
        }
        tc::fence_proxy_async();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full);
      }
      for (int j = 0; j < e.chunks; ++j, ++jg) {
        const int sb = jg & 1;
        if (!warp_wait(&s_full[sb], (jg >> 1) & 1, &abort_flag)) {
          ok = false;
          break;
        }
        if (active) {
          tc::fence_after();
          uint32_t sr[CW];
          if constexpr (RF == 4) {
            tc::ld16(srow + sb * CK + rep * CW, sr);
          } else {
            tc::ld32(srow + sb * CK + rep * CW, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
            if constexpr (RF == 1) tc::ld32(srow + sb * CK + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
          }
          tc::wait_ld();
          const int32_t k0 = e.begin + j * CK + t * C + rep * CW;
          float x[CW], amax = 0.f;
#pragma unroll
          for (int c = 0; c < CW; ++c) x[c] = __uint_as_float(sr[c]);
          if (!__all_sync(0xffffffffu, k0 >= lo && k0 + CW - 1 <= hi))
            amax = masked_amax(x, lo - k0, hi - k0);
          else if (a.score.cap_log2 > 0.f)
            amax = row_amax(x);
          float alpha;
          bool resc;
          uint32_t ph[CW / 2];
          if (a.score.cap_log2 > 0.f)
            row_weights<true>(a.score, x, amax, poly, m, l, alpha, resc, ph);
          else
            row_weights<false>(a.score, x, 0.f, poly, m, l, alpha, resc, ph);
          uint32_t pw[C / 2];  // the weights of the half's 64 keys: zeros where another replica has them
#pragma unroll
          for (int c = 0; c < C / 2; ++c) pw[c] = RF == 1 || c / (CW / 2) == rep ? ph[c % (CW / 2)] : 0u;
          __syncwarp();
          tc::st32(srow + sb * CK, pw);
          if (__any_sync(0xffffffffu, resc)) {
            // O must hold P(j-1) V(j-1) before it is rescaled
            if (!warp_wait(&o_bar[t], (jg - 1) & 1, &abort_flag)) {
              tc::wait_st();
              ok = false;
              break;
            }
            tc::fence_after();
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[32];
              __syncwarp();
              tc::ld32(trow + q * 32, o);
              tc::wait_ld();
              if (resc) {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              }
              __syncwarp();
              tc::st32(trow + q * 32, o);
            }
          }
          __syncwarp();
          tc::wait_st();
          tc::fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t][sb]);
      }
      m = final_ref(m, l);
      if (ok) ok = warp_wait(&o_last[t], qi & 1, &abort_flag);
      ++qi;
      // fold: half 1 leaves (m, l, o) of its rows in the stages (no MMA or copy
      // uses them once both halves' last P V have completed), half 0 folds its own
      // in, then every thread stores rows, folding the replicas. A warp that gave
      // up a wait joins every barrier; thread 0 decides for all.
      auto bar = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
      const bool live = active && ok;
      tc::fence_after();
      bar();
      if (t == 1 && active) {
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          __syncwarp();
          if (live) {
            tc::ld32(trow + q * 32, o);
            tc::wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(stg + q * 32 + 4 * i) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
        ml[2 * r] = m;
        ml[2 * r + 1] = l;
      }
      bar();
      if (t == 0 && active) {
        const float m1 = ml[2 * r], l1 = ml[2 * r + 1], M = fmaxf(m, m1);
        const float f0 = M == -INFINITY ? 0.f : exp2f(m - M), f1 = M == -INFINITY ? 0.f : exp2f(m1 - M);
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          __syncwarp();
          if (live) {
            tc::ld32(trow + q * 32, o);
            tc::wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float4* d = reinterpret_cast<float4*>(stg + q * 32 + 4 * i);
            const float4 y = *d;
            *d = make_float4(fmaf(y.x, f1, __uint_as_float(o[4 * i]) * f0), fmaf(y.y, f1, __uint_as_float(o[4 * i + 1]) * f0),
                             fmaf(y.z, f1, __uint_as_float(o[4 * i + 2]) * f0),
                             fmaf(y.w, f1, __uint_as_float(o[4 * i + 3]) * f0));
          }
        }
        ml[2 * r] = M;
        ml[2 * r + 1] = l * f0 + l1 * f1;
      }
      if (tid == 0) stop = *static_cast<volatile int*>(&abort_flag);
      bar();
      if (stop) break;
      constexpr int LR = D / 4;  // threads of a row: whole lines
      const int d = (tid % LR) * 4;
      for (int row = tid / LR; row < e.rows; row += 256 / LR) {
        float M = ml[2 * row], L = ml[2 * row + 1];
        float4 y = *reinterpret_cast<const float4*>(stage0 + row * Cfg::kRowPitch + d);
#pragma unroll
        for (int u = 1; u < RF; ++u) {
          const float m1 = ml[2 * (row + u * RC)], l1 = ml[2 * (row + u * RC) + 1], Mn = fmaxf(M, m1);
          const float4 z = *reinterpret_cast<const float4*>(stage0 + (row + u * RC) * Cfg::kRowPitch + d);
          const float f0 = Mn == -INFINITY ? 0.f : exp2f(M - Mn), f1 = Mn == -INFINITY ? 0.f : exp2f(m1 - Mn);
          L = L * f0 + l1 * f1;
          y = make_float4(y.x * f0 + z.x * f1, y.y * f0 + z.y * f1, y.z * f0 + z.z * f1, y.w * f0 + z.w * f1);
          M = Mn;
        }
        store_multi<D>(a, e, row, d, M, L, y);
      }
      tc::fence_proxy_async();  // these reads and writes before the next segment's copies
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_done);
    }
    tc::fence_before();
  }
  pdl_launch_dependents();
  __syncthreads();
  if (warp == Cfg::kMmaWarp) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

}  // namespace pa
