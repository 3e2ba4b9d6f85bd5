// pa_decode_multi with more than 16 rows (new tokens x query heads) per
// (sequence, kv head), on tcgen05.mma with the accumulators in tensor memory.
// The mathematics, the masks and the partitions are those of decode_multi.cuh.
//
// From 24 rows or so the mma.sync form is bound by its products, not by HBM (40
// rows: 1.15 ms for 1.15 GB). Here the rows of a (sequence, kv head), at most
// 16 x 8 = 128, are the M of one MMA (rows past them are not computed on: their
// softmax warps idle), so every K/V byte is read once whatever the row count.
// The tensor cores have the padding to spare: S and P V of 64 keys take about
// 640 cycles at M 128, the 32 KB of those keys 1400 cycles of the SM's share of
// HBM. What has to be kept short is the chain S -> softmax -> P -> P V, so two
// softmax warpgroups work on two 64-key halves of a 128-key stage, each with its
// own running maximum, sum and O in tensor memory; they are merged at the end.
//
// Warps: 0-3 and 4-7 softmax of half t (thread = row = TMEM lane), 8 producer
// (K; over an 8-bit cache K and V codes), 9 MMA issuer, 10-13 converter (V bf16
// -> f16 in place, or codes -> f16 K and V; rows outside [kbeg, kend) as zeros),
// 14 V producer (bf16). A kind::f16 MMA takes both operands of one type, and
// the weights are f16 (11 bits): so V is f16.
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
  static constexpr uint32_t kTileCols = D + 2 * kHalf;      // TMEM of a half: O, then two S/P buffers
  static constexpr int kRowPitch = D + 4;                   // floats of a row in the merge
  static_assert(kSmemBytes <= 226 * 1024, "shared memory");
  static_assert(128 * (kRowPitch + 2) * 4 <= kStages * kStageBytes, "merge buffer");
};

template <int D, int CF>
__global__ void __launch_bounds__(MultiTcCfg<D, CF>::kThreads, 1)
    decode_multi_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                           const MultiArgs a) {
  using Cfg = MultiTcCfg<D, CF>;
  constexpr bool F8 = Cfg::F8;
  constexpr int S = Cfg::kStages, C = Cfg::kHalf, CK = Cfg::kKeys, CS = F8 ? Cfg::kCodeStages : 1;

  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t kfull[S], kempty[S];            // 16-bit stages (bf16: their K)
  __shared__ uint64_t vfull[S], vempty[S], vready[S];  // bf16: V of a stage, and V rewritten as f16
  __shared__ uint64_t cfull[CS], cempty[CS];           // 8-bit: code staging ring
  __shared__ uint64_t s_full[2][2], p_full[2][2], o_bar[2], o_last[2], q_full, drain;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw);
  const uint32_t kv0 = sbase + Cfg::kQBytes;
  const uint32_t cs0 = kv0 + S * Cfg::kStageBytes;

  const int g = blockIdx.x, s = blockIdx.y, p = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const MultiSeq ms = load_multi_seq(a, s, g == 0 && p == 0 && tid == 0);
  const int rows = ms.n << a.gshift;
  if (rows <= 0 || p >= ms.nparts) return;
  const int32_t pos0 = ms.L - ms.n;
  const int32_t t0 = ms.nparts > 1 ? ms.first + p * a.part_tokens : 0;
  const int32_t t1 = ms.nparts > 1 && p < ms.nparts - 1 ? t0 + a.part_tokens : ms.L;
  const int32_t kbeg = max(t0, max(0, pos0 - a.window + 1)), kend = t1;
  const int32_t c_begin = kbeg & ~(C - 1);
  const int nchunks = kend > kbeg ? (kend - c_begin + CK - 1) / CK : 0;
  const int na = (rows + 31) / 32;  // softmax warps of a half with rows
  auto out_row = [&](int rho) {
    return static_cast<int64_t>(ms.q0 + (rho >> a.gshift)) * a.hq + (g << a.gshift) + (rho & ((1 << a.gshift) - 1));
  };

  if (tid == 0) {
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
    mbar_init(&q_full, 2 * na);
    mbar_init(&drain, 1);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t][0], 1);
      mbar_init(&s_full[t][1], 1);
      mbar_init(&p_full[t][0], na);
      mbar_init(&p_full[t][1], na);
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
  TableAhead ta;
  if (warp == Cfg::kProducerWarp || (!F8 && warp == Cfg::kVProducerWarp))
    ta.init(a.tables + static_cast<int64_t>(s) * a.max_blocks, c_begin / a.bs,
            min(a.max_blocks, (kend + a.bs - 1) / a.bs), lane);
  if (warp == Cfg::kMmaWarp) {
    tc::alloc(smem_u32(&tmem_base_sh), 512);
    tc::relinquish();
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_base_sh;

  if (warp == Cfg::kProducerWarp || (!F8 && warp == Cfg::kVProducerWarp)) {
    // ---- producers: chunk i's blocks that hold a key in [kbeg, kend) ----
    const bool is_v = !F8 && warp == Cfg::kVProducerWarp;
    constexpr int R = F8 ? CS : S;
    uint64_t* full = F8 ? cfull : (is_v ? vfull : kfull);
    uint64_t* empty = F8 ? cempty : (is_v ? vempty : kempty);
    const CUtensorMap* map = is_v ? &tmv : &tmk;
    const uint32_t box_bytes = static_cast<uint32_t>(a.bs) * (F8 ? D : 128);  // of one box column
    const uint64_t pol = kv_stream_policy();
    int i = 0;
    for (; i < nchunks; ++i) {
      const int st = i % R;
      if (i >= R && !warp_wait(&empty[st], ((i / R) - 1) & 1, &abort_flag)) break;
      const int32_t c0 = c_begin + i * CK;
      bool ok[2] = {false, false};
      int32_t blk[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {  // 64 keys at a time: at most 8 blocks each
        const int32_t h0 = c0 + u * C;
        const int32_t nb = h0 < kend ? (min(C, kend - h0) + a.bs - 1) / a.bs : 0;
        blk[u] = ta.get(h0 / a.bs, nb, lane);
        if (lane < nb && h0 + (lane + 1) * a.bs > kbeg) {
          ok[u] = blk[u] >= 0 && blk[u] < a.num_blocks;
          if (!ok[u] && !is_v) record_error(PA_ERR_DEVICE_BOUNDS, blk[u]);
        }
      }
      const int cnt = __popc(__ballot_sync(0xffffffffu, ok[0])) + __popc(__ballot_sync(0xffffffffu, ok[1]));
      if (lane == 0) mbar_arrive_expect_tx(&full[st], (F8 ? 2u : Cfg::kCols) * cnt * box_bytes);
      __syncwarp();
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (ok[u]) {
          const int32_t y = (blk[u] * a.hkv + g) * a.bs;
          const uint32_t off = u * (C * (F8 ? D : 128)) + lane * box_bytes;
          if constexpr (F8) {
            const uint32_t dst = cs0 + st * Cfg::kCodeStageBytes + off;
            tma_load_2d(dst, &tmk, 0, y, &full[st], pol);
            tma_load_2d(dst + Cfg::kCodeTileBytes, &tmv, 0, y, &full[st], pol);
          } else {
            const uint32_t dst = kv0 + st * Cfg::kStageBytes + (is_v ? Cfg::kTileBytes : 0) + off;
#pragma unroll
            for (int hf = 0; hf < Cfg::kCols; ++hf) tma_load_2d(dst + hf * Cfg::kColBytes, map, hf * 64, y, &full[st], pol);
          }
        }
    }
    if (abort_flag && lane == 0)  // copies already started land before exit
      for (int j = (i > R ? i - R : 0); j < i; ++j) mbar_wait(&full[j % R], (j / R) & 1);
  } else if (warp >= Cfg::kConvWarp0 && warp < Cfg::kConvWarp0 + Cfg::kConvWarps) {
    // ---- converter: thread = (row of a half, half of its dims), both halves ----
    const int ct = tid - 32 * Cfg::kConvWarp0;
    const int row = ct >> 1, half = ct & 1;
    for (int i = 0; i < nchunks; ++i) {
      const int st = i % S;
      uint8_t* stage = sgen + Cfg::kQBytes + st * Cfg::kStageBytes;
      if constexpr (F8) {
        const int cst = i % CS;
        if (!warp_wait(&cfull[cst], (i / CS) & 1, &abort_flag)) break;
        if (i >= S && !warp_wait(&kempty[st], ((i / S) - 1) & 1, &abort_flag)) break;
        const uint8_t* src = sgen + (cs0 - sbase) + cst * Cfg::kCodeStageBytes;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int rr = u * C + row;
          const int32_t key = c_begin + i * CK + rr;
          const bool live = key >= kbeg && key < kend;
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
        if (!warp_wait(&vfull[st], (i / S) & 1, &abort_flag)) break;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int rr = u * C + row;
          const int32_t key = c_begin + i * CK + rr;
          v_to_f16_inplace<D, Cfg::kColBytes>(stage + Cfg::kTileBytes, rr, half, key >= kbeg && key < kend);
        }
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&vready[st]);
      }
    }
  } else if (warp == Cfg::kMmaWarp) {
    // ---- MMA issuer: S_t(j + 1) of both halves, then O_t += P_t(j) V_t(j) ----
    constexpr uint32_t kIdS = F8 ? tc::idesc_f16(128, C, false) : tc::idesc_bf16(128, C, false);
    constexpr uint32_t kIdPV = tc::idesc_f16(128, D, true);
    const uint64_t qdesc0 = tc::smem_desc(sbase, 16, 1024);
    const uint64_t kdesc0 = tc::smem_desc(kv0, 16, 1024);
    const uint64_t vdesc0 = tc::smem_desc(kv0 + Cfg::kTileBytes, Cfg::kCols > 1 ? Cfg::kColBytes : 1024, 1024);
    auto issue_s = [&](int t, int j) {
      const uint64_t kb = kdesc0 + static_cast<uint64_t>(((j % S) * Cfg::kStageBytes + t * C * 128) >> 4);
      const uint32_t dst = tmem + t * Cfg::kTileCols + D + (j & 1) * C;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t offq = static_cast<uint32_t>((kk >> 2) * Cfg::kQColBytes + (kk & 3) * 32) >> 4;
        const uint32_t offk = static_cast<uint32_t>((kk >> 2) * Cfg::kColBytes + (kk & 3) * 32) >> 4;
        tc::mma_ss(dst, qdesc0 + offq, kb + offk, kIdS, kk > 0);
      }
      tc::commit(smem_u32(&s_full[t][j & 1]));
    };
    auto issue_pv = [&](int t, int j) -> bool {
      const int sb = j & 1;
      if (!warp_wait(&p_full[t][sb], (j >> 1) & 1, &abort_flag)) return false;
      tc::fence_after();
      const uint64_t vb = vdesc0 + static_cast<uint64_t>(((j % S) * Cfg::kStageBytes + t * C * 128) >> 4);
      const uint32_t to = tmem + t * Cfg::kTileCols, tp = to + D + sb * C;
#pragma unroll
      for (int ks = 0; ks < C / 16; ++ks)
        tc::mma_ts(to, tp + ks * 8, vb + static_cast<uint64_t>((ks * 16 * 128) >> 4), kIdPV, j > 0 || ks > 0);
      tc::commit(smem_u32(&o_bar[t]));
      if (j == nchunks - 1) tc::commit(smem_u32(&o_last[t]));
      return true;
    };
    bool ok = nchunks > 0 && warp_wait(&q_full, 0, &abort_flag) && warp_wait(&kfull[0], 0, &abort_flag);
    tc::fence_after();
    if (ok) {
      issue_s(0, 0);
      issue_s(1, 0);
      if constexpr (!F8) tc::commit(smem_u32(&kempty[0]));  // K of stage 0 is read once these finish
    }
    for (int j = 0; ok && j < nchunks; ++j) {
      if (j + 1 < nchunks) {
        if (!warp_wait(&kfull[(j + 1) % S], ((j + 1) / S) & 1, &abort_flag)) break;
        tc::fence_after();
        issue_s(0, j + 1);
        issue_s(1, j + 1);
        if constexpr (!F8) tc::commit(smem_u32(&kempty[(j + 1) % S]));
      }
      if constexpr (!F8) {
        if (!warp_wait(&vready[j % S], (j / S) & 1, &abort_flag)) break;
        tc::fence_after();
      }
      ok = issue_pv(0, j) && issue_pv(1, j);
      if (ok) tc::commit(smem_u32(F8 ? &kempty[j % S] : &vempty[j % S]));
    }
    if (nchunks > 0) {
      tc::commit(smem_u32(&drain));  // every MMA issued has finished before TMEM is released
      mbar_wait(&drain, 0);
    }
    __syncwarp();
  } else if (warp < 8 && (warp & 3) < na) {
    // ---- softmax of half t: thread = row ----
    const int t = warp >> 2, r = tid & 127;
    const bool valid = r < rows;
    const int32_t pos = valid ? pos0 + (r >> a.gshift) : pos0;
    const int32_t lo = max(kbeg, pos - a.window + 1), hi = min(kend - 1, pos);  // the keys the row sees here
    {
      // q: each warpgroup half of the row's 16-byte pieces
      constexpr int NP = D / 16;
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (valid ? out_row(r) : 0) * D) + t * NP;
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
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full);
    }
    const uint32_t trow = tmem + t * Cfg::kTileCols + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const bool capped = a.cap_log2 > 0.f;
    const float sl2 = capped ? 1.f : a.scale_log2;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nchunks; ++j) {
      const int sb = j & 1;
      if (!warp_wait(&s_full[t][sb], (j >> 1) & 1, &abort_flag)) {
        ok = false;
        break;
      }
      tc::fence_after();
      uint32_t sr[C];
      tc::ld32(trow + D + sb * C, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
      tc::ld32(trow + D + sb * C + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
      tc::wait_ld();
      const int32_t k0 = c_begin + j * CK + t * C;
      float x[C];
      if (capped) {
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = capped_score(__uint_as_float(sr[c]) * a.cap_arg, a.cap_log2);
      } else {
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = __uint_as_float(sr[c]);
      }
      if (!__all_sync(0xffffffffu, k0 >= lo && k0 + C - 1 <= hi)) {
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = k0 + c >= lo && k0 + c <= hi ? x[c] : -INFINITY;
      }
      float pm[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) pm[u] = -INFINITY;
#pragma unroll
      for (int c = 0; c < C / 2; ++c) pm[c & 3] = fmax3(pm[c & 3], x[2 * c], x[2 * c + 1]);
      const float mx = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])) * sl2;  // scale > 0 keeps the order
      float alpha = 1.f;
      bool resc = false;
      if (mx > m + 8.f) {
        alpha = fast_exp2(m - mx);
        l *= alpha;
        resc = m != -INFINITY;  // (O is 0 while m is -inf)
        m = mx;
      }
      uint32_t ph[C / 2];
      const float nm = m == -INFINITY ? 0.f : -m;
      const float2 sc2 = make_float2(sl2, sl2), nm2 = make_float2(nm, nm);
      float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < C / 2; ++c) {
        const float2 y = ffma2(make_float2(x[2 * c], x[2 * c + 1]), sc2, nm2);
        const float2 pp = make_float2(fast_exp2(y.x), fast_exp2(y.y));
        part[c & 1] = fadd2(part[c & 1], pp);
        ph[c] = pack_f16(pp.x, pp.y);  // weights <= 2^8
      }
      l += (part[0].x + part[0].y) + (part[1].x + part[1].y);
      __syncwarp();
      tc::st32(trow + D + sb * C, ph);
      if (__any_sync(0xffffffffu, resc)) {
        // O must hold P(j-1) V(j-1) before it is rescaled
        if (!warp_wait(&o_bar[t], (j - 1) & 1, &abort_flag)) {
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
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          }
          __syncwarp();
          tc::st32(trow + q * 32, o);
        }
      }
      __syncwarp();
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[t][sb]);
    }
    if (ok && nchunks > 0) ok = warp_wait(&o_last[t], 0, &abort_flag);
    // merge of the halves: half 1 leaves (m, l, o) in shared memory (every MMA
    // that reads it has completed once both halves' last P V have), half 0 folds
    // it into its own and stores the rows. A half that gave up joins the barriers.
    float* stg = reinterpret_cast<float*>(sgen + Cfg::kQBytes) + r * Cfg::kRowPitch;
    float* ml1 = reinterpret_cast<float*>(sgen + Cfg::kQBytes) + 128 * Cfg::kRowPitch + 2 * r;
    tc::fence_after();
    asm volatile("bar.sync 1, %0;" ::"r"(2 * na * 32) : "memory");
    if (t == 1) {
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        __syncwarp();
        if (ok && nchunks > 0) {
          tc::ld32(trow + q * 32, o);
          tc::wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<uint4*>(stg + q * 32 + 4 * e) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      }
      ml1[0] = m;
      ml1[1] = l;
    }
    asm volatile("bar.sync 1, %0;" ::"r"(2 * na * 32) : "memory");
    if (t == 0 && ok && !*static_cast<volatile int*>(&abort_flag)) {
      const float m1 = ml1[0], l1 = ml1[1], M = fmaxf(m, m1);
      float f0 = M == -INFINITY ? 0.f : exp2f(m - M), f1 = M == -INFINITY ? 0.f : exp2f(m1 - M);
      l = l * f0 + l1 * f1;
      const int64_t orow = valid ? out_row(r) : 0;
      if (ms.nparts > 1) {
        if (valid) *reinterpret_cast<float2*>(a.ws_ml + (orow * a.max_parts + p) * 2) = make_float2(M, l);
      } else {
        float lse;
        const float f = finish_row(a.sinks, (g << a.gshift) + (r & ((1 << a.gshift) - 1)), M, l, lse) * a.v_scale;
        f0 *= f;
        f1 *= f;
        if (valid && a.lse) a.lse[orow] = lse;
      }
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        __syncwarp();
        if (nchunks > 0) {
          tc::ld32(trow + q * 32, o);
          tc::wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float4* d = reinterpret_cast<float4*>(stg + q * 32 + 4 * e);
          const float4 y = *d;
          *d = make_float4(fmaf(y.x, f1, __uint_as_float(o[4 * e]) * f0), fmaf(y.y, f1, __uint_as_float(o[4 * e + 1]) * f0),
                           fmaf(y.z, f1, __uint_as_float(o[4 * e + 2]) * f0), fmaf(y.w, f1, __uint_as_float(o[4 * e + 3]) * f0));
        }
      }
      __syncwarp();
      // the warp's rows as whole lines: D / 4 lanes per row
      constexpr int LR = D / 4, RW = 32 / LR;
      const float* src = reinterpret_cast<const float*>(sgen + Cfg::kQBytes);
      for (int i = 0; i < 32; i += RW) {
        const int rr = warp * 32 + i + lane / LR, d = (lane % LR) * 4;
        if (rr >= rows) continue;
        const float4 y = *reinterpret_cast<const float4*>(src + rr * Cfg::kRowPitch + d);
        const int64_t orr = out_row(rr);
        if (ms.nparts > 1) {
          *reinterpret_cast<float4*>(a.ws_o + (orr * a.max_parts + p) * D + d) = y;
        } else {
          const __nv_bfloat162 y0 = __floats2bfloat162_rn(y.x, y.y), y1 = __floats2bfloat162_rn(y.z, y.w);
          *reinterpret_cast<uint2*>(a.out + orr * D + d) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
        }
      }
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
