// Causal attention of whole prompts or prompt chunks over the paged cache with a
// sliding window, capped scores, sinks and the log-sum-exp of every row, on
// tcgen05.mma with the accumulators in tensor memory (the rule: score_rule.cuh).
//
// P2 = "PagedAttention：操作系统级 KV 缓存虚拟内存管理", §3.2.1 and §1.1.
//
// Tiles and operands are those of prefill_tc_kernel: a query tile is 128 rows (row
// r = token r / G, query head r % G, so the G heads of a kv head read every K/V
// tile once), two tiles of a sequence share a CTA's key stream of 64-key stages,
// P and V enter their product as f16. What differs:
//   * A CTA (kv head, pair of tiles) streams the keys its rows see, from the
//     first key of its first row's window on; each tile joins the stream at the
//     chunk of its own window and leaves it at its last key. Blocks wholly before
//     the window are not read; V rows outside [klo, kend) are written as zeros. A
//     row may see nothing in its tile's first chunks: weights 0.
//   * An MMA warp for each tile: a warp's waits and issues are the longest chain
//     of a chunk, and one's waits pass while the other's MMAs run. No tcgen05
//     fence after waits for what the TMA or the converter wrote (K, V, q): only
//     P, which other threads store by tcgen05.st, needs one.
//   * The producers read block ids one chunk ahead without divisions (a window of
//     ids shared by shuffles and block numbers by division take 1500 cycles of a
//     64-key chunk's 2000).
//   * O goes out as bf16, half as wide, through shared memory for every tile.
// Grid (kv heads, sequences, pairs), the last (longest) pair first. One CTA per
// SM that walks the pairs, the key ring running on from one to the next, was
// slower (window of 1024: 340 us where this form took 297; why was not found).
//
// Measured (launches back to back in a graph): two prompts of 3001 and 4096 tokens, 64/8
// heads, window 1024: 281 us over bf16, 725 TFLOP/s, 297 over e4m3, 310 over int8; eight
// of 700..2048, 32/32 heads, cap 50: 252 us, 567 TFLOP/s; with an L2 flush before each
// launch 303 and 264 us. Bound by a CTA's ends (5 us) and the chain of a chunk (1.1 us),
// not by a unit's rate. A chunk behind a long context has few CTAs, each of which walks
// all its keys: 17 to 256 tokens of 64/8 heads behind 8192 keys 146 to 150 us, behind
// 32768 549 to 567.
//
// Warps: 0-3 and 4-7 softmax of tile t (thread = row = TMEM lane), 8 producer
// (bf16: K; 8-bit: K and V codes), 9 and 10 MMA of tile 0 and 1, 11-14 converter,
// 15 V producer (bf16).
#pragma once

#include "prefill_tc.cuh"
#include "score_rule.cuh"

namespace pa {

struct WindowArgs {
  const __nv_bfloat16* q;  // [num_tokens][hq][D]
  const int32_t* cu_q;     // [num_seqs + 1]
  const int32_t* tables;   // [num_seqs][max_blocks]
  const int32_t* lens;     // [num_seqs], with the new tokens
  const float* sinks;      // [hq] or null
  __nv_bfloat16* out;      // [num_tokens][hq][D]
  float* lse;              // [num_tokens][hq] or null
  int64_t num_blocks;
  int32_t num_tokens, max_q, hq, hkv, bs, max_blocks, max_ctx;
  int32_t gshift, bshift;  // log2 of hq / hkv and of block_size
  int32_t window;          // >= 1; max_ctx or more: every earlier key
  ScoreScale score;
  float v_scale;
};

// A wait for a phase that is mostly complete or nearly: polls before it reads the
// clock that bounds the wait.
__device__ __forceinline__ bool warp_wait_soon(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return warp_wait(bar, parity, abort_flag);
}

template <int D, int CF>
struct WindowCfg {
  static constexpr bool F8 = CF != 0;
  static constexpr int kChunk = 64;                        // keys per stage
  static constexpr int kCols = D / 64;                     // 128-byte box columns of a 16-bit row
  static constexpr int kColBytes = kChunk * 128;
  static constexpr int kTileBytes = kCols * kColBytes;     // K (or V) of one stage
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = F8 ? 3 : 4;
  static constexpr int kCodeTileBytes = kChunk * D;
  static constexpr int kCodeStageBytes = 2 * kCodeTileBytes;
  static constexpr int kCodeStages = F8 ? 2 : 0;
  static constexpr int kQColBytes = 128 * 128;
  static constexpr int kQTileBytes = kCols * kQColBytes;
  static constexpr int kSmemBytes = 1024 + 2 * kQTileBytes + kStages * kStageBytes + kCodeStages * kCodeStageBytes;
  static constexpr int kProducerWarp = 8, kMmaWarp = 9, kConvWarp0 = 11, kConvWarps = 4, kVProducerWarp = 15;
  static constexpr int kThreads = 32 * (F8 ? 15 : 16);
  static constexpr uint32_t kTileCols = D + 2 * kChunk;    // TMEM of a tile: O, then two S/P buffers
  static_assert(kSmemBytes <= 226 * 1024, "shared memory");
};

template <int D, int CF, bool CAPPED>
__global__ void __launch_bounds__(WindowCfg<D, CF>::kThreads, 1)
    prefill_window_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                          const __grid_constant__ CUtensorMap tmq, const WindowArgs a) {
  using Cfg = WindowCfg<D, CF>;
  constexpr bool F8 = Cfg::F8;
  constexpr int S = Cfg::kStages, C = Cfg::kChunk, CS = F8 ? Cfg::kCodeStages : 1;
  // A K stage is released by the softmax warps, which see S done, or with capped
  // scores, where they have the most to do, by a commit of the MMA warps (a commit
  // waits behind the MMAs in the issue queue: back to back, by the softmax warps and by
  // a commit, window of 1024 288 and 297 us, capped 247 and 242, with weights not yet
  // scaled)
  constexpr bool kSoftmaxFreesK = !CAPPED;

  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t kfull[S], kempty[S];             // 16-bit stages (bf16: their K)
  __shared__ uint64_t vfull[S], vempty[S], vready[S];  // bf16: V of a stage, and V rewritten as f16
  __shared__ uint64_t cfull[CS], cempty[CS];           // 8-bit: code staging ring
  __shared__ uint64_t s_full[2][2], p_full[2][2];
  // per tile: q in place; its last P V but one, its last P V done
  __shared__ uint64_t q_full[2], o_prev[2], o_last[2], drain[2];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw);
  const uint32_t kv0 = sbase + 2 * Cfg::kQTileBytes;
  const uint32_t cs0 = kv0 + S * Cfg::kStageBytes;

  const int g = blockIdx.x, s = blockIdx.y;
  const int pair = gridDim.z - 1 - static_cast<int>(blockIdx.z);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t q0 = __ldg(a.cu_q + s);
  int32_t n = __ldg(a.cu_q + s + 1) - q0;
  int32_t L = __ldg(a.lens + s);
  const bool report = tid == 0 && g == 0 && pair == 0;
  if (q0 < 0 || n < 0 || n > a.max_q || q0 > a.num_tokens - n) {  // left out
    if (report) record_error(PA_ERR_DEVICE_BOUNDS, n);
    n = 0;
  }
  if (L < 0 || L > a.max_ctx || n > L) {
    if (report) record_error(PA_ERR_DEVICE_BOUNDS, L);
    L = L < 0 ? 0 : min(L, a.max_ctx);
    n = min(n, L);
  }
  const int32_t base = L - n;                  // position of the sequence's first new token
  const int32_t tt = 128 >> a.gshift;          // tokens of a tile
  const int32_t tok0 = 2 * pair * tt;
  if (tok0 >= n) return;
  // the key stream from the first chunk any row sees; tile t takes its chunks jb .. je - 1 (none: jb = je)
  const int32_t klo = max(0, base + tok0 - a.window + 1), first = klo & ~(C - 1);
  int32_t kend = 0, chunks = 0, jb[2], je[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int32_t tok = tok0 + t * tt;
    jb[t] = je[t] = 0;
    if (tok < n) {
      kend = base + min(tok + tt, n);
      jb[t] = (max(0, base + tok - a.window + 1) - first) / C;
      je[t] = chunks = (kend - first + C - 1) / C;
    }
  }
  // q of a tile arrives by TMA where its rows all lie in the sequence (bf16
  // cache); otherwise the softmax warps write it row by row
  auto q_by_tma = [&](int t) { return !F8 && tok0 + (t + 1) * tt <= n; };

  if (tid == 0) {
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
    prefetch_tmap(&tmq);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t][0], 1);
      mbar_init(&s_full[t][1], 1);
      mbar_init(&p_full[t][0], 4);
      mbar_init(&p_full[t][1], 4);
      mbar_init(&q_full[t], q_by_tma(t) ? 1 : 4);
      mbar_init(&o_prev[t], 1);
      mbar_init(&o_last[t], 1);
      mbar_init(&drain[t], 1);
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
      mbar_init(&kfull[i], F8 ? Cfg::kConvWarps : 1);
      mbar_init(&kempty[i], 2);  // an arrival for each tile
      mbar_init(&vfull[i], 1);
      mbar_init(&vempty[i], 2);
      mbar_init(&vready[i], Cfg::kConvWarps);
    }
#pragma unroll
    for (int i = 0; i < CS; ++i) {
      mbar_init(&cfull[i], 1);
      mbar_init(&cempty[i], Cfg::kConvWarps);
    }
    abort_flag = 0;
    fence_mbar_init();
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if (q_by_tma(t)) {
        mbar_arrive_expect_tx(&q_full[t], Cfg::kQTileBytes);
        const uint64_t pol = l2_evict_first_policy();
#pragma unroll
        for (int hf = 0; hf < Cfg::kCols; ++hf)
          tma_load_3d(sbase + t * Cfg::kQTileBytes + hf * Cfg::kQColBytes, &tmq, hf * 64, g << a.gshift,
                      q0 + tok0 + t * tt, &q_full[t], pol);
      }
  }
  // the producers' block ids: lane i holds that of the chunk's block i, read one
  // chunk ahead
  const int32_t* blocks = a.tables + static_cast<int64_t>(s) * a.max_blocks;
  const int32_t blocks_end = min(a.max_blocks, (kend + a.bs - 1) >> a.bshift);
  auto block_at = [&](int32_t key) {
    const int32_t i = (key >> a.bshift) + lane;
    return lane < (C >> a.bshift) && i < blocks_end ? __ldg(blocks + i) : -1;
  };
  int32_t blk_next = -1;
  if (warp == Cfg::kProducerWarp || (!F8 && warp == Cfg::kVProducerWarp)) blk_next = block_at(first);
  __syncwarp();
  if (warp == Cfg::kMmaWarp) {
    tc::alloc(smem_u32(&tmem_base_sh), 512);
    tc::relinquish();
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_base_sh;

  if (warp == Cfg::kProducerWarp || (!F8 && warp == Cfg::kVProducerWarp)) {
    // ---- producers: every chunk's blocks that hold a key in [klo, kend) ----
    const bool is_v = !F8 && warp == Cfg::kVProducerWarp;
    constexpr int R = F8 ? CS : S;
    uint64_t* full = F8 ? cfull : (is_v ? vfull : kfull);
    uint64_t* empty = F8 ? cempty : (is_v ? vempty : kempty);
    const CUtensorMap* map = is_v ? &tmv : &tmk;
    const uint32_t box_bytes = static_cast<uint32_t>(a.bs) * (F8 ? D : 128);  // of one box column
    const uint64_t pol = l2_evict_last_policy();  // later pairs of this sequence read the same keys
    int i = 0;
    for (; i < chunks; ++i) {
      const int st = i % R;
      if (i >= R && !warp_wait(&empty[st], ((i / R) - 1) & 1, &abort_flag)) break;
      const int32_t key = first + i * C;
      const int32_t blk = blk_next;
      blk_next = block_at(key + C);
      bool in = false;
      if (lane < (C >> a.bshift) && (key >> a.bshift) + lane < blocks_end && key + ((lane + 1) << a.bshift) > klo) {
        in = blk >= 0 && blk < a.num_blocks;
        if (!in && !is_v) record_error(PA_ERR_DEVICE_BOUNDS, blk);
      }
      const int cnt = __popc(__ballot_sync(0xffffffffu, in));
      if (lane == 0) mbar_arrive_expect_tx(&full[st], (F8 ? 2u : Cfg::kCols) * cnt * box_bytes);
      __syncwarp();
      if (in) {
        const int32_t y = (blk * a.hkv + g) * a.bs;
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
    if (abort_flag && lane == 0)  // copies already started land before exit
      for (int j = (i > R ? i - R : 0); j < i; ++j) mbar_wait(&full[j % R], (j / R) & 1);
  } else if (warp >= Cfg::kConvWarp0 && warp < Cfg::kConvWarp0 + Cfg::kConvWarps) {
    // ---- converter: thread = (row of the chunk, half of its dims); rows outside
    // [klo, kend) become zeros ----
    const int ct = tid - 32 * Cfg::kConvWarp0;
    const int row = ct >> 1, half = ct & 1;
    for (int i = 0; i < chunks; ++i) {
      const int st = i % S;
      const int32_t key = first + i * C + row;
      const bool live = key >= klo && key < kend;
      uint8_t* stage = sgen + 2 * Cfg::kQTileBytes + st * Cfg::kStageBytes;
      if constexpr (F8) {
        const int cst = i % CS;
        if (!warp_wait(&cfull[cst], (i / CS) & 1, &abort_flag)) break;
        if (i >= S && !warp_wait(&kempty[st], ((i / S) - 1) & 1, &abort_flag)) break;
        const uint8_t* src = sgen + (cs0 - sbase) + cst * Cfg::kCodeStageBytes;
        widen_row_half<D, CF, Cfg::kColBytes>(src, stage, row, half, live);
        widen_row_half<D, CF, Cfg::kColBytes>(src + Cfg::kCodeTileBytes, stage + Cfg::kTileBytes, row, half, live);
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&kfull[st]);
          mbar_arrive(&cempty[cst]);
        }
      } else {
        if (!warp_wait(&vfull[st], (i / S) & 1, &abort_flag)) break;
        v_to_f16_inplace<D, Cfg::kColBytes>(stage + Cfg::kTileBytes, row, half, live);
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&vready[st]);
      }
    }
  } else if (warp == Cfg::kMmaWarp || warp == Cfg::kMmaWarp + 1) {
    // ---- MMA issuer of tile t: S(j + 1), then O += P(j) V(j); the whole warp
    // walks the schedule, one elected lane issues ----
    const int t = warp - Cfg::kMmaWarp;
    constexpr uint32_t kIdS = F8 ? tc::idesc_f16(128, C, false) : tc::idesc_bf16(128, C, false);
    constexpr uint32_t kIdPV = tc::idesc_f16(128, D, true);
    const uint32_t qs = sbase + t * Cfg::kQTileBytes;
    const uint64_t qdesc = tc::smem_desc(qs, 16, 1024);
    const uint64_t kdesc0 = tc::smem_desc(kv0, 16, 1024);
    const uint64_t vdesc0 = tc::smem_desc(kv0 + Cfg::kTileBytes, Cfg::kCols > 1 ? Cfg::kColBytes : 1024, 1024);
    const uint32_t to = tmem + t * Cfg::kTileCols;
    // S of the stream's chunk j (jl: the tile's own count, for its buffers)
    auto issue_s = [&](int j, int jl) {
      const uint64_t kb = kdesc0 + static_cast<uint64_t>(((j % S) * Cfg::kStageBytes) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t offq = static_cast<uint32_t>((kk >> 2) * Cfg::kQColBytes + (kk & 3) * 32) >> 4;
        const uint32_t offk = static_cast<uint32_t>((kk >> 2) * Cfg::kColBytes + (kk & 3) * 32) >> 4;
        tc::mma_ss(to + D + (jl & 1) * C, qdesc + offq, kb + offk, kIdS, kk > 0);
      }
      tc::commit(smem_u32(&s_full[t][jl & 1]));
    };
    bool ok = true;
    for (int j = -1; ok && j < chunks; ++j) {
      // S one chunk ahead
      if (j + 1 < chunks) {
        const int jn = j + 1;
        // (a stage that the tile does not use is waited for and released too: a
        // release ahead of its stage would count for the one before)
        if (!(ok = warp_wait_soon(&kfull[jn % S], (jn / S) & 1, &abort_flag))) break;
        if (jn >= jb[t] && jn < je[t]) {
          if (jn == jb[t] && !(ok = warp_wait(&q_full[t], 0, &abort_flag))) break;
          issue_s(jn, jn - jb[t]);
          if (!F8 && !kSoftmaxFreesK) tc::commit(smem_u32(&kempty[jn % S]));
        } else if (!F8 && lane == 0) {
          mbar_arrive(&kempty[jn % S]);
        }
      }
      if (j < 0) continue;
      if constexpr (!F8)
        if (!(ok = warp_wait_soon(&vready[j % S], (j / S) & 1, &abort_flag))) break;
      if (j >= jb[t] && j < je[t]) {
        const int jl = j - jb[t], sb = jl & 1;
        if (!(ok = warp_wait_soon(&p_full[t][sb], (jl >> 1) & 1, &abort_flag))) break;
        tc::fence_after();
        const uint64_t vb = vdesc0 + static_cast<uint64_t>(((j % S) * Cfg::kStageBytes) >> 4);
#pragma unroll
        for (int ks = 0; ks < C / 16; ++ks)
          tc::mma_ts(to, to + D + sb * C + ks * 8, vb + static_cast<uint64_t>((ks * 16 * 128) >> 4), kIdPV,
                     jl > 0 || ks > 0);
        if (j + 2 == je[t]) tc::commit(smem_u32(&o_prev[t]));
        if (j + 1 == je[t]) tc::commit(smem_u32(&o_last[t]));
      }
      tc::commit(smem_u32(F8 ? &kempty[j % S] : &vempty[j % S]));
    }
    tc::commit(smem_u32(&drain[t]));  // every MMA issued has finished before TMEM is released
    mbar_wait(&drain[t], 0);
    __syncwarp();
  } else if (warp < 8) {
    // ---- softmax of tile t: thread = row = TMEM lane ----
    const int t = warp >> 2, r = tid & 127, h = r & ((1 << a.gshift) - 1);
    const uint32_t trow = tmem + t * Cfg::kTileCols + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    uint8_t* stg = sgen + t * Cfg::kQTileBytes + (warp & 3) * 32 * 128;  // (on the way out: q is done with)
    const CapPoly poly(CAPPED ? a.score.cap_log2 : 0.f);
    const int nch = je[t] - jb[t];
    if (nch > 0) {
      const int32_t tokt = tok0 + t * tt, tok = tokt + (r >> a.gshift);
      const bool valid = tok < n;
      const int32_t pos = base + (valid ? tok : n - 1);  // the last key the row sees, and the first
      const int32_t lo = pos - a.window + 1;
      const int64_t orow = (static_cast<int64_t>(q0) + (valid ? tok : 0)) * a.hq + (g << a.gshift) + h;
      if (!q_by_tma(t)) {
        const uint4* src = reinterpret_cast<const uint4*>(a.q + orow * D);
        uint8_t* qdst = sgen + t * Cfg::kQTileBytes;
        uint4 qv[D / 8];
#pragma unroll
        for (int c16 = 0; c16 < D / 8; ++c16) qv[c16] = valid ? __ldg(src + c16) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int c16 = 0; c16 < D / 8; ++c16) {
          uint4 v = qv[c16];
          if constexpr (F8)
            v = make_uint4(pack_f16(bf16lo(v.x), bf16hi(v.x)), pack_f16(bf16lo(v.y), bf16hi(v.y)),
                           pack_f16(bf16lo(v.z), bf16hi(v.z)), pack_f16(bf16lo(v.w), bf16hi(v.w)));
          const int hf = c16 >> 3, cc = c16 & 7;
          *reinterpret_cast<uint4*>(qdst + hf * Cfg::kQColBytes + r * 128 + ((cc ^ (r & 7)) << 4)) = v;
        }
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[t]);
      }
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < nch; ++j) {
        const int sb = j & 1;
        if (!warp_wait(&s_full[t][sb], (j >> 1) & 1, &abort_flag)) {
          ok = false;
          break;
        }
        if (!F8 && kSoftmaxFreesK && (warp & 3) == 0 && lane == 0) mbar_arrive(&kempty[(jb[t] + j) % S]);
        __syncwarp();
        tc::fence_after();
        uint32_t sr[C];
        tc::ld32(trow + D + sb * C, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tc::ld32(trow + D + sb * C + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        tc::wait_ld();
        const int32_t k0 = first + (jb[t] + j) * C;
        float x[C], amax = 0.f;
        // warp-uniform choice: tcgen05.ld/st below need the whole warp converged
        if (__all_sync(0xffffffffu, k0 + C - 1 <= pos && k0 >= lo)) {
#pragma unroll
          for (int c = 0; c < C; ++c) x[c] = __uint_as_float(sr[c]);
          if constexpr (CAPPED) amax = row_amax(x);
        } else {
#pragma unroll
          for (int c = 0; c < C; ++c) x[c] = __uint_as_float(sr[c]);
          amax = masked_amax(x, lo - k0, pos - k0);
        }
        float alpha;
        bool resc;
        uint32_t ph[C / 2];
        row_weights<CAPPED>(a.score, x, amax, poly, m, l, alpha, resc, ph);
        __syncwarp();
        tc::st32(trow + D + sb * C, ph);
        if (__any_sync(0xffffffffu, resc)) {
          // O must hold P(j-1) V(j-1) before it is rescaled: S(j+1) was issued
          // behind it, and at the last chunk it has a barrier of its own
          if (!(j + 1 < nch ? warp_wait(&s_full[t][sb ^ 1], ((j + 1) >> 1) & 1, &abort_flag)
                            : warp_wait(&o_prev[t], 0, &abort_flag))) {
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
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t][sb]);
      }
      if (ok && warp_wait(&o_last[t], 0, &abort_flag)) {
      tc::fence_after();
      float lse;
      const float inv = finish_row(a.sinks, (g << a.gshift) + h, final_ref(m, l), l, 1.f / kWeightF16, lse);
      const float vs = F8 ? a.v_scale : 1.f;
      uint32_t w[D / 2];  // O as bf16
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        tc::ld32(trow + q * 32, o);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const __nv_bfloat162 b =
              __floats2bfloat162_rn(__uint_as_float(o[2 * i]) * inv * vs, __uint_as_float(o[2 * i + 1]) * inv * vs);
          w[q * 16 + i] = *reinterpret_cast<const uint32_t*>(&b);
        }
      }
      if (valid && a.lse) a.lse[orow] = lse;
      // out through shared memory, 64 columns (128 bytes) of the warp's rows at a
      // time: each thread writes its row's pieces (rotated by row: no bank
      // conflicts), then the warp stores whole 128-byte segments
      const int pc = lane & 7;
      const int64_t col = static_cast<int64_t>(g << a.gshift) * D + pc * 8;
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(stg + lane * 128 + ((i ^ (lane & 7)) << 4)) =
              make_uint4(w[q * 32 + 4 * i], w[q * 32 + 4 * i + 1], w[q * 32 + 4 * i + 2], w[q * 32 + 4 * i + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rw = 4 * i + (lane >> 3), rr = (warp & 3) * 32 + rw;
          const int32_t tk = tokt + (rr >> a.gshift);
          if (tk < n)
            *reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(q0 + tk) * a.hq * D + col +
                                      (rr & ((1 << a.gshift) - 1)) * D + q * 64) =
                *reinterpret_cast<const uint4*>(stg + rw * 128 + ((pc ^ (rw & 7)) << 4));
        }
      }
      }
    }
    tc::fence_before();
  }
  __syncthreads();
  if (warp == Cfg::kMmaWarp) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

}  // namespace pa
