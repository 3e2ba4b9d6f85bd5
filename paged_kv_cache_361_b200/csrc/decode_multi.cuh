// Decode attention of one or a few new tokens per sequence over the paged
// cache: with a sliding window, a cap on the scores, per-head sinks, and the
// log-sum-exp of every row.
//
// P2 = "PagedAttention：操作系统级 KV 缓存虚拟内存管理", §1.1 and §4.1 (the softmax
// accumulated tile by tile). For the new token at position p and query head h:
//   x_j = scale q.k_j, or cap tanh(scale q.k_j / cap);  w_j = exp(x_j)
//   for the keys p - window < j <= p
//   out = sum_j w_j v_j / (sum_j w_j + exp(sink_h)),  lse = log(that denominator)
// kept as a running maximum m, sum l and o in base 2, and merged over warps and
// partitions by M = max m_i, l = sum l_i 2^(m_i - M), o = sum o_i 2^(m_i - M).
//
// Bound by HBM: a K/V byte feeds G n multiply-adds (G query heads of a kv head,
// n new tokens), so the reads take longer than the products.
// Rows are (token, head) pairs of one (sequence, kv head): a CTA takes all of
// them, up to 16 (NG groups of 8, the MMA's N; more rows: decode_multi_tc.cuh),
// and a partition of the visible keys, so every K/V byte is read once. Its
// products are those of the single-token decode with the tokens as the MMA's M
// (S^T = K q^T, O^T += V^T P^T), with each K and V fragment used for all NG
// groups. The keys the rows see start at kbeg, inside a 64-key chunk and inside a block:
// blocks wholly before it are not read, scores outside a row's window are
// replaced by -inf, V rows outside [kbeg, kend) are zeroed in registers (a
// freed block may hold anything, NaN too).
// A split sequence's partials are merged by decode_multi_merge_kernel, launched
// as the programmatic dependent of this grid.
#pragma once

#include "decode_f8.cuh"
#include "decode_mma.cuh"
#include "score_rule.cuh"

namespace pa {

struct MultiArgs {
  const __nv_bfloat16* q;  // [num_tokens][hq][D]
  const int32_t* cu_q;     // [num_seqs + 1], or null: row s is sequence s's one token
  const int32_t* tables;   // [num_seqs][max_blocks]
  const int32_t* lens;     // [num_seqs], with the new tokens
  const float* sinks;      // [hq] or null
  __nv_bfloat16* out;      // [num_tokens][hq][D]
  float* lse;              // [num_tokens][hq] or null
  float* ws_ml;            // [num_tokens][hq][max_parts][2]
  float* ws_o;             // [num_tokens][hq][max_parts][D]
  int64_t num_blocks;
  int32_t num_seqs, num_tokens, max_q, hq, hkv, bs, max_blocks, max_ctx;
  int32_t gshift;          // log2 of hq / hkv
  int32_t window;          // >= 1; max_ctx or more: every earlier key
  int32_t part_tokens;     // a multiple of 64, INT32_MAX: one partition
  int32_t max_parts;
  float scale_log2;        // scale * log2 e (times the K scale of an 8-bit cache)
  float cap_log2;          // softcap * log2 e, 0: none
  float cap_arg;           // with a cap: 2 log2 e * scale / softcap (times the K scale)
  float v_scale;
};

// The new rows, lengths and key range of a sequence.
struct MultiSeq {
  int32_t q0, n, L;
  int32_t first;   // 64-aligned start of the sequence's partitions
  int32_t nparts;
};

__device__ __forceinline__ MultiSeq load_multi_seq(const MultiArgs& a, int s, bool report) {
  MultiSeq m;
  m.q0 = s;
  m.n = 1;
  if (a.cu_q) {
    m.q0 = __ldg(a.cu_q + s);
    m.n = __ldg(a.cu_q + s + 1) - m.q0;
    if (m.q0 < 0 || m.q0 > a.num_tokens || m.n < 0 || m.n > a.max_q || m.n > a.num_tokens - m.q0) {
      if (report) record_error(PA_ERR_DEVICE_BOUNDS, m.n);
      m.n = 0;
    }
  }
  m.L = __ldg(a.lens + s);
  if (m.L < 0 || m.L > a.max_ctx || (a.cu_q && m.n > m.L)) {
    if (report) record_error(PA_ERR_DEVICE_BOUNDS, m.L);
    m.L = m.L < 0 ? 0 : min(m.L, a.max_ctx);
  }
  m.first = max(0, m.L - m.n - a.window + 1) & ~63;
  const int32_t span = m.L - m.first;
  m.nparts = span > a.part_tokens ? (span + a.part_tokens - 1) / a.part_tokens : 1;
  return m;
}

template <int D, int NG, int CF>
struct MultiCfg {
  static constexpr int kConsumerWarps = 4;
  static constexpr int kThreads = 32 * (kConsumerWarps + 1);
  static constexpr int kChunk = 64;
  static constexpr int kRows = 8 * NG;
  static constexpr int kEl = CF != 0 ? 1 : 2;
  static constexpr int kTileBytes = kChunk * D * kEl;  // K (or V) of one stage
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kMinCtas = 3;
  // the ring of a CTA: its share of the SM's shared memory, and the merge of the warps has to fit
  static constexpr int kStages = 64 * 1024 / kStageBytes;
  static constexpr int kRowPitch = D + 4;  // floats of a row in the merge: lanes' rows in different banks
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes;
  static_assert(kConsumerWarps * kRows * (kRowPitch + 2) * 4 <= kStages * kStageBytes, "merge buffer");
};

// One group's scores of a warp's 16 keys (x: keys r, r + 8 of rows 2c, 2c + 1,
// base 2, -inf where unseen) folded into its running state; leaves the weights
// in x. The reference maximum moves only when a score exceeds it by 8, so
// weights stay <= 2^8 and o is rarely rescaled.
template <int DT>
__device__ __forceinline__ void multi_softmax(float (&x)[4], float (&m_run)[2], float (&l_run)[2], float (&o)[DT][4]) {
  float mloc[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float v = fmaxf(x[j], x[2 + j]);
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
    mloc[j] = v;
  }
  const bool move[2] = {mloc[0] > m_run[0] + 8.f, mloc[1] > m_run[1] + 8.f};
  if (__any_sync(0xffffffffu, move[0] || move[1])) {
    float alpha[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      alpha[j] = move[j] ? fast_exp2(m_run[j] - mloc[j]) : 1.f;  // 0 from -inf
      if (move[j]) m_run[j] = mloc[j];
      l_run[j] *= alpha[j];
    }
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][e] *= alpha[e & 1];
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float ref = m_run[j] == -INFINITY ? 0.f : m_run[j];  // a row that has seen nothing: weights 0
    x[j] = fast_exp2(x[j] - ref);
    x[2 + j] = fast_exp2(x[2 + j] - ref);
    l_run[j] += x[j] + x[2 + j];
  }
}

template <int D, int NG, int CF>
__global__ void __launch_bounds__(MultiCfg<D, NG, CF>::kThreads, MultiCfg<D, NG, CF>::kMinCtas)
    decode_multi_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                        const MultiArgs a) {
  using Cfg = MultiCfg<D, NG, CF>;
  constexpr int NW = Cfg::kConsumerWarps, C = Cfg::kChunk, S = Cfg::kStages, KS = D / 16;

  extern __shared__ uint8_t smem_raw[];
  __shared__ PipeSmem<S> ps;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - smem_u32(smem_raw));

  const int g = blockIdx.x, s = blockIdx.y;
  const int p = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;
  const MultiSeq ms = load_multi_seq(a, s, g == 0 && p == 0 && tid == 0);
  const int rows = ms.n << a.gshift;
  if (rows <= 0 || p >= ms.nparts) return;
  // keys that some row sees, within the partition
  const int32_t pos0 = ms.L - ms.n;  // position of the sequence's first new token
  const int32_t pos_lo = pos0, pos_hi = pos0 + ms.n - 1;
  const int32_t t0 = ms.nparts > 1 ? ms.first + p * a.part_tokens : 0;
  const int32_t t1 = ms.nparts > 1 && p < ms.nparts - 1 ? t0 + a.part_tokens : ms.L;
  const int32_t kbeg = max(t0, max(0, pos_lo - a.window + 1));
  const int32_t kend = t1;
  const int32_t c_begin = kbeg & ~(C - 1);
  const int nchunks = kend > kbeg ? (kend - c_begin + C - 1) / C : 0;

  TableAhead ta;
  if (warp == NW)
    ta.init(a.tables + static_cast<int64_t>(s) * a.max_blocks, c_begin / a.bs,
            min(a.max_blocks, (kend + a.bs - 1) / a.bs), lane);
  if (tid == 0) {
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
    pipe_init<S>(ps, NW);
  }
  // q as the B fragments of S^T (column r of group gi = row 8 gi + r, zeros
  // past the last): dims (2c, 2c + 1) and (+8) of a 16-dim step, or
  // over an 8-bit cache, as f16, dims (4c, 4c + 1) and (4c + 2, 4c + 3)
  auto q_frag = [&](int gi, int kk) -> uint2 {
    const int rho = 8 * gi + r;
    if (rho >= rows) return make_uint2(0u, 0u);
    const int64_t qrow = static_cast<int64_t>(ms.q0 + (rho >> a.gshift)) * a.hq + (g << a.gshift) +
                         (rho & ((1 << a.gshift) - 1));
    const uint32_t* w = reinterpret_cast<const uint32_t*>(a.q + qrow * D) + kk * 8;
    if constexpr (CF != 0) {
      const uint2 x = *reinterpret_cast<const uint2*>(w + 2 * c);
      return make_uint2(pack_f16(bf16lo(x.x), bf16hi(x.x)), pack_f16(bf16lo(x.y), bf16hi(x.y)));
    } else {
      return make_uint2(__ldg(w + c), __ldg(w + 4 + c));
    }
  };
  uint2 qr[NG][KS];
  if (warp < NW) {
#pragma unroll
    for (int gi = 0; gi < NG; ++gi)
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) qr[gi][kk] = q_frag(gi, kk);
  }
  __syncthreads();

  float o[NG][KS][4], m_run[NG][2], l_run[NG][2];
#pragma unroll
  for (int gi = 0; gi < NG; ++gi) {
    m_run[gi][0] = m_run[gi][1] = -INFINITY;
    l_run[gi][0] = l_run[gi][1] = 0.f;
#pragma unroll
    for (int t = 0; t < KS; ++t) o[gi][t][0] = o[gi][t][1] = o[gi][t][2] = o[gi][t][3] = 0.f;
  }

  if (warp == NW) {
    // ---- producer: the blocks of chunk i that hold a key in [kbeg, kend) ----
    const uint32_t box_bytes = static_cast<uint32_t>(a.bs) * D * Cfg::kEl;
    const uint64_t pol = kv_stream_policy();
    pipe_produce<S>(ps, nchunks, [&](int i, int st) {
      const int32_t c0 = c_begin + i * C;
      const int32_t nb = (min(C, kend - c0) + a.bs - 1) / a.bs;  // <= 8 (bs >= 8)
      const int32_t blk = ta.get(c0 / a.bs, nb, lane);
      bool ok = false;
      if (lane < nb && c0 + (lane + 1) * a.bs > kbeg) {
        ok = blk >= 0 && blk < a.num_blocks;
        if (!ok) record_error(PA_ERR_DEVICE_BOUNDS, blk);
      }
      const unsigned okmask = __ballot_sync(0xffffffffu, ok);
      if (lane == 0) mbar_arrive_expect_tx(&ps.full[st], 2u * __popc(okmask) * box_bytes);
      __syncwarp();
      if (ok) {
        const int32_t y = (blk * a.hkv + g) * a.bs;
        const uint32_t kdst = sbase + st * Cfg::kStageBytes + lane * box_bytes;
        if constexpr (CF != 0) {
          tma_load_2d(kdst, &tmk, 0, y, &ps.full[st], pol);
          tma_load_2d(kdst + Cfg::kTileBytes, &tmv, 0, y, &ps.full[st], pol);
        } else {
          tma_block<D>(kdst, &tmk, y, &ps.full[st], pol);
          tma_block<D>(kdst + Cfg::kTileBytes, &tmv, y, &ps.full[st], pol);
        }
      }
    });
  } else {
    // ---- consumers: warp w has keys [16w, 16w + 16) of every chunk ----
    // positions of this lane's rows 8 gi + 2c + j: the last key each sees
    int32_t pos[NG][2];
#pragma unroll
    for (int gi = 0; gi < NG; ++gi)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = 8 * gi + 2 * c + j;
        pos[gi][j] = row < rows ? pos0 + (row >> a.gshift) : -1;
      }
    const int mk = lane >> 3, ik = lane & 7;
    for (int i = 0; i < nchunks; ++i) {
      const int st = i % S;
      if (!pipe_wait(&ps.full[st], (i / S) & 1, &ps.abort_flag)) break;
      const int32_t key0 = c_begin + i * C + warp * 16;  // this warp's first key
      if (key0 + 16 > kbeg && key0 < kend) {             // warp-uniform
        const uint32_t kst = sbase + st * Cfg::kStageBytes, vst = kst + Cfg::kTileBytes;
        float x[NG][4];
        if constexpr (CF == 0) {
          // stage layout as in mma_chunk: block-major, 64-element halves, swizzled rows
          const int tokK = warp * 16 + (mk >> 1) * 8 + ik, dK = (mk & 1) * 8;
          const uint32_t hstride = static_cast<uint32_t>(a.bs) * 128u;
          const uint32_t kbase = kst + (tokK + (tokK & ~(a.bs - 1)) * (D / 64 - 1)) * 128;
          float s1[NG == 1 ? 4 : 1] = {};
#pragma unroll
          for (int gi = 0; gi < NG; ++gi) x[gi][0] = x[gi][1] = x[gi][2] = x[gi][3] = 0.f;
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
            const int d0 = kk * 16 + dK;
            uint32_t m0, m1, m2, m3;
            ldsm_x4(kbase + (d0 >> 6) * hstride + ((((d0 & 63) >> 3) ^ (tokK & 7)) << 4), m0, m1, m2, m3);
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
              const uint2 qq = qr[gi][kk];
              if constexpr (NG == 1)
                mma16x8(kk & 1 ? s1 : x[gi], m0, m2, m1, m3, qq.x, qq.y);  // two chains
              else
                mma16x8(x[gi], m0, m2, m1, m3, qq.x, qq.y);
            }
          }
          if constexpr (NG == 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[0][e] += s1[e];
        } else {
          uint32_t rb[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = warp * 16 + h * 8 + r;
            const uint32_t key = D == 128 ? static_cast<uint32_t>(row & 7) : static_cast<uint32_t>((row >> 1) & 3);
            rb[h] = (kst + static_cast<uint32_t>(row * D)) | (key << 4) | static_cast<uint32_t>(4 * c);
          }
          float s1[NG == 1 ? 4 : 1] = {};
#pragma unroll
          for (int gi = 0; gi < NG; ++gi) x[gi][0] = x[gi][1] = x[gi][2] = x[gi][3] = 0.f;
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
            uint32_t w0, w1;
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w0) : "r"(rb[0] ^ static_cast<uint32_t>(kk << 4)));
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w1) : "r"(rb[1] ^ static_cast<uint32_t>(kk << 4)));
            uint32_t k00, k01, k10, k11;
            widen4<CF>(w0, k00, k01);
            widen4<CF>(w1, k10, k11);
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
              const uint2 qq = qr[gi][kk];
              if constexpr (NG == 1)
                mma16x8_f16(kk & 1 ? s1 : x[gi], k00, k10, k01, k11, qq.x, qq.y);
              else
                mma16x8_f16(x[gi], k00, k10, k01, k11, qq.x, qq.y);
            }
          }
          if constexpr (NG == 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[0][e] += s1[e];
        }
        // base-2 scores; -inf outside a row's keys (every row sees all 16 keys
        // in most chunks). A key past kend is past its row's position
        // or in the next partition, one before kbeg before every window.
        if (a.cap_log2 > 0.f) {
#pragma unroll
          for (int gi = 0; gi < NG; ++gi)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[gi][e] = capped_score(x[gi][e] * a.cap_arg, a.cap_log2);
        } else {
#pragma unroll
          for (int gi = 0; gi < NG; ++gi)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[gi][e] *= a.scale_log2;
        }
        const bool inside = key0 >= kbeg && key0 + 16 <= kend;
        if (!inside || key0 + 15 > pos_lo || key0 <= pos_hi - a.window) {
#pragma unroll
          for (int gi = 0; gi < NG; ++gi)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int32_t key = key0 + r + (e >> 1) * 8, ps_ = pos[gi][e & 1];
              if (key < kbeg || key >= kend || key > ps_ || key <= ps_ - a.window) x[gi][e] = -INFINITY;
            }
        }
        // weights, and P^T as B fragments (K 16 keys x N 8 rows)
        uint32_t pb[NG][CF != 0 ? 2 : 4];
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
          multi_softmax<KS>(x[gi], m_run[gi], l_run[gi], o[gi]);
          if constexpr (CF != 0) {
            pb[gi][0] = movmatrix_t(pack_f16(x[gi][0], x[gi][1]));
            pb[gi][1] = movmatrix_t(pack_f16(x[gi][2], x[gi][3]));
          } else {
            uint32_t h01, l01, h23, l23;
            split_pair(x[gi][0], x[gi][1], h01, l01);
            split_pair(x[gi][2], x[gi][3], h23, l23);
            pb[gi][0] = movmatrix_t(h01);
            pb[gi][1] = movmatrix_t(h23);
            pb[gi][2] = movmatrix_t(l01);
            pb[gi][3] = movmatrix_t(l23);
          }
        }
        // V rows outside [kbeg, kend) as zeros: this lane's keys 2c, 2c + 1 (mlo) and + 8 (mhi)
        uint32_t mlo = 0xffffffffu, mhi = 0xffffffffu;
        if (!inside) {
          auto live = [&](int k) { return key0 + k >= kbeg && key0 + k < kend; };
          mlo = (live(2 * c) ? 0x0000ffffu : 0u) | (live(2 * c + 1) ? 0xffff0000u : 0u);
          mhi = (live(2 * c + 8) ? 0x0000ffffu : 0u) | (live(2 * c + 9) ? 0xffff0000u : 0u);
        }
        if constexpr (CF == 0) {
          const int tokV = warp * 16 + (mk & 1) * 8 + ik, dV = (mk >> 1) * 8;
          const uint32_t hstride = static_cast<uint32_t>(a.bs) * 128u;
          const uint32_t vbase = vst + (tokV + (tokV & ~(a.bs - 1)) * (D / 64 - 1)) * 128;
#pragma unroll
          for (int t = 0; t < KS; ++t) {
            const int d0 = t * 16 + dV;
            uint32_t v0, v1, v2, v3;
            ldsm_x4_t(vbase + (d0 >> 6) * hstride + ((((d0 & 63) >> 3) ^ (tokV & 7)) << 4), v0, v1, v2, v3);
            v0 &= mlo;
            v1 &= mhi;
            v2 &= mlo;
            v3 &= mhi;
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
              mma16x8(o[gi][t], v0, v2, v1, v3, pb[gi][0], pb[gi][1]);
              mma16x8(o[gi][t], v0, v2, v1, v3, pb[gi][2], pb[gi][3]);
            }
          }
        } else {
          constexpr int W = D == 128 ? 4 : 2;  // 32-bit words of V per key this thread reads
          const uint8_t* vt = sgen + (vst - sbase);
          const int col = f8_dim<D>(0, r), ta0 = warp * 16 + 2 * c, tb0 = ta0 + 8;
          const uint8_t* pa_ = vt + f8_off<D>(ta0, col);
          const uint8_t* pb_ = vt + f8_off<D>(ta0 + 1, col);
          const uint8_t* pc_ = vt + f8_off<D>(tb0, col);
          const uint8_t* pd_ = vt + f8_off<D>(tb0 + 1, col);
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const uint32_t xa = *reinterpret_cast<const uint32_t*>(pa_ + 4 * w);
            const uint32_t xb = *reinterpret_cast<const uint32_t*>(pb_ + 4 * w);
            const uint32_t xc = *reinterpret_cast<const uint32_t*>(pc_ + 4 * w);
            const uint32_t xd = *reinterpret_cast<const uint32_t*>(pd_ + 4 * w);
            uint32_t b[8];
            widen4<CF>(__byte_perm(xa, xb, 0x5140), b[0], b[1]);
            widen4<CF>(__byte_perm(xa, xb, 0x7362), b[2], b[3]);
            widen4<CF>(__byte_perm(xc, xd, 0x5140), b[4], b[5]);
            widen4<CF>(__byte_perm(xc, xd, 0x7362), b[6], b[7]);
            if (!inside) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                b[k] &= mlo;
                b[4 + k] &= mhi;
              }
            }
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
              mma16x8_f16(o[gi][2 * w], b[0], b[1], b[4], b[5], pb[gi][0], pb[gi][1]);
              mma16x8_f16(o[gi][2 * w + 1], b[2], b[3], b[6], b[7], pb[gi][0], pb[gi][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ps.empty[st]);
    }
#pragma unroll
    for (int gi = 0; gi < NG; ++gi) sum_l(l_run[gi]);
  }

  pdl_launch_dependents();
  __syncthreads();  // every copy consumed; the stage ring is free
  if (ps.abort_flag) return;

  // merge of the warps: wm, wl [NW][rows], wacc [NW][rows][pitch]
  constexpr int RT = Cfg::kRows, RP = Cfg::kRowPitch;
  float* wacc = reinterpret_cast<float*>(sgen);
  float* wm = wacc + NW * RT * RP;
  float* wl = wm + NW * RT;
  if (warp < NW) {
#pragma unroll
    for (int gi = 0; gi < NG; ++gi)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = 8 * gi + 2 * c + j;
        if (r == 0) {
          wm[warp * RT + row] = m_run[gi][j];
          wl[warp * RT + row] = l_run[gi][j];
        }
        float* dst = wacc + (warp * RT + row) * RP;
#pragma unroll
        for (int t = 0; t < KS; ++t) {
          dst[CF != 0 ? f8_dim<D>(t, r) : 16 * t + r] = o[gi][t][j];
          dst[CF != 0 ? f8_dim<D>(t, r) + 1 : 16 * t + r + 8] = o[gi][t][2 + j];
        }
      }
  }
  __syncthreads();
  for (int idx = tid; idx < rows * (D / 4); idx += Cfg::kThreads) {
    const int row = idx / (D / 4), d = (idx - row * (D / 4)) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, wm[w * RT + row]);
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (M != -INFINITY) {
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = exp2f(wm[w * RT + row] - M);
        const float4 v = *reinterpret_cast<const float4*>(wacc + (w * RT + row) * RP + d);
        l = fmaf(wl[w * RT + row], f, l);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
    }
    const int h = (g << a.gshift) + (row & ((1 << a.gshift) - 1));
    const int64_t orow = static_cast<int64_t>(ms.q0 + (row >> a.gshift)) * a.hq + h;
    if (ms.nparts > 1) {
      const int64_t prow = orow * a.max_parts + p;
      *reinterpret_cast<float4*>(a.ws_o + prow * D + d) = acc;
      if (d == 0) *reinterpret_cast<float2*>(a.ws_ml + prow * 2) = make_float2(M, l);
      continue;
    }
    float lse;
    const float f = finish_row(a.sinks, h, M, l, lse) * a.v_scale;
    const __nv_bfloat162 y0 = __floats2bfloat162_rn(acc.x * f, acc.y * f), y1 = __floats2bfloat162_rn(acc.z * f, acc.w * f);
    *reinterpret_cast<uint2*>(a.out + orow * D + d) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
    if (d == 0 && a.lse) a.lse[orow] = lse;
  }
}

// Merge of a split sequence's partials: one warp per (new token, query head)
// row, grid (rows of the longest sequence / warps, sequences). A lane owns D / 32
// dims, so a partial is one coalesced read; four are in flight at a time.
constexpr int kMultiMergeWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kMultiMergeWarps) decode_multi_merge_kernel(const MultiArgs a) {
  constexpr int VEC = D / 32, U = 4;
  const int s = blockIdx.y, lane = threadIdx.x & 31;
  const int ri = blockIdx.x * kMultiMergeWarps + (threadIdx.x >> 5);
  const MultiSeq ms = load_multi_seq(a, s, false);
  pdl_wait();  // the partials are written by the grid this one was launched behind
  if (ms.nparts <= 1 || ri >= ms.n * a.hq) return;
  const int64_t row = static_cast<int64_t>(ms.q0) * a.hq + ri;
  const float* ml = a.ws_ml + row * a.max_parts * 2;
  const float* po = a.ws_o + row * a.max_parts * D + lane * VEC;
  float M = -INFINITY;
  for (int q = lane; q < ms.nparts; q += 32) M = fmaxf(M, __ldcg(ml + 2 * q));
  M = warp_max(M);
  float l = 0.f, acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  if (M != -INFINITY) {
    for (int q0 = 0; q0 < ms.nparts; q0 += U) {
      float f[U], lq[U], x[U][VEC];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = min(q0 + u, ms.nparts - 1);
        f[u] = __ldcg(ml + 2 * q);
        lq[u] = __ldcg(ml + 2 * q + 1);
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[u][e] = __ldcg(po + static_cast<int64_t>(q) * D + e);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float w = q0 + u < ms.nparts ? exp2f(f[u] - M) : 0.f;
        l = fmaf(lq[u], w, l);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = fmaf(x[u][e], w, acc[e]);
      }
    }
  }
  float lse;
  const float f = finish_row(a.sinks, ri % a.hq, M, l, lse) * a.v_scale;
  __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(a.out + row * D + lane * VEC);
#pragma unroll
  for (int e = 0; e < VEC / 2; ++e) dst[e] = __floats2bfloat162_rn(acc[2 * e] * f, acc[2 * e + 1] * f);
  if (lane == 0 && a.lse) a.lse[row] = lse;
}

}  // namespace pa
