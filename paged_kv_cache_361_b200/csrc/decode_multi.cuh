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
// n new tokens), so the reads take longer than the products. The rows, (token,
// head) pairs of one (sequence, kv head), are handled together, so every K/V byte
// is read once; what is left is to keep the reads going to the end on every SM,
// whatever the lengths: see MultiWork. This kernel takes up to 8 rows, the N of
// its MMAs (more: decode_multi_tc.cuh); its products are those of the single-token
// decode with the tokens as the MMA's M (S^T = K q^T, O^T += V^T P^T), over an
// 8-bit cache two 16-key tiles of a warp at a time (twice the conversions per
// byte: two independent chains hide each other's latency). The keys the rows see
// start inside a chunk and inside a block: blocks wholly before them are not
// read, scores outside a row's window are replaced by -inf, V rows outside [kbeg,
// kend) are zeroed in registers (a freed block may hold anything, NaN too).
//
// Measured (kernels back to back in a graph, inputs larger than L2, as all figures of
// this file): 64 sequences of 1024..8192 keys, 1 token of 64/8 heads: 185 to 192 us over
// bf16, 6.3 to 6.5 TB/s, 0.96 to 0.99 of a copy's rate, 102 to 108 us over e4m3 (0.85 to
// 0.90: the conversions show); 64 of 128..8192 in a window of 1024, 32/8 heads: 50 us,
// 5.1 TB/s (some 10 us of every call are lengths, first copies and merge).
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
  float* ws_ml;            // [2 workers][slot_rows][2]
  float* ws_o;             // [2 workers][slot_rows][D]
  int64_t num_blocks;
  int32_t num_seqs, num_tokens, max_q, hq, hkv, bs, max_blocks, max_ctx;
  int32_t gshift;          // log2 of hq / hkv
  int32_t bshift;          // log2 of block_size
  int32_t window;          // >= 1; max_ctx or more: every earlier key
  int32_t per;             // chunks of a worker; 0: even shares, kWholeUnits: a unit each
  int32_t unit_cost;       // of a unit in an even share, in chunks: see MultiWork
  int32_t slot_rows;       // rows of a partial: max_q hq / hkv
  ScoreScale score;
  float v_scale;
  float o_unit;            // of o: 1 / kWeightF16 where the weights are f16, 1 otherwise
};

// The new rows and length of a sequence, and the start of its chunks.
struct MultiSeq {
  int32_t q0, n, L;
  int32_t first;  // the first key any of its rows sees, down to a multiple of 64
  __device__ __forceinline__ int32_t chunks(int keys) const {
    return n <= 0 ? 0 : max(1, (L - first + keys - 1) / keys);
  }
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
  return m;
}

// The division of the work. A unit is one (sequence, kv head); its chunks are
// KEYS keys each from MultiSeq::first on. The units' chunks, one after another
// (the kv heads of sequence 0, of sequence 1, ...), are cut into even shares, one
// per worker (CTA), so that the CTAs end together whatever the lengths. A worker
// takes its share unit by unit: a unit that lies in one share is finished by its
// worker; of a unit that does not, each worker leaves a partial (m, l, o): in
// slot 2w if it is the worker's first segment, in slot 2w + 1 otherwise (it is
// then the last), and the merge kernel folds them in order. The same lengths give
// the same shares, so results do not change from call to call. Beginning a unit
// costs a worker as much as unit_cost chunks (its rows are loaded, the pipeline
// runs empty and a result is written), so the even shares count each unit as that
// many chunks more, before its first: a share that begins among them has the unit
// from its first chunk on, one that ends among them none of it.
constexpr int32_t kWholeUnits = INT32_MAX;

// Beginning a unit takes a tcgen05 CTA some 6 us, four chunks' time; the three CTAs
// of an SM of the other kernel hide most of it. Measured on tcgen05 at 2 / 5 / 8 chunks:
// 16 sequences of 1000..32768 keys, 5 tokens of 64/8 heads 209 / 190 / 199 us; 64 of
// 300..2000, 8 tokens of 16/8 heads 84 / 83 / 91; but 32 of 1024..8192, 3 tokens of
// 32/8 heads 114 / 130 / 133. On mma.sync at 1 / 2 / 4: 32 of 128..2048, 1 to 4 tokens of
// 32/32 heads over int8 67 / 66 / 72; 64 of 1024..8192, 1 token of 64/8 heads 188 / 185 /
// 189 over bf16, 102 / 102 / 104 over e4m3.
constexpr int32_t kMultiUnitCost = 2, kMultiTcUnitCost = 5;

// Keys of an even share at least: a smaller one costs more than its part of the work.
// At half / this / twice: on mma.sync, 1 token of 64/8 heads, 4 sequences of 1000..4000
// keys 20.0 / 18.9 / 20.4 us, 1 of 3000 12.2 / 13.9 / 17.3, 16 of 300..1000 (32/8 heads)
// 18.8 / 18.1 / 20.3; on tcgen05, 64/8 heads, 4 tokens of 2 sequences of 2000..4000 keys
// 22.3 / 23.6 / 27.5, 5 of 1 of 6000 22.1 / 23.5 / 27.3, 5 of 16 of 300..1000 26.6 / 26.6 /
// 18.9 (whole units then, without a merge).
constexpr int32_t kMultiMinKeys = 256, kMultiTcMinKeys = 512;

struct MultiWork {
  int32_t s, g, c;   // where the share starts: sequence, kv head, chunk of the unit
  int64_t per;       // chunks of a share
  int64_t left;      // chunks of this one, 0: none
  int32_t cost;      // the part of `left` that beginning the first unit takes
};

// Chunks and costs of one kv head over all sequences and over those before s0, and
// the length of a share; by one warp, the same in every lane.
struct MultiSpan {
  int64_t total, before, per;
};

template <int KEYS>
__device__ __forceinline__ MultiSpan multi_span(const MultiArgs& a, int s0, int64_t workers, int min_per,
                                                bool report = false) {
  MultiSpan p;
  p.total = p.before = 0;
  for (int s = threadIdx.x & 31; s < a.num_seqs; s += 32) {
    const int c = load_multi_seq(a, s, report).chunks(KEYS);
    const int x = c > 0 ? c + a.unit_cost : 0;
    p.total += x;
    if (s < s0) p.before += x;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    p.total += __shfl_xor_sync(0xffffffffu, p.total, o);
    p.before += __shfl_xor_sync(0xffffffffu, p.before, o);
  }
  p.per = a.per > 0 ? a.per
                    : max(static_cast<int64_t>(min_per + a.unit_cost), (p.total * a.hkv + workers - 1) / workers);
  return p;
}

// The share of worker w of `workers`, at least min_per chunks each; by one warp,
// the same in every lane.
template <int KEYS>
__device__ __forceinline__ MultiWork find_work(const MultiArgs& a, int64_t w, int64_t workers, int min_per, bool report) {
  const int lane = threadIdx.x & 31;
  MultiWork k;
  k.s = k.g = k.c = k.cost = 0;
  if (a.per == kWholeUnits) {
    k.s = static_cast<int32_t>(w / a.hkv);
    k.g = static_cast<int32_t>(w - static_cast<int64_t>(k.s) * a.hkv);
    k.per = kWholeUnits;
    k.left = load_multi_seq(a, k.s, report && k.g == 0 && lane == 0).chunks(KEYS);
    return k;
  }
  const MultiSpan sp = multi_span<KEYS>(a, 0, workers, min_per, report && w == 0);
  const int64_t total = sp.total * a.hkv;
  k.per = sp.per;
  const int64_t x = w * k.per;
  k.left = x >= total ? 0 : min(k.per, total - x);
  if (k.left == 0) return k;
  int64_t base = 0;  // chunks and costs (of one kv head) of the sequences before s0
  for (int s0 = 0;; s0 += 32) {
    int c = s0 + lane < a.num_seqs ? load_multi_seq(a, s0 + lane, false).chunks(KEYS) : 0;
    if (c > 0) c += a.unit_cost;
    int64_t upto = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, (base + upto) * a.hkv > x);
    if (hit) {
      const int at = __ffs(hit) - 1;
      const int64_t from = (base + __shfl_sync(0xffffffffu, upto - c, at)) * a.hkv;
      const int cs = __shfl_sync(0xffffffffu, c, at);
      k.s = s0 + at;
      k.g = static_cast<int32_t>((x - from) / cs);
      const int32_t at_unit = static_cast<int32_t>(x - from - static_cast<int64_t>(k.g) * cs);
      k.c = max(0, at_unit - a.unit_cost);
      k.cost = max(0, a.unit_cost - at_unit);
      return k;
    }
    base += __shfl_sync(0xffffffffu, upto, 31);
  }
}

// One segment of a worker's share: some chunks of one unit.
struct MultiSegment {
  MultiSeq ms;
  int32_t s, g, rows;
  int32_t kbeg, kend;     // keys that some row sees, within the segment
  int32_t begin, chunks;  // its first chunk's first key, and how many are read (0: no key to see)
  bool whole;             // the whole unit
  int64_t slot;           // of its partial otherwise
};

// Walks the segments of a share (every warp for itself).
template <int KEYS>
struct MultiWalk {
  MultiWork k;
  int64_t w;
  bool started;
  __device__ __forceinline__ MultiWalk(const MultiWork& work, int64_t worker) : k(work), w(worker), started(false) {}
  __device__ __forceinline__ bool next(const MultiArgs& a, MultiSegment& e) {
    k.left -= k.cost;
    if (k.left <= 0) return false;
    int32_t cs;
    for (;; ++k.s) {  // a share is left, so some sequence from here on has chunks
      e.ms = load_multi_seq(a, k.s, false);
      cs = e.ms.chunks(KEYS);
      if (cs > 0) break;
    }
    const int32_t nc = static_cast<int32_t>(min(k.left, static_cast<int64_t>(cs - k.c)));
    e.s = k.s;
    e.g = k.g;
    e.rows = e.ms.n << a.gshift;
    e.begin = e.ms.first + k.c * KEYS;
    e.kend = k.c + nc == cs ? e.ms.L : e.begin + nc * KEYS;
    e.kbeg = max(e.begin, e.ms.L - e.ms.n - a.window + 1);
    e.chunks = e.kend > e.kbeg ? (e.kend - e.begin + KEYS - 1) / KEYS : 0;
    e.whole = k.c == 0 && nc == cs;
    e.slot = 2 * w + (started ? 1 : 0);
    started = true;
    k.left -= nc;
    k.c = 0;
    k.cost = a.unit_cost;
    if (++k.g == a.hkv) {
      k.g = 0;
      ++k.s;
    }
    return true;
  }
};

// A producer warp's block ids: lane i holds that of the chunk's block i, read
// from the table one chunk ahead. (A window of ids shared by shuffles, and block
// numbers by division, took the producer 2000 cycles a chunk, which set the
// kernel's pace.)
template <int KEYS>
struct BlocksAhead {
  const int32_t* row;
  int32_t end, nxt;  // blocks of the segment end before `end`
  __device__ __forceinline__ int32_t fetch(const MultiArgs& a, int32_t key, int lane) const {
    const int32_t i = (key >> a.bshift) + lane;
    return lane < (KEYS >> a.bshift) && i < end ? __ldg(row + i) : -1;
  }
  __device__ __forceinline__ void init(const MultiArgs& a, const MultiSegment& e, int lane) {
    row = a.tables + static_cast<int64_t>(e.s) * a.max_blocks;
    end = min(a.max_blocks, (e.kend + a.bs - 1) >> a.bshift);
    nxt = fetch(a, e.begin, lane);
  }
  // Block of this lane in the chunk at `key`; true if it holds a key in [kbeg,
  // kend) and its id is in the pool (if not, that is recorded).
  __device__ __forceinline__ bool next(const MultiArgs& a, const MultiSegment& e, int32_t key, int lane, bool report,
                                       int32_t& blk) {
    blk = nxt;
    nxt = fetch(a, key + KEYS, lane);
    if (lane >= (KEYS >> a.bshift) || (key >> a.bshift) + lane >= end || key + ((lane + 1) << a.bshift) <= e.kbeg)
      return false;
    const bool ok = blk >= 0 && blk < a.num_blocks;
    if (!ok && report) record_error(PA_ERR_DEVICE_BOUNDS, blk);
    return ok;
  }
};

// Row of q, out and lse of row rho of a segment.
__device__ __forceinline__ int64_t multi_row(const MultiArgs& a, const MultiSegment& e, int rho) {
  return static_cast<int64_t>(e.ms.q0 + (rho >> a.gshift)) * a.hq + (e.g << a.gshift) + (rho & ((1 << a.gshift) - 1));
}

// Four dims d of row rho, from its (m, l) and unnormalised o: the result, or the
// segment's partial.
template <int D>
__device__ __forceinline__ void store_multi(const MultiArgs& a, const MultiSegment& e, int rho, int d, float m, float l,
                                            float4 o) {
  if (!e.whole) {
    const int64_t prow = e.slot * a.slot_rows + rho;
    *reinterpret_cast<float4*>(a.ws_o + prow * D + d) = o;
    if (d == 0) *reinterpret_cast<float2*>(a.ws_ml + prow * 2) = make_float2(m, l);
    return;
  }
  float lse;
  const float f = finish_row(a.sinks, (e.g << a.gshift) + (rho & ((1 << a.gshift) - 1)), m, l, a.o_unit, lse);
  const float s = a.v_scale;
  const int64_t row = multi_row(a, e, rho);
  const __nv_bfloat162 y0 = __floats2bfloat162_rn(o.x * f * s, o.y * f * s),
                       y1 = __floats2bfloat162_rn(o.z * f * s, o.w * f * s);
  *reinterpret_cast<uint2*>(a.out + row * D + d) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
  if (d == 0 && a.lse) a.lse[row] = lse;
}

template <int D, int CF>
struct MultiCfg {
  static constexpr int kConsumerWarps = 4;
  static constexpr int kThreads = 32 * (kConsumerWarps + 1);
  static constexpr int kTiles = CF != 0 ? 2 : 1;   // 16-key MMA tiles of a warp per chunk
  static constexpr int kChunk = 64 * kTiles;
  static constexpr int kEl = CF != 0 ? 1 : 2;
  static constexpr int kTileBytes = kChunk * D * kEl;  // K (or V) of one stage
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kCtas = 3;                  // per SM
  static constexpr int kStages = 64 * 1024 / kStageBytes;
  static constexpr int kFoldFloats = 32 * (D / 4 + 4);  // one warp's state
  static constexpr int kRowPitch = D + 4;          // floats of a row of the result
  static constexpr int kMinChunks = kMultiMinKeys / kChunk;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + 2 * kFoldFloats * 4;
  static_assert(8 * (kRowPitch + 2) <= kFoldFloats, "the result takes the place of a state");
};

// Up to 8 rows. Warp 4 streams K/V into a ring of stages, on into the next
// segment while the others finish one; warps 0-3 take 16 (8-bit: 32) keys each
// of every chunk and fold their states in two rounds.
template <int D, int CF>
__global__ void __launch_bounds__(MultiCfg<D, CF>::kThreads, MultiCfg<D, CF>::kCtas)
    decode_multi_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                        const MultiArgs a) {
  using Cfg = MultiCfg<D, CF>;
  constexpr int NW = Cfg::kConsumerWarps, C = Cfg::kChunk, S = Cfg::kStages, KS = D / 16, MT = Cfg::kTiles;

  extern __shared__ uint8_t smem_raw[];
  __shared__ PipeSmem<S> ps;
  __shared__ int stop;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - smem_u32(smem_raw));
  float* fold = reinterpret_cast<float*>(sgen + S * Cfg::kStageBytes);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;
  if (tid == 0) {
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
    pipe_init<S>(ps, NW);
  }
  MultiWalk<C> walk(find_work<C>(a, blockIdx.x, gridDim.x, Cfg::kMinChunks, warp == 0), blockIdx.x);
  MultiSegment e;
  __syncthreads();

  if (warp == NW) {
    // ---- producer: the blocks of every chunk that hold a key in [kbeg, kend) ----
    const uint32_t box_bytes = static_cast<uint32_t>(a.bs) * D * Cfg::kEl;
    const uint64_t pol = kv_stream_policy();
    int jg = 0;
    while (walk.next(a, e)) {
      BlocksAhead<C> ahead;
      ahead.init(a, e, lane);
      bool gave_up = false;
      for (int j = 0; j < e.chunks; ++j, ++jg) {
        const int st = jg % S;
        if (jg >= S && !pipe_wait(&ps.empty[st], ((jg / S) - 1) & 1, &ps.abort_flag)) {
          gave_up = true;
          break;
        }
        int32_t blk;
        const bool ok = ahead.next(a, e, e.begin + j * C, lane, true, blk);
        const int cnt = __popc(__ballot_sync(0xffffffffu, ok));
        if (lane == 0) mbar_arrive_expect_tx(&ps.full[st], 2u * cnt * box_bytes);
        __syncwarp();
        if (ok) {
          const int32_t y = (blk * a.hkv + e.g) * a.bs;
          const uint32_t kdst = sbase + st * Cfg::kStageBytes + lane * box_bytes;
          if constexpr (CF != 0) {
            tma_load_2d(kdst, &tmk, 0, y, &ps.full[st], pol);
            tma_load_2d(kdst + Cfg::kTileBytes, &tmv, 0, y, &ps.full[st], pol);
          } else {
            tma_block<D>(kdst, &tmk, y, &ps.full[st], pol);
            tma_block<D>(kdst + Cfg::kTileBytes, &tmv, y, &ps.full[st], pol);
          }
        }
      }
      if (gave_up) break;
    }
    if (ps.abort_flag)  // copies already started land before exit
      for (int j = (jg > S ? jg - S : 0); j < jg; ++j) mbar_wait(&ps.full[j % S], (j / S) & 1);
  } else {
    // ---- consumers: warp w has keys [16 MT w, 16 MT (w + 1)) of every chunk ----
    const int mk = lane >> 3, ik = lane & 7;
    int jg = 0;
    while (walk.next(a, e)) {
      const int32_t pos0 = e.ms.L - e.ms.n, pos_hi = e.ms.L - 1;  // positions of the first and last new token
      // q as the B fragments of S^T (column r = row r, zeros past the last): dims
      // (2c, 2c + 1) and (+8) of a 16-dim step, or over an 8-bit cache, as f16,
      // dims (4c, 4c + 1) and (4c + 2, 4c + 3)
      uint2 qr[KS];
      {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(a.q + multi_row(a, e, r < e.rows ? r : 0) * D);
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
          qr[kk] = make_uint2(0u, 0u);
          if (r < e.rows) {
            if constexpr (CF != 0) {
              const uint2 x = __ldg(reinterpret_cast<const uint2*>(w + kk * 8 + 2 * c));
              qr[kk] = make_uint2(pack_f16(bf16lo(x.x), bf16hi(x.x)), pack_f16(bf16lo(x.y), bf16hi(x.y)));
            } else {
              qr[kk] = make_uint2(__ldg(w + kk * 8 + c), __ldg(w + kk * 8 + 4 + c));
            }
          }
        }
      }
      // positions of this lane's rows 2c, 2c + 1: the last key each sees
      int32_t pos[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) pos[j] = 2 * c + j < e.rows ? pos0 + ((2 * c + j) >> a.gshift) : -1;
      float o[KS][4], m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
#pragma unroll
      for (int t = 0; t < KS; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;

      for (int j = 0; j < e.chunks; ++j, ++jg) {
        const int st = jg % S;
        if (!pipe_wait(&ps.full[st], (jg / S) & 1, &ps.abort_flag)) break;
        const int32_t key0 = e.begin + j * C + warp * (16 * MT);  // this warp's first key
        if (key0 + 16 * MT > e.kbeg && key0 < e.kend) {           // warp-uniform
          const uint32_t kst = sbase + st * Cfg::kStageBytes, vst = kst + Cfg::kTileBytes;
          float x[MT][4];  // scores of keys r, r + 8 of a tile, rows 2c, 2c + 1; two chains
#pragma unroll
          for (int u = 0; u < MT; ++u) {
            float s1[4] = {0.f, 0.f, 0.f, 0.f};
            x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0.f;
            if constexpr (CF == 0) {
              // stage layout as in mma_chunk: block-major, 64-element halves, swizzled rows
              const int tok = warp * 16 + (mk >> 1) * 8 + ik, dK = (mk & 1) * 8;
              const uint32_t hstride = static_cast<uint32_t>(a.bs) * 128u;
              const uint32_t kbase = kst + (tok + (tok & ~(a.bs - 1)) * (D / 64 - 1)) * 128;
#pragma unroll
              for (int kk = 0; kk < KS; ++kk) {
                const int d0 = kk * 16 + dK;
                uint32_t m0, m1, m2, m3;
                ldsm_x4(kbase + (d0 >> 6) * hstride + ((((d0 & 63) >> 3) ^ (tok & 7)) << 4), m0, m1, m2, m3);
                mma16x8(kk & 1 ? s1 : x[u], m0, m2, m1, m3, qr[kk].x, qr[kk].y);
              }
            } else {
              uint32_t rb[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int row = (warp * MT + u) * 16 + h * 8 + r;
                const uint32_t key = D == 128 ? static_cast<uint32_t>(row & 7) : static_cast<uint32_t>((row >> 1) & 3);
                rb[h] = (kst + static_cast<uint32_t>(row * D)) | (key << 4) | static_cast<uint32_t>(4 * c);
              }
#pragma unroll
              for (int kk = 0; kk < KS; ++kk) {
                uint32_t w0, w1;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w0) : "r"(rb[0] ^ static_cast<uint32_t>(kk << 4)));
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w1) : "r"(rb[1] ^ static_cast<uint32_t>(kk << 4)));
                uint32_t k00, k01, k10, k11;
                widen4<CF>(w0, k00, k01);
                widen4<CF>(w1, k10, k11);
                mma16x8_f16(kk & 1 ? s1 : x[u], k00, k10, k01, k11, qr[kk].x, qr[kk].y);
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x[u][i] += s1[i];
          }
          // base-2 scores; -inf outside a row's keys (every row sees all of the
          // warp's keys in most chunks)
          if (a.score.cap_log2 > 0.f) {
            float amax = 0.f;
#pragma unroll
            for (int u = 0; u < MT; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fabsf(x[u][i]));
            if (__all_sync(0xffffffffu, amax * a.score.cap_k <= kCapMedium)) {
#pragma unroll
              for (int u = 0; u < MT; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[u][i] = capped_medium(a.score, x[u][i]);
            } else {
#pragma unroll
              for (int u = 0; u < MT; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[u][i] = capped_score(a.score, x[u][i]);
            }
          } else {
#pragma unroll
            for (int u = 0; u < MT; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) x[u][i] *= a.score.scale_log2;
          }
          const bool inside = key0 >= e.kbeg && key0 + 16 * MT <= e.kend;
          if (!inside || key0 + 16 * MT - 1 > pos0 || key0 <= pos_hi - a.window) {
#pragma unroll
            for (int u = 0; u < MT; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int32_t key = key0 + u * 16 + r + (i >> 1) * 8, last = pos[i & 1];
                if (key < e.kbeg || key >= e.kend || key > last || key <= last - a.window) x[u][i] = -INFINITY;
              }
          }
          // weights. The reference maximum moves only when a score exceeds it by
          // 8, so weights stay <= 2^8 and o is rarely rescaled
          float mloc[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v = fmaxf(x[0][h], x[0][2 + h]);
            if constexpr (MT == 2) v = fmax3(v, x[1][h], x[1][2 + h]);
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            mloc[h] = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          }
          const bool move[2] = {mloc[0] > m_run[0] + 8.f, mloc[1] > m_run[1] + 8.f};
          if (__any_sync(0xffffffffu, move[0] || move[1])) {
            float alpha[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              alpha[h] = move[h] ? fast_exp2(m_run[h] - mloc[h]) : 1.f;  // 0 from -inf
              if (move[h]) m_run[h] = mloc[h];
              l_run[h] *= alpha[h];
            }
#pragma unroll
            for (int t = 0; t < KS; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[t][i] *= alpha[i & 1];
          }
          // P^T as B fragments (K 16 keys x N 8 rows): f16 (times kWeightF16), or over a
          // bf16 cache a bf16 and its remainder
          uint32_t pb[MT][CF != 0 ? 2 : 4];
          const float ref[2] = {m_run[0] == -INFINITY ? 0.f : m_run[0],   // a row that has seen
                                m_run[1] == -INFINITY ? 0.f : m_run[1]};  // nothing: weights 0
#pragma unroll
          for (int u = 0; u < MT; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[u][i] = fast_exp2(x[u][i] - ref[i & 1]);
            l_run[0] += x[u][0] + x[u][2];
            l_run[1] += x[u][1] + x[u][3];
            if constexpr (CF != 0) {
              pb[u][0] = movmatrix_t(pack_f16(x[u][0] * kWeightF16, x[u][1] * kWeightF16));
              pb[u][1] = movmatrix_t(pack_f16(x[u][2] * kWeightF16, x[u][3] * kWeightF16));
            } else {
              uint32_t h01, l01, h23, l23;
              split_pair(x[u][0], x[u][1], h01, l01);
              split_pair(x[u][2], x[u][3], h23, l23);
              pb[u][0] = movmatrix_t(h01);
              pb[u][1] = movmatrix_t(h23);
              pb[u][2] = movmatrix_t(l01);
              pb[u][3] = movmatrix_t(l23);
            }
          }
          // V rows outside [kbeg, kend) as zeros: this lane's keys 2c, 2c + 1 (mlo) and + 8 (mhi)
#pragma unroll
          for (int u = 0; u < MT; ++u) {
            uint32_t mlo = 0xffffffffu, mhi = 0xffffffffu;
            if (!inside) {
              auto live = [&](int k) {
                return key0 + u * 16 + k >= e.kbeg && key0 + u * 16 + k < e.kend;
              };
              mlo = (live(2 * c) ? 0x0000ffffu : 0u) | (live(2 * c + 1) ? 0xffff0000u : 0u);
              mhi = (live(2 * c + 8) ? 0x0000ffffu : 0u) | (live(2 * c + 9) ? 0xffff0000u : 0u);
            }
            if constexpr (CF == 0) {
              const int tok = warp * 16 + (mk & 1) * 8 + ik, dV = (mk >> 1) * 8;
              const uint32_t hstride = static_cast<uint32_t>(a.bs) * 128u;
              const uint32_t vbase = vst + (tok + (tok & ~(a.bs - 1)) * (D / 64 - 1)) * 128;
#pragma unroll
              for (int t = 0; t < KS; ++t) {
                const int d0 = t * 16 + dV;
                uint32_t v0, v1, v2, v3;
                ldsm_x4_t(vbase + (d0 >> 6) * hstride + ((((d0 & 63) >> 3) ^ (tok & 7)) << 4), v0, v1, v2, v3);
                v0 &= mlo;
                v1 &= mhi;
                v2 &= mlo;
                v3 &= mhi;
                mma16x8(o[t], v0, v2, v1, v3, pb[u][0], pb[u][1]);
                mma16x8(o[t], v0, v2, v1, v3, pb[u][2], pb[u][3]);
              }
            } else {
              constexpr int W = D == 128 ? 4 : 2;  // 32-bit words of V per key this thread reads
              const uint8_t* vt = sgen + (vst - sbase);
              const int col = f8_dim<D>(0, r), ta0 = (warp * MT + u) * 16 + 2 * c, tb0 = ta0 + 8;
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
                mma16x8_f16(o[2 * w], b[0], b[1], b[4], b[5], pb[u][0], pb[u][1]);
                mma16x8_f16(o[2 * w + 1], b[2], b[3], b[6], b[7], pb[u][0], pb[u][1]);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ps.empty[st]);
      }
      sum_l(l_run);
#pragma unroll
      for (int h = 0; h < 2; ++h) m_run[h] = final_ref(m_run[h], l_run[h]);
      // fold the warps' states: 2 and 3 into 0 and 1, 1 into 0, then out as rows. A
      // warp that gave up a wait joins every barrier; thread 0 decides for all.
      float* mine = fold + (warp & 1) * Cfg::kFoldFloats + lane * (D / 4 + 4);
      if (warp >= 2) store_state<D>(mine, m_run, l_run, o);
      consumer_bar();
      if (warp < 2) fold_state<D>(m_run, l_run, o, mine);
      consumer_bar();
      if (warp == 1) store_state<D>(fold + lane * (D / 4 + 4), m_run, l_run, o);
      consumer_bar();
      float* rowsf = fold + Cfg::kFoldFloats;
      float* ml = rowsf + 8 * Cfg::kRowPitch;
      if (warp == 0) {
        fold_state<D>(m_run, l_run, o, fold + lane * (D / 4 + 4));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float* dst = rowsf + (2 * c + h) * Cfg::kRowPitch;
#pragma unroll
          for (int t = 0; t < KS; ++t) {
            dst[CF != 0 ? f8_dim<D>(t, r) : 16 * t + r] = o[t][h];
            dst[CF != 0 ? f8_dim<D>(t, r) + 1 : 16 * t + r + 8] = o[t][2 + h];
          }
          if (r == 0) {
            ml[2 * (2 * c + h)] = m_run[h];
            ml[2 * (2 * c + h) + 1] = l_run[h];
          }
        }
        if (lane == 0) stop = *static_cast<volatile int*>(&ps.abort_flag);
      }
      consumer_bar();
      if (stop) break;
      for (int i = tid; i < e.rows * (D / 4); i += 32 * NW) {
        const int rho = i / (D / 4), d = (i - rho * (D / 4)) * 4;
        store_multi<D>(a, e, rho, d, ml[2 * rho], ml[2 * rho + 1],
                       *reinterpret_cast<const float4*>(rowsf + rho * Cfg::kRowPitch + d));
      }
      consumer_bar();  // the buffer is free for the next segment
    }
  }
  // (at the start it was slower: 54 against 51 us under a window of 1024, 60 against 53
  // for one sequence of 131072 keys)
  pdl_launch_dependents();
}

// Merge of the units that several workers share; the first of the `n` partials of a
// row is worker w's, the others are of the workers after it.
//
// kMultiMergeWarps rows a CTA, a warp each: CTA row w looks at the boundary between
// workers w - 1 and w (grid.x: w from 1, grid.y: rows). The first boundary inside a
// unit merges it, over the partials of worker w - 1 and of those from w on until the
// unit's end.
// WIDE, for few units (grid.x) over many workers: a CTA per unit and row, whose warps
// share the row's partials: at 55 workers a unit (1 sequence of 131072 keys, 64/8 heads,
// e4m3) the step takes 50 us, against 70 by single warps, at 13.9 49 against 54, at 6.9
// 51 either way; on tcgen05 at 18.5 37 against 42, at 9.3 55.5 against 59, at 4.6 95
// against 93.
constexpr int kMultiMergeWarps = 4, kMultiWideWarps = 8, kMultiWideParts = 8;

template <int D, int KEYS, int MIN_CHUNKS, bool WIDE>
__global__ void __launch_bounds__(32 * (WIDE ? kMultiWideWarps : kMultiMergeWarps))
    decode_multi_merge_kernel(const MultiArgs a, int64_t workers) {
  constexpr int VEC = D / 32, U = 4, NW = WIDE ? kMultiWideWarps : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rho = WIDE ? blockIdx.y : blockIdx.y * kMultiMergeWarps + warp;
  int64_t slot0, w;  // slot of the first partial, and the worker after its
  int nparts;
  MultiSegment e;
  e.whole = true;
  e.slot = 0;
  if constexpr (WIDE) {
    e.s = blockIdx.x / a.hkv;
    e.g = blockIdx.x - e.s * a.hkv;
    e.ms = load_multi_seq(a, e.s, false);
    const int32_t cs = e.ms.chunks(KEYS);
    const MultiSpan sp = multi_span<KEYS>(a, e.s, workers, MIN_CHUNKS);
    const int64_t at = sp.before * a.hkv + static_cast<int64_t>(e.g) * (cs + a.unit_cost), x = at + a.unit_cost;
    w = x / sp.per;
    nparts = cs > 0 ? static_cast<int>((x + cs - 1) / sp.per - w) + 1 : 0;
    slot0 = 2 * w + (w * sp.per >= at ? 0 : 1);
    ++w;
  } else {
    w = blockIdx.x + 1;
    const MultiWork k = find_work<KEYS>(a, w, workers, MIN_CHUNKS, false);
    e.s = k.s;
    e.g = k.g;
    e.ms = load_multi_seq(a, k.s, false);
    // worker w - 1 has the first k.c chunks (in its slot 0 if the unit is its first),
    // the workers from w on the rest
    const int32_t rest = e.ms.chunks(KEYS) - k.c;
    nparts = k.left == 0 || k.c == 0 || k.c > k.per ? 0 : 1 + static_cast<int>((rest + k.per - 1) / k.per);
    slot0 = 2 * (w - 1) + (k.c + a.unit_cost >= k.per ? 0 : 1);
  }
  e.rows = e.ms.n << a.gshift;
  pdl_wait();  // the partials are written by the grid this one was launched behind
  if (nparts < 2 || rho >= e.rows) return;
  auto slot = [&](int q) { return (q == 0 ? slot0 : 2 * (w + q - 1)) * a.slot_rows + rho; };
  float M = -INFINITY;
  for (int q = lane; q < nparts; q += 32) M = fmaxf(M, __ldcg(a.ws_ml + 2 * slot(q)));
  M = warp_max(M);
  float l = 0.f, acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
  if (M != -INFINITY) {
    for (int q0 = WIDE ? warp : 0; q0 < nparts; q0 += U * NW) {  // U partials in flight at a time
      float f[U], lq[U], x[U][VEC];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = slot(min(q0 + u * NW, nparts - 1));
        f[u] = __ldcg(a.ws_ml + 2 * row);
        lq[u] = __ldcg(a.ws_ml + 2 * row + 1);
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[u][i] = __ldcg(a.ws_o + row * D + lane * VEC + i);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float wt = q0 + u * NW < nparts ? exp2f(f[u] - M) : 0.f;
        l = fmaf(lq[u], wt, l);
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = fmaf(x[u][i], wt, acc[i]);
      }
    }
  }
  if constexpr (WIDE) {
    __shared__ float sl[NW], so[NW][D];
    if (lane == 0) sl[warp] = l;
#pragma unroll
    for (int i = 0; i < VEC; ++i) so[warp][lane * VEC + i] = acc[i];
    __syncthreads();
    if (warp > 0) return;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
#pragma unroll
    for (int q = 0; q < NW; ++q) {
      l += sl[q];
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] += so[q][lane * VEC + i];
    }
  }
  float lse;
  const float f = finish_row(a.sinks, (e.g << a.gshift) + (rho & ((1 << a.gshift) - 1)), M, l, a.o_unit, lse);
  const int64_t row = multi_row(a, e, rho);
  __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(a.out + row * D + lane * VEC);
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) dst[i] = __floats2bfloat162_rn(acc[2 * i] * f * a.v_scale, acc[2 * i + 1] * f * a.v_scale);
  if (lane == 0 && a.lse) a.lse[row] = lse;
}

}  // namespace pa
