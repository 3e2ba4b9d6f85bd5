// Rotary positions applied on the way into the cache: q and k are rotated by
// their positions, k and v written to their slots, q written out.
//
//   (a', b') = (a cos - b sin, b cos + a sin)
//
// for every pair (a, b) of a head's first rotary_dim dims; the angle of a pair
// belongs to its position and is read from a table of cosines and sines (which
// its maker computes in 64 bits: in 32, the angle of position 10^5 has an error
// of 4e-3). P2 = "PagedAttention：操作系统级 KV 缓存虚拟内存管理", §3.2.2 step 3: the
// new K, V written at their block position.
//
// Bound by HBM: every input byte is read once and every output byte written
// once, three operations per rotated element. A thread owns 16 elements of one
// head row, as two 8-element pieces that hold both members of its pairs: with
// halves paired, piece u and the piece rotary_dim / 2 later; with neighbours
// paired, and for what is not rotated, two pieces side by side. Either way its
// 8 cosines and 8 sines are adjacent, and neighbouring threads read
// neighbouring pieces. The rotation is computed in fp32, each operation
// rounded by itself (no fused multiply-add), and rounded once to the stored
// type: for an 8-bit cache the rotated fp32 value is quantised directly, not
// by way of bf16.
#pragma once

#include "cache_ops.cuh"

namespace pa {

struct RotateArgs {
  const void *q, *k, *v;         // rows [tokens][heads][D] of the input type
  int64_t q_stride, k_stride, v_stride;  // elements from one token to the next
  const int32_t* positions;      // [tokens]
  const float* cos_sin;          // [max_positions][rd]: rd / 2 cosines, rd / 2 sines
  const int64_t* slots;          // [tokens], -1: not cached
  void *q_out, *kc, *vc;
  int64_t num_slots;
  int32_t num_tokens, max_positions, rd, interleaved;
  int32_t hq, hkv, bs;
  int32_t dshift;                // log2 of D / 16, the units of a head row
  int32_t units;                 // per token: (hq + 2 hkv) D / 16
  int32_t tokens_per_cta;
  float k_scale, v_scale;
};

// Eight elements in the registers they are loaded in, as floats, and back.
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16lo(x[i]);
      f[2 * i + 1] = bf16hi(x[i]);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      x[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    w = make_uint4(x[0], x[1], x[2], x[3]);
  }
};
template <>
struct Piece<float> {
  float4 w[2];
  __device__ __forceinline__ void load(const float* p) {
    w[0] = __ldcs(reinterpret_cast<const float4*>(p));
    w[1] = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = w[0];
    reinterpret_cast<float4*>(p)[1] = w[1];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = w[0].x, f[1] = w[0].y, f[2] = w[0].z, f[3] = w[0].w;
    f[4] = w[1].x, f[5] = w[1].y, f[6] = w[1].z, f[7] = w[1].w;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    w[0] = make_float4(f[0], f[1], f[2], f[3]);
    w[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// Eight codes of an 8-bit cache.
template <int CF>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&f)[8], float scale) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = quantize_code<CF>(f[4 * i], scale) | (quantize_code<CF>(f[4 * i + 1], scale) << 8) |
           (quantize_code<CF>(f[4 * i + 2], scale) << 16) | (quantize_code<CF>(f[4 * i + 3], scale) << 24);
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// T: input type; CF: 0 for a cache of the input type, kCodeE4M3 / kCodeS8 for
// an 8-bit cache.
template <typename T, int CF>
__global__ void __launch_bounds__(256) rotate_and_cache_kernel(const RotateArgs a) {
  const int32_t tok0 = blockIdx.x * a.tokens_per_cta;
  const int32_t n = min(a.tokens_per_cta, a.num_tokens - tok0) * a.units;
  const int32_t umask = (1 << a.dshift) - 1;
  const int32_t D = 16 << a.dshift;
  for (int32_t i = threadIdx.x; i < n; i += blockDim.x) {
    const int32_t lt = i / a.units, r = i - lt * a.units;
    const int64_t t = tok0 + lt;
    const int32_t u = r & umask;
    int32_t h = r >> a.dshift;
    const int32_t pos = __ldg(a.positions + t);
    const int64_t slot = __ldg(a.slots + t);
    const bool is_q = h < a.hq, is_v = h >= a.hq + a.hkv;
    h -= is_q ? 0 : (is_v ? a.hq + a.hkv : a.hq);
    const bool rotated = !is_v && 16 * u < a.rd;
    const bool halves = rotated && !a.interleaved;
    const int32_t e0 = halves ? 8 * u : 16 * u;
    const int32_t e1 = e0 + (halves ? a.rd / 2 : 8);
    const T* src = static_cast<const T*>(is_q ? a.q : (is_v ? a.v : a.k)) +
                   t * (is_q ? a.q_stride : (is_v ? a.v_stride : a.k_stride)) + h * D;
    Piece<T> x0, x1;
    x0.load(src + e0);
    x1.load(src + e1);
    if (pos < 0 || pos >= a.max_positions) {  // the token is left out whole
      if (r == 0) record_error(PA_ERR_DEVICE_BOUNDS, pos);
      continue;
    }
    float f0[8], f1[8];
    if (rotated || CF != 0) {
      x0.get(f0);
      x1.get(f1);
    }
    if (rotated) {
      const float4* cp = reinterpret_cast<const float4*>(a.cos_sin + static_cast<int64_t>(pos) * a.rd + 8 * u);
      const float4* sp = reinterpret_cast<const float4*>(a.cos_sin + static_cast<int64_t>(pos) * a.rd + a.rd / 2 + 8 * u);
      const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
      const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
      const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
      auto turn = [](float& p, float& q, float co, float si) {
        const float p0 = p, q0 = q;
        p = __fsub_rn(__fmul_rn(p0, co), __fmul_rn(q0, si));
        q = __fadd_rn(__fmul_rn(q0, co), __fmul_rn(p0, si));
      };
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          turn(f0[2 * e], f0[2 * e + 1], c[e], s[e]);
          turn(f1[2 * e], f1[2 * e + 1], c[4 + e], s[4 + e]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn(f0[e], f1[e], c[e], s[e]);
      }
      x0.set(f0);
      x1.set(f1);
    }
    if (is_q) {
      T* dst = static_cast<T*>(a.q_out) + (t * a.hq + h) * D;
      x0.store(dst + e0);
      x1.store(dst + e1);
      continue;
    }
    if (slot == -1) continue;
    if (slot < -1 || slot >= a.num_slots) {
      if (u == 0 && h == 0 && !is_v) record_error(PA_ERR_DEVICE_BOUNDS, slot);
      continue;
    }
    const int64_t blk = slot / a.bs;
    const int64_t row = ((blk * a.hkv + h) * a.bs + (slot - blk * a.bs)) * D;
    if constexpr (CF != 0) {
      uint8_t* dst = static_cast<uint8_t*>(is_v ? a.vc : a.kc) + row;
      const float sc = is_v ? a.v_scale : a.k_scale;
      store_codes<CF>(dst + e0, f0, sc);
      store_codes<CF>(dst + e1, f1, sc);
    } else {
      T* dst = static_cast<T*>(is_v ? a.vc : a.kc) + row;
      x0.store(dst + e0);
      x1.store(dst + e1);
    }
  }
}

}  // namespace pa
