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
// once, three operations per rotated element (back to back: 16231 tokens of 32 / 32
// heads in bf16 138 us, 5.9 TB/s, 0.89 of a copy's rate, in fp32 312 us, 5.1 TB/s, 0.78;
// 20011 of 64 / 8 heads, half of each rotated, into an e4m3 cache 138 us, 5.7 TB/s, int8
// 148 us, 5.3 TB/s). A thread owns one unit (16
// elements) of several head rows of a token: its cosines, sines and offsets are
// read and computed once for all of them. A unit is two 8-element pieces that
// hold both members of its pairs: with halves paired, piece u and the piece
// rotary_dim / 2 later; with neighbours paired, two adjacent pieces. Either way
// its 8 cosines and 8 sines are adjacent. The rotation is computed in fp32, each
// operation rounded by itself (no fused multiply-add; in packed pairs, mul and
// add came out fused), and rounded once to the stored type: for an 8-bit cache the
// rotated fp32 value is quantised directly, not by way of bf16.
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
  int32_t hq, hkv;
  int32_t bshift;                // log2 of block_size
  int32_t dshift;                // log2 of D / 16, the units of a head row
  int32_t lanes;                 // head rows of a token that are in flight side by side
  int32_t tokens;                // tokens of a CTA side by side: lanes * tokens * D / 16 <= 256
  float k_scale, v_scale, k_rcp, v_rcp;  // 8-bit: scales, and 1 / scale rounded (0: divide)
};

// Eight elements in the registers they are loaded in. Their pairs of
// neighbours, and the elements one by one, as floats.
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 x = __ldcs(reinterpret_cast<const uint4*>(p));
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ float2 pair(int i) const { return make_float2(bf16lo(w[i]), bf16hi(w[i])); }
  __device__ __forceinline__ void set_pair(int i, float2 f) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Piece<float> {
  float w[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 x = __ldcs(reinterpret_cast<const float4*>(p)), y = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = make_float4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(w[4], w[5], w[6], w[7]);
  }
  __device__ __forceinline__ float2 pair(int i) const { return make_float2(w[2 * i], w[2 * i + 1]); }
  __device__ __forceinline__ void set_pair(int i, float2 f) {
    w[2 * i] = f.x;
    w[2 * i + 1] = f.y;
  }
};

// The codes of two values that are already divided by the scale.
template <int CF>
__device__ __forceinline__ uint32_t code_pair(float2 y) {
  if constexpr (CF == kCodeS8) {
    auto code = [](float v) {
      return static_cast<uint32_t>(__float2int_rn(v != v ? 0.f : fminf(fmaxf(v, -127.f), 127.f))) & 0xffu;
    };
    return code(y.x) | (code(y.y) << 8);
  } else {
    return __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
  }
}

// Eight codes of an 8-bit cache: the nearest codes of f / scale, the quotient
// rounded to fp32 as in quantize_e4m3 and quantize_s8. An IEEE division is some
// ten times a multiplication, and only its code is wanted: with rcp = 1 / scale
// rounded, f rcp (1 - 2^-21) and f rcp (1 + 2^-21), each off by three roundings
// of 2^-24, enclose the quotient and its own rounding, and codes rise with their
// argument: where the two have the same code, the quotient has it too. Elsewhere
// (about one element in 2^16) the division decides, and everywhere for an rcp of
// 0 (a scale outside 2^+-100).
template <int CF>
__device__ __forceinline__ void store_codes(uint8_t* p, const float2 (&f)[4], float scale, float rcp) {
  const float2 lo = make_float2(rcp * (1.f - 0x1p-21f), rcp * (1.f - 0x1p-21f));
  const float2 hi = make_float2(rcp * (1.f + 0x1p-21f), rcp * (1.f + 0x1p-21f));
  uint32_t w[2], v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = code_pair<CF>(fmul2(f[2 * i], lo)) | (code_pair<CF>(fmul2(f[2 * i + 1], lo)) << 16);
    v[i] = code_pair<CF>(fmul2(f[2 * i], hi)) | (code_pair<CF>(fmul2(f[2 * i + 1], hi)) << 16);
  }
  if (rcp == 0.f || w[0] != v[0] || w[1] != v[1]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = quantize_code<CF>(f[2 * i].x, scale) | (quantize_code<CF>(f[2 * i].y, scale) << 8) |
             (quantize_code<CF>(f[2 * i + 1].x, scale) << 16) | (quantize_code<CF>(f[2 * i + 1].y, scale) << 24);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// T: input type; CF: 0 for a cache of the input type, kCodeE4M3 / kCodeS8 for
// an 8-bit cache. The grid is at most the four CTAs that fit on every SM, walking
// the tokens: a second wave would cost more than the walk. q rows and k, v rows have
// loops of their own, fewer instructions for each. Side by side, each pair as the kernel
// was at that step: prompts of 16231 tokens, 32 / 32 heads 146 us, 167 at one CTA per
// token; 20011 tokens, 64 / 8 heads over e4m3 133 us, 147 in one loop, 150 with three CTAs
// and the next row's loads in flight.
template <typename T, int CF>
__global__ void __launch_bounds__(256, 4) rotate_and_cache_kernel(const RotateArgs a) {
  const int32_t D = 16 << a.dshift;
  const int32_t u = threadIdx.x & ((1 << a.dshift) - 1), hr = threadIdx.x >> a.dshift;
  const int32_t side = hr / a.lanes;
  int32_t lane = hr - side * a.lanes;
  if (side >= a.tokens) return;
  const int32_t rows = a.hq + 2 * a.hkv, shift = rows % a.lanes;
  // this unit's pieces in a q or k row and in a v row. What is not rotated is
  // taken in halves too, so that neighbouring threads read neighbouring pieces
  const bool turns = 16 * u < a.rd;
  const bool adjacent = turns && a.interleaved;
  const int32_t from = turns ? 0 : a.rd;
  const int32_t e0 = adjacent ? 16 * u : from + 8 * u - from / 2;
  const int32_t e1 = e0 + (adjacent ? 8 : (turns ? a.rd : D - a.rd) / 2);
  const int32_t stride = gridDim.x * a.tokens;
  int64_t t = static_cast<int64_t>(blockIdx.x) * a.tokens + side;
  if (t >= a.num_tokens) return;
  int32_t pos = __ldg(a.positions + t);
  int64_t slot = __ldg(a.slots + t);
  for (;;) {
    const bool known = pos >= 0 && pos < a.max_positions;  // otherwise the token is left out whole
    const bool cached = slot >= 0 && slot < a.num_slots;
    if (u == 0 && lane == 0) {
      if (!known)
        record_error(PA_ERR_DEVICE_BOUNDS, pos);
      else if (!cached && slot != -1)
        record_error(PA_ERR_DEVICE_BOUNDS, slot);
    }
    // cosines and sines of this unit's pairs: pairs 2i, 2i + 1 in one register pair
    float2 co[4], si[4];
    if (turns && known) {
      const float4* cp = reinterpret_cast<const float4*>(a.cos_sin + static_cast<int64_t>(pos) * a.rd + 8 * u);
      const float4* sp = cp + a.rd / 8;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 c = __ldg(cp + i), s = __ldg(sp + i);
        co[2 * i] = make_float2(c.x, c.y);
        co[2 * i + 1] = make_float2(c.z, c.w);
        si[2 * i] = make_float2(s.x, s.y);
        si[2 * i + 1] = make_float2(s.z, s.w);
      }
    }
    // element of kv head 0 of the token's slot
    const int64_t blk = slot >> a.bshift;
    const int64_t crow = ((blk * a.hkv) << a.bshift) + (slot - (blk << a.bshift));
    // the pairs of two pieces turned, as (p, q) = (p c - q s, q c + p s)
    auto rotate = [&](float2 (&f0)[4], float2 (&f1)[4]) {
      auto turn1 = [](float& p, float& q, float c, float s) {
        const float p0 = p;
        p = __fsub_rn(__fmul_rn(p0, c), __fmul_rn(q, s));
        q = __fadd_rn(__fmul_rn(q, c), __fmul_rn(p0, s));
      };
      auto turn = [&](float2& p, float2& q, float2 c, float2 s) {
        turn1(p.x, q.x, c.x, s.x);
        turn1(p.y, q.y, c.y, s.y);
      };
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // pairs 2i, 2i + 1 of each piece: (x, y), (x, y)
          float2 p = make_float2(f0[2 * i].x, f0[2 * i + 1].x), q = make_float2(f0[2 * i].y, f0[2 * i + 1].y);
          turn(p, q, co[i], si[i]);
          f0[2 * i] = make_float2(p.x, q.x);
          f0[2 * i + 1] = make_float2(p.y, q.y);
          p = make_float2(f1[2 * i].x, f1[2 * i + 1].x);
          q = make_float2(f1[2 * i].y, f1[2 * i + 1].y);
          turn(p, q, co[2 + i], si[2 + i]);
          f1[2 * i] = make_float2(p.x, q.x);
          f1[2 * i + 1] = make_float2(p.y, q.y);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) turn(f0[i], f1[i], co[i], si[i]);
      }
    };
    auto unpack = [](const Piece<T>& x, float2 (&f)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = x.pair(i);
    };
    auto pack = [](Piece<T>& x, const float2 (&f)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x.set_pair(i, f[i]);
    };
    int32_t r = known ? lane : rows;
    const T* src = static_cast<const T*>(a.q) + t * a.q_stride + r * D;
    T* dst = static_cast<T*>(a.q_out) + (t * a.hq + r) * D;
    for (; r < a.hq; r += a.lanes) {
      Piece<T> x0, x1;
      x0.load(src + e0);
      x1.load(src + e1);
      if (turns) {
        float2 f0[4], f1[4];
        unpack(x0, f0);
        unpack(x1, f1);
        rotate(f0, f1);
        pack(x0, f0);
        pack(x1, f1);
      }
      x0.store(dst + e0);
      x1.store(dst + e1);
      src += a.lanes * D;
      dst += a.lanes * D;
    }
    // k and v rows
    for (; cached && r < rows; r += a.lanes) {
      const bool is_v = r >= a.hq + a.hkv;
      const int32_t h = r - a.hq - (is_v ? a.hkv : 0);
      const T* kv = is_v ? static_cast<const T*>(a.v) + t * a.v_stride + h * D
                         : static_cast<const T*>(a.k) + t * a.k_stride + h * D;
      const int32_t d0 = is_v ? 8 * u : e0, d1 = is_v ? 8 * u + D / 2 : e1;
      Piece<T> x0, x1;
      x0.load(kv + d0);
      x1.load(kv + d1);
      const int64_t row = (crow + (static_cast<int64_t>(h) << a.bshift)) * D;
      float2 f0[4], f1[4];
      if (CF != 0 || (turns && !is_v)) {
        unpack(x0, f0);
        unpack(x1, f1);
      }
      if (turns && !is_v) rotate(f0, f1);
      if constexpr (CF != 0) {
        uint8_t* to = static_cast<uint8_t*>(is_v ? a.vc : a.kc) + row;
        const float sc = is_v ? a.v_scale : a.k_scale, rcp = is_v ? a.v_rcp : a.k_rcp;
        store_codes<CF>(to + d0, f0, sc, rcp);
        store_codes<CF>(to + d1, f1, sc, rcp);
      } else {
        if (turns && !is_v) {
          pack(x0, f0);
          pack(x1, f1);
        }
        T* to = static_cast<T*>(is_v ? a.vc : a.kc) + row;
        x0.store(to + d0);
        x1.store(to + d1);
      }
    }
    t += stride;
    if (t >= a.num_tokens) return;
    pos = __ldg(a.positions + t);
    slot = __ldg(a.slots + t);
    // the lanes that took one row less take the first ones now
    lane += lane < a.lanes - shift ? shift : shift - a.lanes;
  }
}

}  // namespace pa
