// Rotary positions: the angle of one pair, and the 16-byte row chunks the kernels move.
// Shared by rope.cu (queries and keys) and cache.cu (keys on their way into the cache).
#pragma once

#include <cuda_fp16.h>

#include "tc_ptx.cuh"

namespace focus {

// cos and sin of pos * f_i, times g.  turn = f_i / 2 pi as a fraction of 2^64, so the
// 64-bit product's wrap-around is the reduction modulo one turn, exactly, for every
// position (in fp32 the product alone would be off by 0.06 rad at a million tokens).
// Its upper half is the angle in units of 2^-32 turns.  What it is away from the nearest quarter
// of a turn goes to fp32, so that the rounding is of an eighth of a turn at most and of next to
// nothing next to a zero of the cosine or the sine.  Their Taylor series there, z = x pi / 4 with |x| <= 1:
// the first terms left out are z^11 / 11! (2^-29) and z^12 / 12! (2^-33); the first factor of the sine
// is held as two numbers, so both are within one step.  (sincospif reduces its argument again:
// as exact, but 200K tokens of one head took 72 us against 60.)
__device__ __forceinline__ void rope_angle(int64_t pos, uint64_t turn, float g, float& c, float& s) {
  const uint32_t t = (uint32_t)(((uint64_t)pos * turn) >> 32);
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  constexpr double z = 0.78539816339744830962, z2 = z * z;  // pi / 4
  constexpr float s1 = (float)z, s1_rest = (float)(z - (double)s1);
  constexpr float s3 = (float)(-z * z2 / 6), s5 = (float)(z * z2 * z2 / 120), s7 = (float)(-z * z2 * z2 * z2 / 5040),
                  s9 = (float)(z * z2 * z2 * z2 * z2 / 362880);
  constexpr float c2 = (float)(-z2 / 2), c4 = (float)(z2 * z2 / 24), c6 = (float)(-z2 * z2 * z2 / 720),
                  c8 = (float)(z2 * z2 * z2 * z2 / 40320), c10 = (float)(-z2 * z2 * z2 * z2 * z2 / 3628800);
  const float a = (float)(int)(t - (quarter << 30)) * 1.862645149230957e-09f, u = a * a;  // 2^-29
  const float y = __fmaf_rn(a, s1, a * __fmaf_rn(u, __fmaf_rn(u, __fmaf_rn(u, __fmaf_rn(u, s9, s7), s5), s3), s1_rest));
  const float x = __fmaf_rn(u, __fmaf_rn(u, __fmaf_rn(u, __fmaf_rn(u, __fmaf_rn(u, c10, c8), c6), c4), c2), 1.0f);
  const bool odd = quarter & 1u;
  c = __uint_as_float(__float_as_uint(g * (odd ? y : x)) ^ ((quarter + 1u) & 2u) << 30);
  s = __uint_as_float(__float_as_uint(g * (odd ? x : y)) ^ (quarter & 2u) << 30);
}

// (a, b) turned: one product and one fused multiply-add each, the same on every path.
__device__ __forceinline__ void rope_turn(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = __fmaf_rn(x, c, -__fmul_rn(y, s));
  b = __fmaf_rn(y, c, __fmul_rn(x, s));
}

// Two pairs at a time: packed fp32 arithmetic, the same roundings.
__device__ __forceinline__ void rope_turn2(float& a0, float& a1, float& b0, float& b1, float c0, float c1, float s0,
                                           float s1) {
  float x0, x1, y0, y1, z0, z1, w0, w1;
  ptx::fmul2(x0, x1, b0, b1, -s0, -s1);
  ptx::fmul2(y0, y1, a0, a1, s0, s1);
  ptx::ffma2(z0, z1, a0, a1, c0, c1, x0, x1);
  ptx::ffma2(w0, w1, b0, b1, c0, c1, y0, y1);
  a0 = z0, a1 = z1, b0 = w0, b1 = w1;
}

// The cosines and sines of a lane's NA pairs where SUBS lanes, LPR apart, need the same
// ones (they hold the same columns of other heads): each works out NA / SUBS and the rest
// comes by shuffles.  pair(e): the number of the lane's e-th pair.  A whole warp.
template <int NA, int LPR, typename F>
__device__ __forceinline__ void rope_angles(const focus_rope& r, int64_t pos, int lane, F&& pair, float (&cs)[NA],
                                            float (&sn)[NA]) {
  constexpr int SUBS = 32 / LPR, OWN = NA / SUBS > 0 ? NA / SUBS : 1;
  static_assert(NA % OWN == 0 && NA / OWN <= SUBS, "each pair has one owner");
  const int sub = lane / LPR, np = r.dim / 2;
  float c[OWN], s[OWN];
#pragma unroll
  for (int k = 0; k < OWN; ++k) {
    int i = np;
#pragma unroll
    for (int e = 0; e < NA; ++e)  // (pair() may index by its argument)
      if (e == (sub * OWN + k) % NA) i = pair(e);
    c[k] = 1.0f, s[k] = 0.0f;
    if (i < np) rope_angle(pos, r.turn[i], r.attn_factor, c[k], s[k]);
  }
#pragma unroll
  for (int e = 0; e < NA; ++e) {
    cs[e] = __shfl_sync(0xffffffffu, c[e % OWN], (e / OWN) * LPR + lane % LPR);
    sn[e] = __shfl_sync(0xffffffffu, s[e % OWN], (e / OWN) * LPR + lane % LPR);
  }
}

template <typename T>
struct RowChunk;  // 16 bytes of a row as V floats

template <>
struct RowChunk<bf16> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void unpack(const uint4& x, float (&f)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float to_float(bf16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ bf16 from_float(float x) { return __float2bfloat16_rn(x); }
};

template <>
struct RowChunk<__half> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void unpack(const uint4& x, float (&f)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 t = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
};

template <>
struct RowChunk<float> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void unpack(const uint4& x, float (&f)[4]) {
    f[0] = __uint_as_float(x.x), f[1] = __uint_as_float(x.y);
    f[2] = __uint_as_float(x.z), f[3] = __uint_as_float(x.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float to_float(float x) { return x; }
  static __device__ __forceinline__ float from_float(float x) { return x; }
};

}  // namespace focus
