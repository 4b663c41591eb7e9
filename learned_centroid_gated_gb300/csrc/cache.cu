// Key/value cache: tokens written (rotated, quantised, scattered to their slots with
// their group masks) and read back as bf16.
//
// A row is one token's key or value of one head.  8-bit formats hold it as codes with one
// scale, max|x| / M: c = round(x M / max|x|), x ~ c max|x| / M with M = 448 (e4m3) or 127
// (int8).  Memory-bound: each bf16 row is read once, its codes written once.  A warp takes
// one token: a key's cosines and sines are computed once and serve all KV heads, the row
// maximum is a shuffle over the row's D / 16 lanes, and the codes leave from registers.
// Measured, e4m3, d = 128: 32K tokens of 32 KV heads written with rotation, 134 us (6.1 TB/s;
// after the memory come the instructions, 0.59 of the issue slots), in bf16 158 us (6.8 TB/s); 128K
// tokens of 8 KV heads read back, 116 us (7.0 TB/s); one token of each of 32 sequences, 4.2 us,
// which is the launch and three dependent reads.
#include <cuda_fp8.h>
#include <math.h>

#include <type_traits>

#include "rope.cuh"

namespace focus {
namespace {

constexpr float kTinyRow = 7.888609052210118e-31f;  // 2^-100: below it M / max|x| nears fp32's end

enum RopeMode { kNoRope = 0, kHalf = 1, kInterleaved = 2, kHalfAny = 3 };

struct CacheArgs {
  focus_rope rope;
  const uint16_t *k, *v;
  focus_strides ks, vs;
  const uint32_t* mask;
  const int32_t *start, *count, *positions;
  void *kc, *vc;
  float *kscale, *vscale;
  uint32_t* mc;
  uint16_t *ko, *vo;  // cache_read's outputs
  int32_t* status;
  int64_t tokens;     // B * T
  int T, cap, H_kv, R, splits, per;
  int lanes_of;       // cache_write, several tokens per warp: groups of lanes of a token
};

// Slot of token t of sequence b; -1 when it is not to be moved.  A slot outside the cache
// or a count outside [0, T] raises FOCUS_ERR_BOUNDS.
__device__ __forceinline__ int slot_of(const CacheArgs& a, int b, int t, bool report) {
  const int64_t first = a.start ? (int64_t)__ldg(a.start + b) : 0;
  const int n = a.count ? __ldg(a.count + b) : a.T;
  bool bad = n < 0 || n > a.T;
  int64_t slot = -1;
  if (t < n) {
    slot = first + t;
    if (slot < 0 || slot >= a.cap) {
      bad = true;
      slot = -1;
    }
  }
  if (bad && report && a.status) raise_status(a.status, FOCUS_ERR_BOUNDS);
  return (int)slot;
}

template <int FMT>
__device__ __forceinline__ uint2 encode(const float (&f)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float* x = f + 4 * i;
    if constexpr (FMT == FOCUS_CACHE_E4M3) {
      float y[4];
      ptx::fmul2(y[0], y[1], x[0], x[1], inv, inv);
      ptx::fmul2(y[2], y[3], x[2], x[3], inv, inv);
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
      w[i] = __byte_perm(lo, hi, 0x5410);
    } else {
      // 1.5 * 2^23 + c has the integer c, rounded to nearest even, in its low bits
      float y[4];
      ptx::ffma2(y[0], y[1], x[0], x[1], inv, inv, 12582912.0f, 12582912.0f);
      ptx::ffma2(y[2], y[3], x[2], x[3], inv, inv, 12582912.0f, 12582912.0f);
      const uint32_t u[4] = {__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3])};
      w[i] = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
    }
  }
  return make_uint2(w[0], w[1]);
}

// The larger of three magnitudes, a NaN if there is one.
__device__ __forceinline__ float abs_max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return d;
}

template <int FMT>
__device__ __forceinline__ void decode8(const uint2& x, float scale, float (&f)[8]) {
  const uint32_t w[2] = {x.x, x.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = (w[i >> 1] >> (16 * (i & 1))) & 0xffffu;
    if constexpr (FMT == FOCUS_CACHE_E4M3) {
      const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h, __NV_E4M3);
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&r));
      f[2 * i] = t.x * scale;
      f[2 * i + 1] = t.y * scale;
    } else {
      f[2 * i] = (float)(int)(int8_t)(h & 0xffu) * scale;
      f[2 * i + 1] = (float)(int)(int8_t)(h >> 8) * scale;
    }
  }
}

// Lane c of a row's D / 16 lanes holds two 8-element chunks (ca, cb).  With kHalf
// (dim a multiple of 16) they are the two halves of eight pairs, with kInterleaved each
// holds four pairs, and with kHalfAny (any other even dim) the partner of each element is
// read from the row (a cached read: the row's other lanes load it too).
//
// FEW: fewer KV heads than a warp's 32 / (D / 16) rows.  A warp then takes several tokens,
// a.lanes_of of those row places each (a power of two, at least H_kv); keys and values are in
// flight together.  4 sequences of up to 175K int8 tokens, one head of 64: 446 us with a warp per token,
// 60 so; 200K e4m3 tokens of two heads of 128: 216 and 103; 32 tokens: 5.7 both.
template <int D, int FMT, int MODE, bool FEW>
__global__ void __launch_bounds__(256, MODE == kHalfAny ? 3 : 4) cache_write(const __grid_constant__ CacheArgs a) {
  using C = RowChunk<bf16>;
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  const int64_t warp = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, c = lane % LPR, sub = lane / LPR;
  const int h_few = FEW ? sub & (a.lanes_of - 1) : 0;
  const int64_t tk = FEW ? warp * (RPW / a.lanes_of) + sub / a.lanes_of : warp / a.splits;
  if (!FEW && tk >= a.tokens) return;
  const int sp = FEW ? 0 : (int)(warp - tk * a.splits);
  const bool there = !FEW || tk < a.tokens;
  const int b = there ? (int)(tk / a.T) : 0, t = there ? (int)(tk - (int64_t)b * a.T) : 0;
  const int slot = there ? slot_of(a, b, t, FEW ? c == 0 && h_few == 0 : lane == 0) : -1;
  if (FEW ? !__any_sync(0xffffffffu, slot >= 0) : slot < 0) return;
  if (sp == 0 && a.mask && slot >= 0)
    for (int r = FEW ? h_few * LPR + c : lane; r < a.R; r += FEW ? a.lanes_of * LPR : 32)
      a.mc[((int64_t)b * a.R + r) * a.cap + slot] = a.mask[((int64_t)b * a.R + r) * a.T + t];
  const int np = a.rope.dim / 2, P = np / 8;
  const bool pair = MODE == kHalf && c < P;
  const int ca = MODE == kHalf && !pair ? 2 * P + 2 * (c - P) : c;
  const int cb = MODE == kHalf ? (pair ? c + P : ca + 1) : c + LPR;
  const int i0 = sp * a.per, i1 = min(2 * a.H_kv, i0 + a.per);  // rows: keys, then values
  constexpr int NA = MODE == kHalfAny ? 16 : 8;
  float cs[NA], sn[NA];
  if constexpr (MODE != kNoRope) {
    auto pair_of = [&](int e) {
      if (MODE == kHalf) return c * 8 + e;
      if (MODE == kInterleaved) return (e < 4 ? ca : cb) * 4 + (e & 3);
      const int x = (e < 8 ? ca : cb) * 8 + (e & 7);
      return x < np ? x : x < 2 * np ? x - np : np;
    };
    if (FEW || i0 < a.H_kv) {
      const int64_t pos = a.positions ? (there ? (int64_t)__ldg(a.positions + tk) : 0) : (int64_t)slot;
      if constexpr (FEW) {
#pragma unroll
        for (int e = 0; e < NA; ++e) {
          const int i = pair_of(e);
          cs[e] = 1.0f, sn[e] = 0.0f;
          if (i < np) rope_angle(pos, a.rope.turn[i], a.rope.attn_factor, cs[e], sn[e]);
        }
      } else {
        rope_angles<NA, LPR>(a.rope, pos, lane, pair_of, cs, sn);
      }
    }
  }
  // One row (of the keys or of the values): its two chunks of each lane, whether it is there, its
  // place in the cache.  Every lane takes part, since the row maximum is a shuffle.
  constexpr int ES = FMT == FOCUS_CACHE_BF16 ? 2 : 1;
  auto put = [&](auto is_key, const uint4& xa, const uint4& xb, const bf16* xr, bool on, char* y, float* scale) {
    constexpr bool KEY = decltype(is_key)::value;
    float mx = 0.0f;
    if constexpr (!KEY && FMT != FOCUS_CACHE_BF16) {
      // magnitudes as 16-bit integers, two at a time; infinities and NaN are the largest
      uint32_t m = 0u;
      const uint32_t w[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) m = __vmaxu2(m, w[e] & 0x7fff7fffu);
      mx = __uint_as_float(max(m << 16, m & 0xffff0000u));
    }
    float fa[8], fb[8];
    C::unpack(xa, fa);
    C::unpack(xb, fb);
    if constexpr (KEY && MODE == kHalf) {
      if (pair) {
#pragma unroll
        for (int e = 0; e < 8; e += 2)
          rope_turn2(fa[e], fa[e + 1], fb[e], fb[e + 1], cs[e], cs[e + 1], sn[e], sn[e + 1]);
      }
    } else if constexpr (KEY && MODE == kInterleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (ca * 4 + e < np) rope_turn(fa[2 * e], fa[2 * e + 1], cs[e], sn[e]);
        if (cb * 4 + e < np) rope_turn(fb[2 * e], fb[2 * e + 1], cs[4 + e], sn[4 + e]);
      }
    } else if constexpr (KEY && MODE == kHalfAny) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int i = (e < 8 ? ca : cb) * 8 + (e & 7);
        if (i < 2 * np && on) {
          float& f = e < 8 ? fa[e & 7] : fb[e & 7];
          float o = __bfloat162float(xr[i < np ? i + np : i - np]);
          if (i < np) rope_turn(f, o, cs[e], sn[e]);
          else rope_turn(o, f, cs[e], sn[e]);
        }
      }
    }
    if constexpr (FMT == FOCUS_CACHE_BF16) {
      if (on) {
        *reinterpret_cast<uint4*>(y + 16 * ca) = C::pack(fa);
        *reinterpret_cast<uint4*>(y + 16 * cb) = C::pack(fb);
      }
    } else {
      constexpr float M = FMT == FOCUS_CACHE_E4M3 ? 448.0f : 127.0f;
      if constexpr (KEY) {
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = abs_max3(mx, fa[e], fb[e]);
      }
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) mx = abs_max3(mx, __shfl_xor_sync(0xffffffffu, mx, o), 0.0f);
      const bool finite = mx < INFINITY, some = finite && mx >= kTinyRow;
      const float inv = some ? M / mx : 0.0f;
      if (on) {
        const uint2 zero = make_uint2(0u, 0u);
        *reinterpret_cast<uint2*>(y + 8 * ca) = some ? encode<FMT>(fa, inv) : zero;
        *reinterpret_cast<uint2*>(y + 8 * cb) = some ? encode<FMT>(fb, inv) : zero;
        if (c == 0)
          *scale =
              some ? mx * (1.0f / M) : finite ? 0.0f : __uint_as_float(0x7fc00000u);
      }
    }
  };
  if constexpr (FEW) {
    const bool on = slot >= 0 && h_few < a.H_kv;
    const bf16* x = reinterpret_cast<const bf16*>(a.k) + b * a.ks.b + t * a.ks.n + h_few * a.ks.h;
    const bf16* y = reinterpret_cast<const bf16*>(a.v) + b * a.vs.b + t * a.vs.n + h_few * a.vs.h;
    uint4 in[4] = {};
    if (on) {
      in[0] = __ldg(reinterpret_cast<const uint4*>(x + 8 * ca));
      in[1] = __ldg(reinterpret_cast<const uint4*>(x + 8 * cb));
      in[2] = __ldg(reinterpret_cast<const uint4*>(y + 8 * ca));
      in[3] = __ldg(reinterpret_cast<const uint4*>(y + 8 * cb));
    }
    const int64_t to = (((int64_t)b * a.cap + slot) * a.H_kv + h_few) * (D * ES);
    const int64_t sc = ((int64_t)b * a.H_kv + h_few) * a.cap + slot;
    put(std::true_type{}, in[0], in[1], x, on, reinterpret_cast<char*>(a.kc) + to, a.kscale + sc);
    put(std::false_type{}, in[2], in[3], y, on, reinterpret_cast<char*>(a.vc) + to, a.vscale + sc);
    return;
  }
  // Rows h0 .. h1 - 1 of the keys or of the values.  Every lane takes part in every pass (the
  // row maximum is a shuffle); rows past the end are not loaded or stored.  The loads of two
  // passes are in flight together, and four blocks on an SM (the prompt above, then
  // 136 us: one pass 152, four 149, three blocks 149).
  auto rows = [&](auto is_key, const uint16_t* src, const focus_strides& st, void* cache, float* scale, int h0, int h1) {
    constexpr int U = 2;
    const bf16* x = reinterpret_cast<const bf16*>(src) + b * st.b + t * st.n + (h0 + sub) * st.h;
    const int64_t step = RPW * st.h;
    char* dst = reinterpret_cast<char*>(cache) + (((int64_t)b * a.cap + slot) * a.H_kv + h0 + sub) * (D * ES);
    for (int h = h0; h < h1; h += U * RPW) {
      uint4 xa[U], xb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        xa[u] = xb[u] = make_uint4(0u, 0u, 0u, 0u);
        if (h + u * RPW + sub < h1) {
          xa[u] = __ldg(reinterpret_cast<const uint4*>(x + u * step + 8 * ca));
          xb[u] = __ldg(reinterpret_cast<const uint4*>(x + u * step + 8 * cb));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h + u * RPW >= h1) break;
        const int row = h + u * RPW + sub;
        put(is_key, xa[u], xb[u], x + u * step, row < h1, dst + u * RPW * (D * ES),
            scale + ((int64_t)b * a.H_kv + row) * a.cap + slot);
      }
      x += U * step;
      dst += U * RPW * (D * ES);
    }
  };
  if (i0 < a.H_kv) rows(std::true_type{}, a.k, a.ks, a.kc, a.kscale, i0, min(i1, a.H_kv));
  if (i1 > a.H_kv) rows(std::false_type{}, a.v, a.vs, a.vc, a.vscale, max(i0, a.H_kv) - a.H_kv, i1 - a.H_kv);
}

template <int D, int FMT>
__global__ void __launch_bounds__(256) cache_read(const __grid_constant__ CacheArgs a) {
  using C = RowChunk<bf16>;
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = 4;
  const int64_t warp = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t tk = warp / a.splits;
  if (tk >= a.tokens) return;
  const int sp = (int)(warp - tk * a.splits);
  const int lane = threadIdx.x & 31, c = lane % LPR, sub = lane / LPR;
  const int b = (int)(tk / a.T), t = (int)(tk - (int64_t)b * a.T);
  const int slot = slot_of(a, b, t, lane == 0);
  const int i0 = sp * a.per, i1 = min(2 * a.H_kv, i0 + a.per);
  for (int p0 = i0 + sub; p0 < i1; p0 += U * RPW) {
    uint4 x[U];
    float sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = p0 + u * RPW;
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      sc[u] = 0.0f;
      if (row < i1 && slot >= 0) {
        const bool key = row < a.H_kv;
        const int h = key ? row : row - a.H_kv;
        const char* src = reinterpret_cast<const char*>(key ? a.kc : a.vc);
        const int64_t at = (((int64_t)b * a.cap + slot) * a.H_kv + h) * D + 8 * c;
        if constexpr (FMT == FOCUS_CACHE_BF16) {
          x[u] = __ldg(reinterpret_cast<const uint4*>(src + 2 * at));
        } else {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(src + at));
          x[u].x = w.x, x[u].y = w.y;
          sc[u] = __ldg((key ? a.kscale : a.vscale) + ((int64_t)b * a.H_kv + h) * a.cap + slot);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = p0 + u * RPW;
      if (row >= i1) continue;
      const bool key = row < a.H_kv;
      const int h = key ? row : row - a.H_kv;
      if constexpr (FMT != FOCUS_CACHE_BF16) {
        float f[8];
        decode8<FMT>(make_uint2(x[u].x, x[u].y), sc[u], f);
        x[u] = slot >= 0 ? C::pack(f) : make_uint4(0u, 0u, 0u, 0u);
      }
      uint16_t* y = key ? a.ko : a.vo;
      *reinterpret_cast<uint4*>(y + (tk * a.H_kv + h) * D + 8 * c) = x[u];
    }
  }
}

// The same for many tokens whose rows fill a warp's places less than twice: all rows of all
// tokens in a row, U * RPW of them to a warp.  400K tokens, one head of 64: bf16 33 us, int8 44
// (a warp per token 111 both); three heads of 64: 94 and 125 (123 and 139); four: 124 and 166 (130
// and 141).  40 tokens of one head: 3.6 to 3.9 us, with a warp per token 3.0.
template <int D, int FMT>
__global__ void __launch_bounds__(256) cache_read_few(const __grid_constant__ CacheArgs a) {
  using C = RowChunk<bf16>;
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = 4;
  const int64_t warp = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, c = lane % LPR, sub = lane / LPR, rows = 2 * a.H_kv;
  const int64_t tk0 = warp * (U * RPW) / rows, b0 = tk0 / a.T;
  const int row0 = (int)(warp * (U * RPW) - tk0 * rows), t0 = (int)(tk0 - b0 * a.T);
  uint4 x[U];
  float sc[U];
  uint16_t* y[U];
  int slot[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int p = row0 + u * RPW + sub, dt = p / rows, row = p - dt * rows, db = (int)((uint32_t)(t0 + dt) / (uint32_t)a.T);
    const int64_t tk = tk0 + dt;
    x[u] = make_uint4(0u, 0u, 0u, 0u);
    sc[u] = 0.0f;
    y[u] = nullptr;
    slot[u] = -1;
    if (tk < a.tokens) {
      const int b = (int)b0 + db, t = t0 + dt - db * a.T;
      const bool key = row < a.H_kv;
      const int h = key ? row : row - a.H_kv;
      slot[u] = slot_of(a, b, t, c == 0 && row == 0);
      y[u] = (key ? a.ko : a.vo) + (tk * a.H_kv + h) * D + 8 * c;
      if (slot[u] >= 0) {
        const char* src = reinterpret_cast<const char*>(key ? a.kc : a.vc);
        const int64_t at = (((int64_t)b * a.cap + slot[u]) * a.H_kv + h) * D + 8 * c;
        if constexpr (FMT == FOCUS_CACHE_BF16) {
          x[u] = __ldg(reinterpret_cast<const uint4*>(src + 2 * at));
        } else {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(src + at));
          x[u].x = w.x, x[u].y = w.y;
          sc[u] = __ldg((key ? a.kscale : a.vscale) + ((int64_t)b * a.H_kv + h) * a.cap + slot[u]);
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!y[u]) continue;
    if constexpr (FMT != FOCUS_CACHE_BF16) {
      float f[8];
      decode8<FMT>(make_uint2(x[u].x, x[u].y), sc[u], f);
      x[u] = slot[u] >= 0 ? C::pack(f) : make_uint4(0u, 0u, 0u, 0u);
    }
    *reinterpret_cast<uint4*>(y[u]) = x[u];
  }
}

// Warps that fill the GPU: 16 per SM on 152 SMs (8: the same 4.2 us for one token of each of
// 32 sequences, 32: 4.9).
constexpr int kCacheWarps = 2432;

// Warps per token and rows (of the 2 H_kv) of each: one warp, or for few tokens several (the
// same 32 tokens with one warp each: 6.2 us).
unsigned split_rows(CacheArgs& a, int step) {
  const int rows = 2 * a.H_kv, most = (rows + step - 1) / step;
  const int64_t want = (kCacheWarps + a.tokens - 1) / a.tokens;
  a.splits = (int)(want < most ? want : most);
  a.per = ((rows + a.splits - 1) / a.splits + step - 1) / step * step;
  a.splits = (rows + a.per - 1) / a.per;
  const int64_t blocks = (a.tokens * a.splits + 7) / 8;
  return blocks > INT32_MAX ? 0u : (unsigned)blocks;
}

template <int D, int FMT, bool FEW>
cudaError_t write_mode(const CacheArgs& a, int mode, unsigned g, cudaStream_t s) {
  switch (mode) {
    case kNoRope: cache_write<D, FMT, kNoRope, FEW><<<g, 256, 0, s>>>(a); break;
    case kHalf: cache_write<D, FMT, kHalf, FEW><<<g, 256, 0, s>>>(a); break;
    case kInterleaved: cache_write<D, FMT, kInterleaved, FEW><<<g, 256, 0, s>>>(a); break;
    default: cache_write<D, FMT, kHalfAny, FEW><<<g, 256, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <int D, int FMT>
cudaError_t write_d(CacheArgs& a, int mode, cudaStream_t s) {
  constexpr int RPW = 512 / D;
  a.lanes_of = 1;
  while (a.lanes_of < a.H_kv && a.lanes_of < RPW) a.lanes_of *= 2;
  if (a.lanes_of < RPW) {
    const int64_t blocks = (a.tokens + RPW / a.lanes_of * 8 - 1) / (RPW / a.lanes_of * 8);
    return blocks > INT32_MAX ? cudaErrorInvalidConfiguration : write_mode<D, FMT, true>(a, mode, (unsigned)blocks, s);
  }
  const unsigned g = split_rows(a, RPW);
  return g ? write_mode<D, FMT, false>(a, mode, g, s) : cudaErrorInvalidConfiguration;
}

template <int D, int FMT>
cudaError_t read_d(CacheArgs& a, cudaStream_t s) {
  if (2 * a.H_kv < 512 / D && a.tokens > kCacheWarps) {
    constexpr int PER = 8 * 4 * 256 / D;  // rows of a block
    const int64_t blocks = (a.tokens * 2 * a.H_kv + PER - 1) / PER;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    cache_read_few<D, FMT><<<(unsigned)blocks, 256, 0, s>>>(a);
    return cudaGetLastError();
  }
  const unsigned g = split_rows(a, 256 / D);
  if (!g) return cudaErrorInvalidConfiguration;
  cache_read<D, FMT><<<g, 256, 0, s>>>(a);
  return cudaGetLastError();
}

CacheArgs args_of(const focus_cache_params& p, const int32_t* start, const int32_t* count, int32_t* status) {
  CacheArgs a{};
  a.start = start, a.count = count, a.status = status;
  a.tokens = (int64_t)p.B * p.T;
  a.T = p.T, a.cap = p.cap, a.H_kv = p.H_kv, a.R = p.R;
  return a;
}

}  // namespace

cudaError_t launch_cache_write(const focus_cache_params& p, const uint16_t* k, const focus_strides& ks,
                               const uint16_t* v, const focus_strides& vs, const uint32_t* mask,
                               const int32_t* start, const int32_t* count, const focus_rope* rope,
                               const int32_t* positions, void* kc, void* vc, float* kscale,
                               float* vscale, uint32_t* mc, int32_t* status, cudaStream_t s) {
  CacheArgs a = args_of(p, start, count, status);
  a.k = k, a.v = v, a.ks = ks, a.vs = vs, a.mask = mask, a.positions = positions;
  a.kc = kc, a.vc = vc, a.kscale = kscale, a.vscale = vscale, a.mc = mc;
  int mode = kNoRope;
  if (rope) {
    a.rope = *rope;
    mode = rope->layout == FOCUS_ROPE_INTERLEAVED ? kInterleaved : rope->dim % 16 == 0 ? kHalf : kHalfAny;
  }
  if (p.d_head == 64)
    return p.format == FOCUS_CACHE_BF16   ? write_d<64, FOCUS_CACHE_BF16>(a, mode, s)
           : p.format == FOCUS_CACHE_E4M3 ? write_d<64, FOCUS_CACHE_E4M3>(a, mode, s)
                                          : write_d<64, FOCUS_CACHE_INT8>(a, mode, s);
  return p.format == FOCUS_CACHE_BF16   ? write_d<128, FOCUS_CACHE_BF16>(a, mode, s)
         : p.format == FOCUS_CACHE_E4M3 ? write_d<128, FOCUS_CACHE_E4M3>(a, mode, s)
                                        : write_d<128, FOCUS_CACHE_INT8>(a, mode, s);
}

cudaError_t launch_cache_read(const focus_cache_params& p, const void* kc, const void* vc,
                              const float* kscale, const float* vscale, const int32_t* start,
                              const int32_t* count, uint16_t* k, uint16_t* v, int32_t* status,
                              cudaStream_t s) {
  CacheArgs a = args_of(p, start, count, status);
  a.kc = const_cast<void*>(kc), a.vc = const_cast<void*>(vc);
  a.kscale = const_cast<float*>(kscale), a.vscale = const_cast<float*>(vscale);
  a.ko = k, a.vo = v;
  if (p.d_head == 64)
    return p.format == FOCUS_CACHE_BF16   ? read_d<64, FOCUS_CACHE_BF16>(a, s)
           : p.format == FOCUS_CACHE_E4M3 ? read_d<64, FOCUS_CACHE_E4M3>(a, s)
                                          : read_d<64, FOCUS_CACHE_INT8>(a, s);
  return p.format == FOCUS_CACHE_BF16   ? read_d<128, FOCUS_CACHE_BF16>(a, s)
         : p.format == FOCUS_CACHE_E4M3 ? read_d<128, FOCUS_CACHE_E4M3>(a, s)
                                        : read_d<128, FOCUS_CACHE_INT8>(a, s);
}

}  // namespace focus
