// Rotary positions of queries and keys, and their backward pass.
//
// Pair (a, b) of a head at position pos becomes g (a cos - b sin, b cos + a sin) at the
// angle pos f_i (include/focus.h has the layouts and scalings); the backward pass is the
// transposed map, the same kernel with the sine's sign changed.  Memory-bound: each row
// is read once and written once.  The cosines and sines depend on the token only, so a
// warp takes one token, computes them once into registers and applies them to that
// token's heads, queries and keys in one launch.
// Measured: bf16, d = 128: 32K tokens of 32 + 32 heads out of a packed projection 154 us (7.0
// TB/s), the gradients of 128K tokens of 32 + 8 heads 379 us (7.1 TB/s); 16 tokens 3.7 us (the
// launch, the angles and one trip to memory).
#include <math.h>

#include "rope.cuh"

namespace focus {
namespace {

struct RopeArgs {
  focus_rope rope;
  const void *q, *k;
  void *qo, *ko;
  focus_strides qs, ks, qos, kos;
  const int32_t* positions;
  int64_t offset, tokens;  // tokens = B * N
  int N, H, heads;         // heads = H + H_kv
  int splits, per;         // warps per token, heads of each
  int lanes_of;            // several tokens per warp: groups of lanes of a token
  float sign;              // +1 forward, -1 backward
};


// Row (b, n, h) of the head list (queries first, then keys), in elements of T.
template <typename T>
__device__ __forceinline__ void row_of(const RopeArgs& a, int64_t b, int64_t n, int h, const T*& x, T*& y) {
  if (h < a.H) {
    x = reinterpret_cast<const T*>(a.q) + b * a.qs.b + n * a.qs.n + h * a.qs.h;
    y = reinterpret_cast<T*>(a.qo) + b * a.qos.b + n * a.qos.n + h * a.qos.h;
  } else {
    x = reinterpret_cast<const T*>(a.k) + b * a.ks.b + n * a.ks.n + (h - a.H) * a.ks.h;
    y = reinterpret_cast<T*>(a.ko) + b * a.kos.b + n * a.kos.n + (h - a.H) * a.kos.h;
  }
}

// 16-byte chunks of V elements.  A row's D / V chunks belong to D / (2 V) lanes, two
// each, so a warp moves several heads at a time.
//   HALF (dim a multiple of 2 V): lane c < P = dim / 2 / V holds chunks c and c + P, the
//     two halves of its V pairs; the lanes behind hold two chunks that are copied.
//   INTERLEAVED: chunks c and c + D / (2 V), V / 2 pairs each.
// FEW: fewer heads than a warp's RPW rows.  A warp then takes U times RPW / a.lanes_of tokens, a
// lane's group one row of each.  400K bf16 tokens of 1 + 1 heads of 64: 197 us with a warp per
// token, 60 so; of 128: 264 and 124; 3000 tokens, where latency counts: 3.9 and 4.4.
template <typename T, int D, bool HALF, bool FEW>
__global__ void __launch_bounds__(256) rope_rows(const __grid_constant__ RopeArgs a) {
  using C = RowChunk<T>;
  constexpr int V = C::V, LPR = D / (2 * V), RPW = 32 / LPR;
  constexpr int U = 2;  // head groups whose loads are in flight together
  const int64_t warp = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, c = lane % LPR, sub = lane / LPR;
  const int64_t tk = FEW ? 0 : warp / a.splits;
  if (!FEW && tk >= a.tokens) return;
  const int sp = FEW ? 0 : (int)(warp - tk * a.splits);
  const int64_t b = tk / a.N, n = tk - b * a.N;
  const int np = a.rope.dim / 2, P = np / V;
  const bool turned = HALF ? c < P : true;
  const int ca = HALF ? (turned ? c : 2 * P + 2 * (c - P)) : c;
  const int cb = HALF ? (turned ? c + P : ca + 1) : c + LPR;
  float cs[V], sn[V];
  bool rot[V];
  auto pair = [&](int e) { return HALF ? c * V + e : (e < V / 2 ? ca * (V / 2) + e : cb * (V / 2) + e - V / 2); };
#pragma unroll
  for (int e = 0; e < V; ++e) rot[e] = pair(e) < np;
  // Both chunks of a row turned (where they are).
  auto turn = [&](uint4& xa, uint4& xb) {
    if (!turned) return;
    float fa[V], fb[V];
    C::unpack(xa, fa);
    C::unpack(xb, fb);
    if constexpr (HALF) {
#pragma unroll
      for (int e = 0; e < V; ++e) rope_turn(fa[e], fb[e], cs[e], sn[e]);
    } else {
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        if (rot[e]) rope_turn(fa[2 * e], fa[2 * e + 1], cs[e], sn[e]);
        if (rot[e + V / 2]) rope_turn(fb[2 * e], fb[2 * e + 1], cs[e + V / 2], sn[e + V / 2]);
      }
    }
    xa = C::pack(fa);
    xb = C::pack(fb);
  };
  if constexpr (FEW) {
    const int tpw = RPW / a.lanes_of, h = sub & (a.lanes_of - 1);
    uint4 xa[U], xb[U];
    T* y[U];
    int64_t at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = (warp * U + u) * tpw + sub / a.lanes_of;
      y[u] = nullptr;
      at[u] = 0;
      if (k < a.tokens && h < a.heads) {
        const int64_t kb = k / a.N, kn = k - kb * a.N;
        const T* x;
        row_of<T>(a, kb, kn, h, x, y[u]);
        xa[u] = *reinterpret_cast<const uint4*>(x + ca * V);
        xb[u] = *reinterpret_cast<const uint4*>(x + cb * V);
        at[u] = a.positions ? (int64_t)__ldg(a.positions + k) : a.offset + kn;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!y[u]) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        cs[e] = 1.0f, sn[e] = 0.0f;
        if (rot[e]) rope_angle(at[u], a.rope.turn[pair(e)], a.rope.attn_factor, cs[e], sn[e]);
        sn[e] *= a.sign;
      }
      turn(xa[u], xb[u]);
      *reinterpret_cast<uint4*>(y[u] + ca * V) = xa[u];
      *reinterpret_cast<uint4*>(y[u] + cb * V) = xb[u];
    }
    return;
  }
  const int64_t pos = a.positions ? (int64_t)__ldg(a.positions + tk) : a.offset + n;
  rope_angles<V, LPR>(a.rope, pos, lane, pair, cs, sn);
#pragma unroll
  for (int e = 0; e < V; ++e) sn[e] *= a.sign;
  const int h1 = min(a.heads, (sp + 1) * a.per);
  for (int h0 = sp * a.per + sub; h0 < h1; h0 += U * RPW) {
    uint4 xa[U], xb[U];
    T* y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h0 + u * RPW < h1) {
        const T* x;
        row_of<T>(a, b, n, h0 + u * RPW, x, y[u]);
        xa[u] = *reinterpret_cast<const uint4*>(x + ca * V);
        xb[u] = *reinterpret_cast<const uint4*>(x + cb * V);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h0 + u * RPW >= h1) continue;
      turn(xa[u], xb[u]);
      *reinterpret_cast<uint4*>(y[u] + ca * V) = xa[u];
      *reinterpret_cast<uint4*>(y[u] + cb * V) = xb[u];
    }
  }
}

// Any alignment and any even dim: one element at a time.  A row's D / 2 slots (its dim / 2
// pairs, then the remaining columns two by two) go to the 32 lanes.
template <typename T, int D>
__global__ void __launch_bounds__(256) rope_elems(const __grid_constant__ RopeArgs a) {
  using C = RowChunk<T>;
  constexpr int S = D / 64, U = 4;
  const int64_t warp = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t tk = warp / a.splits;
  if (tk >= a.tokens) return;
  const int sp = (int)(warp - tk * a.splits), lane = threadIdx.x & 31;
  const int64_t b = tk / a.N, n = tk - b * a.N;
  const int64_t pos = a.positions ? (int64_t)__ldg(a.positions + tk) : a.offset + n;
  const int np = a.rope.dim / 2;
  const bool half = a.rope.layout == FOCUS_ROPE_HALF;
  float cs[S], sn[S];
  int ia[S], ib[S];
  bool rot[S];
#pragma unroll
  for (int k = 0; k < S; ++k) {
    const int i = lane + 32 * k;
    rot[k] = i < np;
    ia[k] = rot[k] && half ? i : 2 * i;
    ib[k] = rot[k] && half ? i + np : 2 * i + 1;
    cs[k] = 1.0f, sn[k] = 0.0f;
    if (rot[k]) rope_angle(pos, a.rope.turn[i], a.rope.attn_factor, cs[k], sn[k]);
    sn[k] *= a.sign;
  }
  const int h1 = min(a.heads, (sp + 1) * a.per);
  for (int h0 = sp * a.per; h0 < h1; h0 += U) {
    T xa[U][S], xb[U][S], *y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h0 + u >= h1) continue;
      const T* x;
      row_of<T>(a, b, n, h0 + u, x, y[u]);
#pragma unroll
      for (int k = 0; k < S; ++k) xa[u][k] = x[ia[k]], xb[u][k] = x[ib[k]];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h0 + u >= h1) continue;
#pragma unroll
      for (int k = 0; k < S; ++k) {
        if (rot[k]) {
          float s = C::to_float(xa[u][k]), t = C::to_float(xb[u][k]);
          rope_turn(s, t, cs[k], sn[k]);
          xa[u][k] = C::from_float(s);
          xb[u][k] = C::from_float(t);
        }
        y[u][ia[k]] = xa[u][k];
        y[u][ib[k]] = xb[u][k];
      }
    }
  }
}

bool chunked(const void* p, const focus_strides& s, int size) {
  return ((uintptr_t)p | (uintptr_t)(s.b * size) | (uintptr_t)(s.n * size) | (uintptr_t)(s.h * size)) % 16 == 0;
}

constexpr int kRopeWarps = 2432;  // warps that fill the GPU: 16 per SM on 152 SMs (8 or 32: the same)

template <typename T, int D>
cudaError_t launch(RopeArgs& a, bool chunks, cudaStream_t s) {
  constexpr int V = RowChunk<T>::V, RPW = 64 * V / D;
  const bool half = a.rope.layout == FOCUS_ROPE_HALF;
  a.lanes_of = 1;
  while (a.lanes_of < a.heads && a.lanes_of < RPW) a.lanes_of *= 2;
  if (chunks && a.lanes_of < RPW && a.tokens > 2 * kRopeWarps) {
    const int64_t per = 8 * 2 * (RPW / a.lanes_of), blocks = (a.tokens + per - 1) / per;  // tokens of a block
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (half) rope_rows<T, D, true, true><<<(unsigned)blocks, 256, 0, s>>>(a);
    else rope_rows<T, D, false, true><<<(unsigned)blocks, 256, 0, s>>>(a);
    return cudaGetLastError();
  }
  // few tokens: several warps share a token's heads, each computing the angles anew (16 tokens of
  // 40 heads: 3.7 us, with one warp per token 7.1)
  const int step = chunks ? RPW : 1;
  const int most = (a.heads + step - 1) / step;
  const int64_t want = (kRopeWarps + a.tokens - 1) / a.tokens;
  a.splits = (int)(want < most ? want : most);
  a.per = ((a.heads + a.splits - 1) / a.splits + step - 1) / step * step;
  a.splits = (a.heads + a.per - 1) / a.per;
  const int64_t blocks = (a.tokens * a.splits + 7) / 8;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const unsigned g = (unsigned)blocks;
  if (!chunks)
    rope_elems<T, D><<<g, 256, 0, s>>>(a);
  else if (half)
    rope_rows<T, D, true, false><<<g, 256, 0, s>>>(a);
  else
    rope_rows<T, D, false, false><<<g, 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_d(RopeArgs& a, int d, bool chunks, cudaStream_t s) {
  return d == 64 ? launch<T, 64>(a, chunks, s) : launch<T, 128>(a, chunks, s);
}

}  // namespace

int rope_check(const focus_rope* r, int d_head) {
  if (r->dim < 2 || r->dim % 2 || r->dim > d_head) return FOCUS_ERR_INVALID_ARG;
  if (r->layout != FOCUS_ROPE_HALF && r->layout != FOCUS_ROPE_INTERLEAVED) return FOCUS_ERR_INVALID_ARG;
  return FOCUS_OK;
}

cudaError_t launch_rope(const focus_rope& rope, int dtype, int B, int N, int H, int H_kv, int d,
                        const void* q, const focus_strides& qs, const void* k, const focus_strides& ks,
                        const int32_t* positions, int64_t offset, bool inverse, void* qo,
                        const focus_strides& qos, void* ko, const focus_strides& kos, cudaStream_t s) {
  RopeArgs a;
  a.rope = rope;
  a.q = q, a.k = k, a.qo = qo, a.ko = ko;
  a.qs = qs, a.ks = ks, a.qos = qos, a.kos = kos;
  a.positions = positions;
  a.offset = offset;
  a.tokens = (int64_t)B * N;
  a.N = N, a.H = H, a.heads = H + H_kv;
  a.sign = inverse ? -1.0f : 1.0f;
  const int size = dtype == FOCUS_DTYPE_F32 ? 4 : 2;
  const bool chunks = (rope.layout != FOCUS_ROPE_HALF || rope.dim % (32 / size) == 0) &&
                      chunked(q, qs, size) && chunked(qo, qos, size) &&
                      (!H_kv || (chunked(k, ks, size) && chunked(ko, kos, size)));
  if (dtype == FOCUS_DTYPE_F32) return launch_d<float>(a, d, chunks, s);
  if (dtype == FOCUS_DTYPE_F16) return launch_d<__half>(a, d, chunks, s);
  return launch_d<bf16>(a, d, chunks, s);
}

namespace {

// Sums of two doubles, about 106 bits: the plan's frequencies are needed to 2^-64 of a turn.
struct Twice {
  double h, l;
};
Twice sum(double a, double b) {  // exact
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
Twice operator+(Twice a, Twice b) {
  const Twice s = sum(a.h, b.h);
  return sum(s.h, s.l + (a.l + b.l));
}
Twice operator-(Twice a, Twice b) { return a + Twice{-b.h, -b.l}; }
Twice operator*(Twice a, Twice b) {
  const double p = a.h * b.h;
  return sum(p, fma(a.h, b.h, -p) + (a.h * b.l + a.l * b.h));
}
Twice operator/(Twice a, Twice b) {  // a quotient, and that of what it leaves
  const Twice q{a.h / b.h, 0.0}, r = a - b * q;
  const Twice q2{r.h / b.h, 0.0}, r2 = r - b * q2;
  return q + q2 + Twice{r2.h / b.h, 0.0};
}
// x^(-1/k), x >= 1: Newton's step for y^-k = x, which doubles the digits, from the library's value.
Twice root(Twice x, int k) {
  Twice y{pow(x.h, -1.0 / k), 0.0};
  for (int step = 0; step < 2; ++step) {
    Twice power{1.0, 0.0}, square = y;
    for (int n = k; n; n >>= 1, square = square * square)
      if (n & 1) power = power * square;
    y = y + y * (Twice{1.0, 0.0} - x * power) / Twice{(double)k, 0.0};
  }
  return y;
}

}  // namespace

int rope_plan(const focus_rope_params& p, focus_rope* out) {
  if (p.dim < 2 || p.dim % 2 || p.dim > 128) return FOCUS_ERR_INVALID_ARG;
  if (p.layout != FOCUS_ROPE_HALF && p.layout != FOCUS_ROPE_INTERLEAVED) return FOCUS_ERR_INVALID_ARG;
  if (p.scaling < FOCUS_ROPE_SCALING_NONE || p.scaling > FOCUS_ROPE_SCALING_BY_PARTS)
    return FOCUS_ERR_INVALID_ARG;
  if (!(p.base >= 1.0) || !isfinite(p.base) || !isfinite(p.attn_factor)) return FOCUS_ERR_INVALID_ARG;
  const bool scaled = p.scaling != FOCUS_ROPE_SCALING_NONE;
  if (scaled && (!(p.factor >= 1.0) || !isfinite(p.factor))) return FOCUS_ERR_INVALID_ARG;
  const bool parts = p.scaling == FOCUS_ROPE_SCALING_BY_PARTS;
  if (parts && (p.orig_len < 1 || !(p.beta_slow >= 0.0) || !(p.beta_fast > p.beta_slow) ||
                !isfinite(p.beta_fast)))
    return FOCUS_ERR_INVALID_ARG;
  const Twice two_pi{6.283185307179586, 2.4492935982947064e-16}, one{1.0, 0.0};
  const Twice factor{p.factor, 0.0};
  Twice base{p.base, 0.0};
  // factor^(dim / (dim - 2)); dim = 2 has pair 0 alone, which no base stretches
  if (p.scaling == FOCUS_ROPE_SCALING_NTK && p.dim > 2) base = base * factor / root(factor, (p.dim - 2) / 2);
  const Twice ratio = root(base, p.dim / 2);  // f_i = ratio^i
  out->dim = p.dim;
  out->layout = p.layout;
  out->reserved = 0;
  out->attn_factor =
      (float)(p.attn_factor > 0.0 ? p.attn_factor : parts ? 0.1 * log(p.factor) + 1.0 : 1.0);
  Twice power = one;
  for (int i = 0; i < 64; ++i) {
    out->turn[i] = 0;
    if (i >= p.dim / 2) continue;
    Twice f = power;
    power = power * ratio;
    if (p.scaling == FOCUS_ROPE_SCALING_LINEAR) f = f / factor;
    if (parts) {
      const Twice turns = Twice{(double)p.orig_len, 0.0} * f / two_pi;
      Twice keep = (turns - Twice{p.beta_slow, 0.0}) / sum(p.beta_fast, -p.beta_slow);
      if (keep.h < 0.0) keep = Twice{0.0, 0.0};
      if (keep.h >= 1.0) keep = one;
      f = f * (one - keep) / factor + f * keep;
    }
    // f <= 1: a turn below 2^62; its whole part, and the rest rounded
    const Twice t = f / two_pi;
    const double high = t.h * 18446744073709551616.0, whole = floor(high);
    out->turn[i] = (uint64_t)whole + (uint64_t)llrint((high - whole) + t.l * 18446744073709551616.0);
  }
  return FOCUS_OK;
}

}  // namespace focus
