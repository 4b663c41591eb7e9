// Decode of drafted tokens over a cache: what its two kernels (tree.cu, tree_tc.cu) share.
// Parameters, the row of work units that is cut into slices, the draft tree's words.
#pragma once

#include <cuda_fp8.h>
#include <limits.h>

#include "common.cuh"

namespace focus {

constexpr int kTreeUnit = 32;        // keys per unit of work
constexpr int kTreeNear = 64;        // weight of a unit near the window
// 8-bit formats: V scales count as at least 2^-80 where the reference of O is chosen, so that it
// stays within 2^113 of that of the logits and the factor between them is a normal number.
constexpr float kTinyScale = 8.271806e-25f;

struct TreeArgs {
  const bf16* q;
  const void *kc, *vc;
  const float *ks, *vs;
  const uint32_t* mask;
  const int32_t* lens;
  const uint64_t* tree;
  float2* part_ml;   // [partial][group rows] (max, sum)
  float* part_acc;   // [partial][group rows][D]
  int32_t* flags;    // [slice] what went wrong in it (tensor-core kernel)
  bf16* o;
  float* lse;
  int32_t* status;
  int B, cap, T, H, H_kv, R, w, gq, rows;
  int grp, nrg;      // rows per row group (8 or 16, or 128 or 256 in tree_tc), row groups
  int G;             // slices at most
  int wfar;
  int tma;           // tensor-core kernel: tensor maps are there
  float sl2;         // softmax scale * log2(e)
  int per;           // drafted tokens of a sequence
  // A batch behind one prefix (PRE): kc .. mask, cap are the prefix's, `plen` tokens of it; the
  // `tokens` drafted tokens of all sequences stand in one row, cut into B runs of T that count as
  // sequences, each over the whole prefix.
  const uint32_t* own_mask;
  int own_cap, plen, tokens;
  // The row sorted by group (NULL: as it is): the token in each place of the runs; the tokens of each
  // run; each token's place, or -1.
  const int4* order;
  const int32_t *run_tokens, *place;
};

// ------------------------------------------------------------- the row of units --
// Host and device agree only on the cache's capacity; the lengths are known to the device
// alone.  Keys come in units of 32 with an integer weight each: far units (no key of them
// is near any drafted token's window) of weight wfar, the expected share of matching masks,
// then near units of weight kTreeNear up to the last drafted token.  All units of all
// sequences, once per (KV head, row group), stand in one row that is cut into slices of
// equal weight, so that a batch of one long and many short sequences keeps the GPU busy.
// A segment is what a slice has of one (KV head, row group, sequence).  Going along the
// row, each new segment begins a new slice or a new sequence: slice + sequence number is
// different for each and numbers its partial results.
struct Stretch {
  int units, far;
  int64_t weight;
};
// Cached keys of a sequence, drafted keys behind them, and where its cache begins.
template <bool PRE>
__device__ __forceinline__ int keys_of(const TreeArgs& a, int b) {
  return PRE ? a.plen : __ldg(a.lens + b);
}
template <bool PRE>
__device__ __forceinline__ int drafts_of(const TreeArgs& a) {
  return PRE ? 0 : a.T;
}
template <bool PRE>
__device__ __forceinline__ int cache_of(int b) {
  return PRE ? 0 : b;
}
template <bool PRE>
__device__ __forceinline__ bool len_ok(const TreeArgs& a, int len) {
  return PRE || (len >= 0 && len <= a.cap - a.T);
}
template <bool PRE>
__device__ __forceinline__ Stretch stretch_of(const TreeArgs& a, int b, int len) {
  Stretch s{0, 0, 0};
  if (!len_ok<PRE>(a, len)) return s;
  if (PRE && a.run_tokens && __ldg(a.run_tokens + b) == 0) return s;
  s.units = (len + drafts_of<PRE>(a) + kTreeUnit - 1) / kTreeUnit;
  s.far = max(0, len - a.w + 1) / kTreeUnit;
  s.weight = (int64_t)s.far * a.wfar + (int64_t)(s.units - s.far) * kTreeNear;
  return s;
}
// Quotient of non-negative numbers, the short way where they fit 32 bits.  They nearly always
// do; beyond, bit by bit (the compiler's 64-bit division takes some hundred instructions at
// each place, and code that is fetched only once costs more than it runs).
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  if (((uint64_t)x | (uint64_t)y) >> 32 == 0ull) return (int64_t)((uint32_t)x / (uint32_t)y);
  int64_t q = 0;
#pragma unroll 1
  for (int i = __clzll(y) - __clzll(x | 1); i >= 0; --i)
    if (y <= x >> i) {
      x -= y << i;
      q |= 1ll << i;
    }
  return q;
}
// Units of a stretch that begin before weight x.
__device__ __forceinline__ int units_before(const TreeArgs& a, const Stretch& s, int64_t x) {
  if (x <= 0) return 0;
  if (x >= s.weight) return s.units;
  const int64_t wf = (int64_t)s.far * a.wfar;
  return x <= wf ? (int)quotient(x + a.wfar - 1, a.wfar) : s.far + (int)((x - wf + kTreeNear - 1) / kTreeNear);
}
__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
// All sequences' weight for one (KV head, row group), and the slices of the whole row (a
// unit at least each: short sequences are spread as far as they go).
template <bool PRE>
__device__ __forceinline__ int64_t total_weight(const TreeArgs& a, int lane) {
  int64_t t = 0;
  for (int b = lane; b < a.B; b += 32) t += stretch_of<PRE>(a, b, keys_of<PRE>(a, b)).weight;
  return warp_sum(t);
}
template <bool PRE>
__device__ __forceinline__ int slices_of(const TreeArgs& a, int64_t row_weight) {
  int64_t n = min((int64_t)a.G, row_weight / kTreeNear);
  // whole slices per (KV head, row group) where that leaves out little: the heads' slices then
  // walk along the same tokens, whose rows lie side by side (12 heads of 64 bytes, 30K keys of 8
  // sequences: 110 -> 77 us).  A 16th of the warps left idle costs no more than 7%.
  // (Over a prefix the runs of tokens too, unless they are sorted: they read the same keys at the same time.)
  const int lanes = a.H_kv * a.nrg * (PRE && !a.order ? a.B : 1), over = n > lanes ? (int)n % lanes : 0;
  if (over * 16 <= n) n -= over;
  return (int)max((int64_t)1, n);
}

// First weight of slice i: the row in ns nearly equal parts.
__device__ __forceinline__ int64_t slice_at(int64_t row, int ns, int64_t part, int i) {  // part = row / ns
  return part * i + (uint32_t)((uint32_t)(row - part * ns) * (uint32_t)i) / (uint32_t)ns;
}

// What a slice has of the row.  A whole warp.
struct Slice {
  int64_t W, lo, hi;  // weight of one (KV head, row group); first and last weight of the slice
  int ln;             // the first (KV head, row group)
};
template <bool PRE>
__device__ __forceinline__ Slice slice_of(const TreeArgs& a, int i, int lane) {
  Slice s{total_weight<PRE>(a, lane), 0, 0, 0};
  const int64_t row = s.W * a.H_kv * a.nrg;
  const int ns = slices_of<PRE>(a, row);
  if (s.W == 0 || i >= ns) return s;
  const int64_t part = quotient(row, ns);
  s.lo = slice_at(row, ns, part, i);
  s.hi = slice_at(row, ns, part, i + 1);
  s.ln = (int)quotient(s.lo, s.W);
  return s;
}

// Calls f(number of the partial, KV head, row group, sequence, its length, first key, end)
// for the segments of a slice, in order; a whole warp.
// S: Slice, or a volatile one in shared memory (read where it is used, no registers held).
template <bool PRE, typename S, typename F>
__device__ __forceinline__ void for_segments(const TreeArgs& a, const S& sl, int slice, int lane, F&& f) {
  for (int ln = sl.ln; ln * sl.W < sl.hi; ++ln) {
    int64_t before = ln * sl.W;
    const int kvh = ln / a.nrg, rg = ln - kvh * a.nrg;
    for (int bc = 0; bc < a.B && before < sl.hi; bc += 32) {
      const bool in = bc + lane < a.B;
      const int lb = in ? keys_of<PRE>(a, bc + lane) : -1;
      const Stretch mine = in ? stretch_of<PRE>(a, bc + lane, lb) : Stretch{0, 0, 0};
      const int64_t upto = warp_scan(mine.weight, lane);
      const int64_t from = before + upto - mine.weight;
      const int my0 = units_before(a, mine, sl.lo - from), my1 = units_before(a, mine, sl.hi - from);
      before += __shfl_sync(0xffffffffu, upto, 31);
      unsigned todo = __ballot_sync(0xffffffffu, my0 < my1);
      while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const int b = bc + src;
        const int len = __shfl_sync(0xffffffffu, lb, src);
        const int js = __shfl_sync(0xffffffffu, my0, src) * kTreeUnit;
        const int je = min(len + drafts_of<PRE>(a), __shfl_sync(0xffffffffu, my1, src) * kTreeUnit);
        f(slice + (int64_t)ln * a.B + b, kvh, rg, b, len, js, je);
      }
    }
  }
}

// Ancestors of drafted token t (itself among them), bits from T on cleared.
__device__ __forceinline__ uint64_t tree_word(const TreeArgs& a, int b, int t) {
  const uint64_t all = a.per == 64 ? ~0ull : (1ull << a.per) - 1;
  return (a.tree ? __ldg(reinterpret_cast<const unsigned long long*>(a.tree) + (int64_t)b * a.per + t)
                 : (2ull << t) - 1) &
         all;
}

// Token i of a run of a batch behind a prefix: its word, not zero where it is one, its number in the batch's
// row (0 where there is none), its window and groups.
struct Drafted {
  uint64_t word;
  int x;
  bool some;  // a token of the batch, whether its sequence's length fits or not
  __device__ __forceinline__ Drafted(const TreeArgs& a, int run, int i) {
    x = run * a.T + i;
    if (a.order) {
      at = __ldg(a.order + x);  // (one load for a row's start in place of four that wait for each other)
      some = at.x >= 0;
      word = some ? 1ull : 0ull;
      x = some ? at.x : 0;
    } else {
      at = make_int4(0, 0, 0, 0);
      word = 0ull, b = t = len = 0;
      some = x < a.tokens;
      if (some) {
        b = x / a.per, t = x % a.per;
        len = __ldg(a.lens + b);
        if (len >= 0 && len <= a.own_cap - a.per) word = tree_word(a, b, t);
      } else {
        x = 0;
      }
    }
  }
  __device__ __forceinline__ int near(const TreeArgs& a) const {  // first position inside its window
    return a.order ? at.y : a.plen + len + __popcll(word) - a.w;
  }
  __device__ __forceinline__ uint32_t groups(const TreeArgs& a, int rho) const {
    return a.order ? (uint32_t)at.z : __ldg(a.own_mask + ((int64_t)b * a.R + rho) * a.own_cap + len + t);
  }

 private:
  int4 at;        // the sorted row's entry: the token or -1, its window, its groups
  int b, t, len;  // its sequence, place in its draft, sequence's own length
};

// Two 8-bit codes (low half of `two`) as a pair of fp16; exact.
template <int FMT>
__device__ __forceinline__ uint32_t codes_f16(uint32_t two) {
  if constexpr (FMT == FOCUS_CACHE_E4M3) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3);
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    // 0x6400 | (c + 128) is 1024 + c + 128 in fp16
    const uint32_t h = __byte_perm(two ^ 0x8080u, 0x64646464u, 0x4140);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), __float2half2_rn(1152.0f));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// Four codes as two pairs of fp16.
template <int FMT>
__device__ __forceinline__ void codes_f16x2(uint32_t four, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == FOCUS_CACHE_E4M3) {
    lo = codes_f16<FMT>(four);
    hi = codes_f16<FMT>(four >> 16);
  } else {
    const uint32_t x = four ^ 0x80808080u;  // c + 128
    const uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
    const __half2 k = __float2half2_rn(1152.0f);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&a), k), z = __hsub2(*reinterpret_cast<const __half2*>(&b), k);
    lo = *reinterpret_cast<const uint32_t*>(&y);
    hi = *reinterpret_cast<const uint32_t*>(&z);
  }
}

// fp16 operands of a bf16 query row (8-bit formats): the row is multiplied by the power of
// two that brings its largest magnitude into [1, 2), which keeps every bf16 digit down to
// 2^-24 of that maximum; the logits are multiplied back.  A row with a NaN or an infinity
// stays as it is (its results are NaN either way).
__device__ __forceinline__ void row_unit(float largest, float& up, float& down) {
  uint32_t ex = __float_as_uint(largest) >> 23;
  ex = ex == 255u ? 127u : min(max(ex, 1u), 253u);  // (both powers are normal numbers)
  up = __uint_as_float((254u - ex) << 23);
  down = __uint_as_float(ex << 23);
}

// tree_tc.cu
cudaError_t launch_tree_tc(const TreeArgs& a, int d_head, int format, bool prefix, cudaStream_t s);
cudaError_t launch_tree_tc_held(const TreeArgs& a, int format, bool prefix, cudaStream_t s);  // self-test; d_head 128, bf16 or int8

}  // namespace focus
