// Sampling a token of each row of logits, with temperature, top-k, top-p and min-p, from a
// uniform random number that the caller gives.
//
// In descending order of the logits (equal ones: the lower index first) top_k leaves the first k,
// top_p of these the fewest whose weights make up top_p of theirs, min_p those with min_p of the
// first one's weight; weights are w_i = 2^(-(max - l_i) log2(e) / temperature).  What is left is a
// prefix of that order: all logits above a threshold, and the first few of those equal to it.  The
// token is the first index i with sum_{j <= i, left} w_j > u W, W the sum of all that are left.
//
// Such a choice is exact or wrong, and a vocabulary has 10^5 borders that u W may fall next to.  So
// weights are 64-bit integers, 2^44 for the largest, right to 2^-29 of their size: the exponent to
// 2^-31 (Weigh), 2^-x from a table of 64 entries and a polynomial.  Integer sums have
// no order, and the thresholds found by digits (radix selection over counts, or over weights for
// top_p) agree with the sums of the draw.
//
// A cluster of up to 16 thread blocks works on a row; each warp has a run of consecutive tokens, so
// that sums per part of a run say where the token is.  The row is read from memory once, later passes
// find it in L1 or L2.  With top_k up to the number of warps, the k-th largest of the warps' largest
// bounds the k-th of all from below; the few tokens from there on go to one block, which compares each
// with each.  Else, as soon as a bound below the threshold is known each warp keeps a list of its
// tokens above it, in their order, and the rest of the work is on the lists where they hold them.
//
// Measured: one row of 32000 with top_k and top_p 12.4 us (27 before the few went to one block, most of it
// fetching instructions that run once); 64 rows of 100003, top_p 62 us; 512 rows of 131072 bf16, no
// limits, 129 us, of which the memory needs 20: 39 instructions a token, at 57% of the issue slots;
// 143 fp32 rows of 69235, the largest of each, 12.4 us (6 for the memory).  In between it is the
// steps' dependent latencies, some 2000 cycles each for a meeting of the blocks and a sum.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "tc_ptx.cuh"

namespace focus {
namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kSampleSms = 152;
constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kBinBits = 9;  // a bin of a selection's step for each thread
constexpr int kBins = 1 << kBinBits;
constexpr int kList = 256;   // tokens of a warp's list
constexpr int kParts = 8;    // parts of a warp's run that have sums of their own
constexpr int kFew = 256;    // tokens that one block chooses from by comparing each with each
constexpr int kOne = 44;     // weights are multiples of 2^-44 of the largest
static_assert(kBins == kSampleThreads, "a bin for each thread");
// Temperatures beyond these count as these: their reciprocals, and the distance of the least min_p (744
// temperatures for a double), added to the lowest fp32 number too, stay inside fp32's range.
constexpr float kColdest = 1e-30f, kHottest = 1e28f;

// 2^(-j / 64) in units of 2^-30
__constant__ uint32_t kPowers[64] = {
    1073741824, 1062175491, 1050733751, 1039415261, 1028218693, 1017142735, 1006186087, 995347464,
    984625594, 974019220, 963527098, 953147997, 942880699, 932724001, 922676710, 912737649,
    902905651, 893179563, 883558244, 874040567, 864625413, 855311680, 846098274, 836984114,
    827968132, 819049271, 810226483, 801498734, 792865000, 784324269, 775875538, 767517817,
    759250125, 751071493, 742980960, 734977579, 727060411, 719228525, 711481005, 703816941,
    696235434, 688735596, 681316545, 673977412, 666717336, 659535466, 652430958, 645402981,
    638450708, 631573326, 624770026, 618040012, 611382493, 604796689, 598281827, 591837143,
    585461881, 579155293, 572916640, 566745190, 560640218, 554601009, 548626854, 542717053};

struct SampleArgs {
  const void* logits;
  int64_t stride;
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float *top_p, *min_p;
  // For all rows, where the arrays above are absent: log2(e) / temperature and the distance of min_p's
  // least logit from the largest, each as a sum of two floats (GB300 has few 64-bit float units: with
  // these sums in doubles a row took 20 us more), top_p as a multiple of 2^-64 (~0: all).
  float ch, cl, rh, rl;
  double t0;  // the temperature, where rows have a min_p of their own
  u64 p0;
  int32_t k0;
  int greedy;
  int V;
  int32_t* token;
  float* logprob;
  int32_t* status;
};

// What the blocks of a cluster tell one another.
struct Mail {
  u64 a;
  uint32_t b;
};

struct SampleShared {
  u64 hist[kBins];                   // this block's bins
  u64 merge[kBins], merged[kBins];   // all blocks' sums: of this block's share of the bins, of all
  float value[kSampleWarps][kList];  // the warps' lists
  int index[kSampleWarps][kList];
  u64 part_a[kSampleWarps][kParts];
  uint32_t part_b[kSampleWarps][kParts];
  uint32_t tops[kMaxCluster * kSampleWarps];  // order keys of all warps' largest
  Mail inbox[2][kMaxCluster];
  u64 warp_a[kSampleWarps];
  uint32_t warp_b[kSampleWarps];
  uint32_t powers[64];
  float m, ch, cl, rh, rl;  // the largest logit; the others as in the arguments, of this row
  float a, xh, xl;          // (see Weigh)
  // the bin that a selection has found, and the sum of those before it
  u64 above;
  int digit;
  uint32_t bound;
  int few;  // block 0: tokens in the list below, which takes the place of the warps' lists
};
// A token of a few: its value's order key and the complement of its index, by which the tokens stand in
// descending order; its weight, and its place in that order.
struct Few {
  u64 key, w;
  int rank, kept;
};
static_assert(sizeof(Few) * kFew <= sizeof(SampleShared::value), "in the lists' place");

// Significant bits of a value's 32-bit order key.
template <typename T>
constexpr int kKeyBits = 32;
template <>
constexpr int kKeyBits<bf16> = 16;
template <>
constexpr int kKeyBits<__half> = 19;

__device__ __forceinline__ uint32_t order_key(float l) {  // ascending; -0 as +0
  const uint32_t b = __float_as_uint(l + 0.0f);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key >> 31 ? key ^ 0x80000000u : ~key);
}
// The largest fp32 number below x (x not -inf).
__device__ __forceinline__ float below(float x) { return key_value(order_key(x) - 1u); }

// A row's logits against its largest, m, as weights 2^-x, x = (m - l) (ch + cl).  The difference rounded
// to fp32 would move x by up to 2^-24 of itself, where |l| and |m| lie 2^13 and more apart, and a row may be
// of such tokens alone.  So x = (a - l) (ch + cl) + xh + xl, with products that stay whole inside an fma:
//   a = 0 up to |m| ch = 2^11: xh + xl = m (ch + cl), xh a multiple of 2^-11, from which k / 64 can be taken
//         without a rounding;
//   a = m beyond, xh = xl = 0: m - l is exact for the tokens with weights, which are nearer to m than |m| / 44.
// Weights are within 2^-29 of themselves (of which the table has 2^-30) but for the bits below 2^-44.
struct Weigh {
  float a, ch, cl, xh, xl;  // ch + cl = log2(e) / temperature
  const uint32_t* powers;

  __device__ __forceinline__ explicit Weigh(const SampleShared& sh) : a(sh.a), ch(sh.ch), cl(sh.cl), xh(sh.xh), xl(sh.xl), powers(sh.powers) {}

  static constexpr float kFar = 45.9f;  // octaves from which on a weight is zero
  static constexpr float kGrid = 6144.0f, kNear = 2048.0f;  // numbers of [2^12, 2^13) are multiples of 2^-11
  // x = k / 64 + r: a sum with this has k in its low bits, and 18 in the next six for weight()'s shift
  static constexpr float kRound = 12582912.0f + 18.0f * 64.0f;
  // 2^-r - 1 = r (C1 + r (C2 + r C3)) = -r ln 2 + (r ln 2)^2 / 2 - (r ln 2)^3 / 6, in units of 2^-32
  static constexpr double kLn2 = 0.6931471805599453, kUnit = 4294967296.0;
  static constexpr float kC1 = (float)(-kUnit * kLn2), kC2 = (float)(kUnit * kLn2 * kLn2 / 2), kC3 = (float)(-kUnit * kLn2 * kLn2 * kLn2 / 6);
  // The row's a, xh and xl.
  __device__ __forceinline__ static void prepare(SampleShared& sh, float m) {
    const float x = m * sh.ch;
    const bool near = fabsf(x) < kNear;
    const float h = __fadd_rn(__fadd_rn(x, kGrid), -kGrid);
    sh.a = near ? 0.0f : m;
    sh.xh = near ? h : 0.0f;
    sh.xl = near ? fmaf(m, sh.cl, fmaf(m, sh.ch, -h)) : 0.0f;
  }
  // x but for 2^-12 + 2^-14, as bins and k take it.
  __device__ __forceinline__ float octaves(float l) const { return fminf(fmaf(a - l, ch, xh), kFar); }

  // sum + the weight of l: no branch (the sum of one row's 131072 weights is what takes longest).  (A logit
  // that is far away, or -inf, makes r infinite or NaN: its weight's digits all go in the shift.)
  __device__ __forceinline__ u64 add(u64 sum, float l) const {
    const float d = a - l;
    const float t = fmaf(octaves(l), 64.0f, kRound);
    const uint32_t k = __float_as_uint(t);
    const float r = fmaf(d, ch, fmaf(t - kRound, -0.015625f, xh)) + fmaf(d, cl, xl);
    const float p = r * fmaf(r, fmaf(r, kC3, kC2), kC1);
    return sum + weight(powers[k & 63u], __float2int_rn(p), k);
  }
  // 2^-(k % 64 / 64) 2^-r, r's part (p) in units of 2^-32, and 2^-(k / 64) by a shift, in units of 2^-44
  __device__ __forceinline__ static u64 weight(uint32_t power, int p, uint32_t k) {
    return (((u64)power << 32) + (u64)((long long)(int)power * p)) >> (k >> 6 & 63u);
  }
  // The same of two, their products and sums two at a time; x0, x1: their octaves, as bin takes them.
  __device__ __forceinline__ void pair(float l0, float l1, u64& w0, u64& w1) const {
    float x0, x1;
    pair(l0, l1, w0, w1, x0, x1);
  }
  __device__ __forceinline__ void pair(float l0, float l1, u64& w0, u64& w1, float& x0, float& x1) const {
    float d0, d1, y0, y1, t0, t1, r0, r1, p0, p1;
    ptx::fadd2(d0, d1, a, a, -l0, -l1);
    ptx::ffma2(x0, x1, d0, d1, ch, ch, xh, xh);
    x0 = fminf(x0, kFar), x1 = fminf(x1, kFar);
    ptx::ffma2(y0, y1, d0, d1, cl, cl, xl, xl);
    ptx::ffma2(t0, t1, x0, x1, 64.0f, 64.0f, kRound, kRound);
    ptx::fadd2(r0, r1, t0, t1, -kRound, -kRound);
    ptx::ffma2(r0, r1, r0, r1, -0.015625f, -0.015625f, xh, xh);
    ptx::ffma2(r0, r1, d0, d1, ch, ch, r0, r1);
    ptx::fadd2(r0, r1, r0, r1, y0, y1);
    ptx::ffma2(p0, p1, r0, r1, kC3, kC3, kC2, kC2);
    ptx::ffma2(p0, p1, r0, r1, p0, p1, kC1, kC1);
    ptx::fmul2(p0, p1, r0, r1, p0, p1);
    const uint32_t k0 = __float_as_uint(t0), k1 = __float_as_uint(t1);
    w0 = weight(powers[k0 & 63u], __float2int_rn(p0), k0);
    w1 = weight(powers[k1 & 63u], __float2int_rn(p1), k1);
  }
  // Bins of equal distances from m, 0 to kBins - 2, by which a first selection goes.
  static constexpr float kBinsPerOctave = 11.1f;
  __device__ __forceinline__ int bin(float l) const { return (int)(octaves(l) * kBinsPerOctave); }
};

// The row's 16-byte pieces: piece c has elements VEC c - lead ..; warps have runs of pieces.
template <typename T>
struct Row {
  static constexpr int VEC = 16 / (int)sizeof(T);
  const T* p;
  int V, lead, first, end;  // this warp's pieces
  int part;                 // pieces (a multiple of 32) of a part of the run

  // f(index of the first element, VEC values) for the pieces of [from, to), a whole warp together
  // (behind the last, lanes have -inf); what is not of the row is -inf.  Ends when f is false.  U pieces
  // are asked for at once: memory's latency, not its rate, bounds a warp's pass over its run.
  template <int U, typename F>
  __device__ __forceinline__ void for_pieces(int from, int to, int lane, F&& f) const {
    const uint4* q = reinterpret_cast<const uint4*>(p - lead);
    const int inner = min(to, (lead + V) / VEC);  // behind the last whole piece
#pragma unroll 1
    for (int c0 = from; c0 < to;) {
      if (c0 + 32 * U <= inner && (lead == 0 || c0 > 0)) {
        uint4 x[U];
#pragma unroll
        for (int i = 0; i < U; ++i) x[i] = __ldg(q + c0 + 32 * i + lane);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float l[VEC];
          unpack(x[i], l);
          if (!f((c0 + 32 * i + lane) * VEC - lead, l)) return;
        }
        c0 += 32 * U;
      } else {  // the ends of a row, and what is less than U pieces for each lane
        const int c = c0 + lane, i0 = c * VEC - lead;
        float l[VEC];
        if (c < to && i0 >= 0 && i0 + VEC <= V) {
          unpack(__ldg(q + c), l);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) l[e] = c < to && i0 + e >= 0 && i0 + e < V ? (float)p[i0 + e] : -INFINITY;
        }
        if (!f(i0, l)) return;
        c0 += 32;
      }
    }
  }
  __device__ __forceinline__ static void unpack(const uint4& x, float (&l)[VEC]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if constexpr (sizeof(T) == 4) l[e] = __uint_as_float(w[e]);
      else if constexpr (std::is_same<T, bf16>::value) l[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
      else l[e] = e & 1 ? __high2float(*reinterpret_cast<const __half2*>(&w[e / 2])) : __low2float(*reinterpret_cast<const __half2*>(&w[e / 2]));
    }
  }
  __device__ __forceinline__ bool whole(int i0) const { return i0 >= 0 && i0 + VEC <= V; }
  // The largest of the warp's run, NaN if there is one.
  __device__ __forceinline__ float largest(int lane) const {
    if constexpr (sizeof(T) == 4) {
      float top = -INFINITY;
      bool nan = false;
      for_pieces<4>(first, end, lane, [&](int, const float(&l)[VEC]) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) top = fmaxf(top, l[e]), nan = nan || l[e] != l[e];
        return true;
      });
      return nan ? __uint_as_float(0x7fc00000u) : top;
    } else {
      using pair = std::conditional_t<std::is_same<T, bf16>::value, __nv_bfloat162, __half2>;
      uint32_t none;
      if constexpr (std::is_same<T, bf16>::value) none = 0xff80ff80u;
      else none = 0xfc00fc00u;
      pair top[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) top[i] = *reinterpret_cast<const pair*>(&none);
      float edge = -INFINITY;
      for (int c0 = first; c0 < end; c0 += 128) {
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = c0 + 32 * i + lane, i0 = c * VEC - lead;
          x[i] = make_uint4(none, none, none, none);
          if (c >= end) continue;
          if (whole(i0)) {
            x[i] = __ldg(reinterpret_cast<const uint4*>(p + i0));
          } else {
            for (int e = 0; e < VEC; ++e)
              if (i0 + e >= 0 && i0 + e < V) {
                const float l = (float)p[i0 + e];
                edge = l != l || edge != edge ? __uint_as_float(0x7fc00000u) : fmaxf(edge, l);
              }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top[e] = __hmax2_nan(top[e], *reinterpret_cast<const pair*>(&w[e]));
        }
      }
      top[0] = __hmax2_nan(__hmax2_nan(top[0], top[1]), __hmax2_nan(top[2], top[3]));
      const float a = __low2float(top[0]), b = __high2float(top[0]);
      return a != a || b != b || edge != edge ? __uint_as_float(0x7fc00000u) : fmaxf(fmaxf(a, b), edge);
    }
  }
};

// A program of many steps that run once: what a step costs is the fetch of its instructions (some 40
// cycles each from L2, when they have not been used before) rather than their number.  So the steps are
// functions, not inlined, that both selections and all sums share, and short loops.  (Inlined, one row of 32000
// with top-k and top-p took 38000 cycles.)
__device__ __noinline__ u64 warp_upto(u64 x) {  // inclusive sums
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
__device__ __forceinline__ u64 warp_total(u64 x) { return __shfl_sync(0xffffffffu, warp_upto(x), 31); }
__device__ __forceinline__ uint32_t warp_upto(uint32_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
__device__ __noinline__ u64 weight(const SampleShared& sh, float l) { return Weigh(sh).add(0, l); }

// The least q with q x >= n, of a quotient below 2^20 (a vocabulary's tokens), n and x positive.
__device__ __noinline__ uint32_t times(u64 n, u64 x) {
  uint32_t q = (uint32_t)__fdividef((float)n, (float)x);  // one off at most, to either side
  q -= q > 0 ? 1u : 0u;
  for (int i = 0; i < 3 && q * x < n; ++i) ++q;
  return q;
}
// A number of [0, 1) as a multiple of 2^-64, cut off.
__device__ __forceinline__ u64 fraction(float f) {
  const uint32_t b = __float_as_uint(f);
  const int e = (int)(b >> 23);  // f = digits 2^(e - 150)
  const u64 digits = (b & 0x7fffffu) | 0x800000u;
  return e >= 86 ? digits << (e - 86) : e > 62 ? digits >> (86 - e) : 0ull;
}
// The least multiple that is no less than `share` of `all`, and one at least.
__device__ __forceinline__ u64 share_of(u64 share, u64 all) {
  return max((u64)1, __umul64hi(share, all) + (share * all != 0));
}

// All values above `at`, and `ties` of those equal to it.
struct Cut {
  float at;
  uint32_t ties;
};

// All threads of the cluster meet, and see what any has written in shared memory.  One thread's fence
// speaks for its block, which has met before it.
__device__ __noinline__ void meet(int C) {
  __syncthreads();
  if (C == 1) return;
  if (threadIdx.x == 0) asm volatile("fence.acq_rel.cluster;" ::: "memory");
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sums of the warps (lane 0's numbers count) to every block: this block's in warp_a and warp_b, all blocks' in the
// returned letters.  Two boxes by turns: one is written again two meetings later, when all have read it.
__device__ __noinline__ const Mail* report(SampleShared& sh, int C, int rank, int turn, u64 a, uint32_t b) {
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  Mail* box = sh.inbox[turn];
  __syncthreads();
  if (lane == 0) sh.warp_a[wp] = a, sh.warp_b[wp] = b;
  __syncthreads();
  if (wp == 0) {
    const bool in = lane < kSampleWarps;
    const Mail l{warp_total(in ? sh.warp_a[lane] : 0), __reduce_add_sync(0xffffffffu, in ? sh.warp_b[lane] : 0u)};
    if (lane < C) *(C > 1 ? cg::this_cluster().map_shared_rank(box + rank, lane) : box) = l;
  }
  meet(C);
  return box;
}

// All blocks' bins together, and of them the one in which the sum reaches `target`, from `above` on
// in front of the first (target 0: `share` of the sum); -1 where it does not.  `above` goes on to the
// sum of those before it.
__device__ __noinline__ int find(SampleShared& sh, int C, int rank, u64& target, u64 share, u64& above) {
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  if (tid == 0) sh.digit = -1;
  meet(C);
  u64 mine = sh.hist[tid];
  if (C > 1) {
    // a block sums its share of the bins over all blocks and sends it to each: one load and one store of
    // another block's memory per thread, which take 700 cycles each (16 blocks: 4000 cycles less than
    // every thread's reading one bin of each)
    const int each = kBins / C, other = tid / each, bin = rank * each + tid % each;
    sh.merge[tid] = cg::this_cluster().map_shared_rank(sh.hist, other)[bin];
    __syncthreads();
    u64 sum = 0;
    for (int i = tid % each; i < kBins; i += each) sum += sh.merge[i];
    cg::this_cluster().map_shared_rank(sh.merged, other)[bin] = sum;
    meet(C);
    mine = sh.merged[tid];
  }
  const u64 upto = warp_upto(mine);
  if (lane == 31) sh.warp_a[wp] = upto;
  __syncthreads();
  const u64 w = warp_upto(lane < kSampleWarps ? sh.warp_a[lane] : 0);
  const u64 before = above + upto - mine + (wp ? __shfl_sync(0xffffffffu, w, wp - 1) : 0);
  if (target == 0) target = share_of(share, __shfl_sync(0xffffffffu, w, 31));
  if (before < target && before + mine >= target) sh.above = before, sh.digit = tid;
  __syncthreads();
  const int digit = sh.digit;
  if (digit >= 0) above = sh.above;
  __syncthreads();  // (before the next round writes there)
  return digit;
}

// Where `target` lies in the running sums of up to 32 parts, a lane each (a sum s and a number of
// ties n, the first `ties` of which count tie_w); target and ties go on to what is left of them there.
__device__ __noinline__ int part_of(u64 s, uint32_t n, u64 tie_w, u64& target, uint32_t& ties) {
  const uint32_t before = warp_upto(n, threadIdx.x & 31) - n, left = ties - min(ties, before);
  s += min(left, n) * tie_w;
  const u64 upto = warp_upto(s);
  const int at = max(0, __ffs(__ballot_sync(0xffffffffu, target < upto)) - 1);
  target -= __shfl_sync(0xffffffffu, upto - s, at);
  ties = __shfl_sync(0xffffffffu, left, at);
  return at;
}

// min_p's least logit, as the least fp32 number that is no less: m - (rh + rl), rounded up
__device__ __forceinline__ float least_of_min_p(const SampleShared& sh) {
  const float m = sh.m, d = m - sh.rh, b = d - m;
  return sh.rh < INFINITY ? __fadd_ru(d, ((m - (d - b)) - (sh.rh + b)) - sh.rl) : -INFINITY;
}
// The result: ln(w / W) = -x ln 2 - ln(1 + (W - 1)), W in units of the largest weight
__device__ __noinline__ void put(const SampleArgs& a, int r, const SampleShared& sh, int token, float l, u64 total) {
  a.token[r] = token;
  if (a.logprob) a.logprob[r] = -((sh.m - l) * sh.ch * 0.69314718f) - log1pf((float)(total - (1ull << kOne)) * 5.6843419e-14f);
}

template <typename T>
struct Sampler {
  static constexpr int VEC = Row<T>::VEC;
  SampleShared& sh;
  int C, rank, lane, wp;
  Row<T> row;
  int turns;
  // Tokens that are looked at: between two bounds, and of one bin alone if it is not negative.
  float from, upto;
  int only;
  int listed;  // those of the warp's run, in its list; -1: too many for it, or none made

  __device__ __forceinline__ u64 weight(float l) const { return focus::weight(sh, l); }

  // The warp's tokens between two bounds into its list, in order (those of other bins than `bin` among them
  // too: there are few).  Given up where it will hardly hold them all.
  __device__ __noinline__ void list(float bound, float top, int bin) {
    from = bound, upto = top, only = bin;
    const Row<T> row = this->row;
    float* value = sh.value[wp];
    int* index = sh.index[wp];
    int n = 0, seen = 0;
    const int all = row.end - row.first;
    row.template for_pieces<2>(row.first, row.end, lane, [&](int i0, const float(&l)[VEC]) {
      unsigned in = 0;
#pragma unroll
      for (int e = 0; e < VEC; ++e) in |= l[e] >= bound && l[e] <= top ? 1u << e : 0u;
      seen += 32;
      if (!__any_sync(0xffffffffu, in)) return true;
      const int sum = warp_upto((uint32_t)__popc(in), lane), more = __shfl_sync(0xffffffffu, sum, 31);
      // (so dense, when a quarter has been seen, that the list is a fifth too short)
      if (n + more > kList || (seen * 4 >= all && (int64_t)(n + more) * all * 4 > (int64_t)5 * kList * seen)) {
        n = -1;
        return false;
      }
      int at = n + sum - __popc(in);
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (in >> e & 1u) value[at] = l[e], index[at] = i0 + e, ++at;
      n += more;
      return true;
    });
    listed = n;
    __syncwarp();
  }
  // f(value) for the warp's tokens to look at; a warp's lanes have their own.
  template <typename F>
  __device__ __forceinline__ void visit(F&& f) const {
    const int n = listed;
    const int only = this->only;
    const Weigh weigh(sh);
    if (n >= 0) {
#pragma unroll 1
      for (int i = lane; i < n; i += 32) {
        const float l = sh.value[wp][i];
        if (only < 0 || weigh.bin(l) == only) f(l);
      }
    } else {
      const float from = this->from, upto = this->upto;
      row.template for_pieces<1>(row.first, row.end, lane, [&](int, const float(&l)[VEC]) {
#pragma unroll 1
        for (int e = 0; e < VEC; ++e)
          if (l[e] >= from && l[e] <= upto && l[e] > -INFINITY && (only < 0 || weigh.bin(l[e]) == only)) f(l[e]);
        return true;
      });
    }
  }
  // Empty bins (every block has read the last ones before it went on from find).
  __device__ __forceinline__ u64* bins() {
    sh.hist[threadIdx.x] = 0;
    __syncthreads();
    return sh.hist;
  }

  // The whole choice among the tokens from `bound` on, top_k at least, by block 0, if they are few: whether
  // they were.  Each is compared with each: three short loops, where the general way has ten times
  // the instructions, that run once.
  __device__ __noinline__ bool choose_few(const SampleArgs& a, int r, float bound, int top_k, u64 top_p, float u) {
    const int tid = threadIdx.x;
    // into block 0's list, in any order
    int* count = C > 1 ? cg::this_cluster().map_shared_rank(&sh.few, 0) : &sh.few;
    Few* few = reinterpret_cast<Few*>(sh.value);
    Few* to = C > 1 ? cg::this_cluster().map_shared_rank(few, 0) : few;
    const uint32_t low = order_key(bound);
    meet(C);  // (block 0 has set its number to zero)
    if (sh.tops[rank * kSampleWarps + wp] >= low) {
      const Row<T> row = this->row;
      row.template for_pieces<1>(row.first, row.end, lane, [&](int i0, const float(&l)[VEC]) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (l[e] >= bound) {
            const int at = atomicAdd(count, 1);
            if (at < kFew) to[at].key = (u64)order_key(l[e]) << 32 | ~(uint32_t)(i0 + e);
          }
        return true;
      });
    }
    meet(C);
    const int n = *count;
    if (n > kFew) {
      meet(C);  // (the list's place is written anew when all have read the number)
      return false;
    }
    if (rank != 0) {
      meet(C);  // (no block leaves while another may read its number)
      return true;
    }
    // Thread i for token i from here on.  In descending order: its place, its weight if top_k leaves it.
    const bool on = tid < n;
    const int last = wp * 32 < n ? n : 0;  // (warps without one have no loops)
    const u64 key = few[on ? tid : 0].key;
    const float value = key_value((uint32_t)(key >> 32));
    int place = 0;
#pragma unroll 8
    for (int j = 0; j < last; ++j) place += few[j].key > key ? 1 : 0;
    const u64 w = place < top_k ? weight(value) : 0;
    meet(C);
    if (on) few[tid].w = w, few[tid].rank = place;
    __syncthreads();
    // top_p: the sum of those before it is short of the target; min_p
    bool keep = on && place < top_k;
    if (top_p != ~0ull) {
      u64 before = 0, all = 0;
#pragma unroll 4
      for (int j = 0; j < last; ++j) {
        const u64 y = few[j].w;
        all += y;
        before += few[j].rank < place ? y : 0;
      }
      keep = keep && before < share_of(top_p, all);
    }
    keep = keep && value >= least_of_min_p(sh);
    if (on) few[tid].kept = keep;
    __syncthreads();
    // the draw, in the order of the vocabulary
    u64 before = 0, total = 0;
#pragma unroll 4
    for (int j = 0; j < last; ++j) {
      const u64 y = few[j].kept ? few[j].w : 0;
      total += y;
      before += (uint32_t)few[j].key > (uint32_t)key ? y : 0;  // a lower index
    }
    const u64 target = __umul64hi(fraction(u), total);
    if (keep && before <= target && target - before < w) put(a, r, sh, (int)~(uint32_t)key, value, total);
    return true;
  }

  // Selection from above: the value with which the sum of (1 or weights) over all larger values and
  // itself first reaches `target` (0: `share` of the sum of all), among those to look at above
  // `out`.  No such value: ties = 0.  Without a bound from which on to look, the first step goes by bins
  // of equal distance from the largest and lists the bin that it finds; further steps are digits of the
  // values' order.
  __device__ __noinline__ Cut select(bool by_weight, u64 target, u64 share, float out) {
    constexpr int KB = kKeyBits<T>, KS = 32 - KB;
    float high = sh.m, least = fmaxf(from, out);
    u64 above = 0;
    if (from == -INFINITY) {
      u64* h = bins();
      {
        const Row<T> row = this->row;
        const Weigh weigh(sh);
        row.template for_pieces<1>(row.first, row.end, lane, [&](int, const float(&l)[VEC]) {
          u64 w[VEC];
          float x[VEC];
#pragma unroll
          for (int e = 0; e < VEC; e += 2) weigh.pair(l[e], l[e + 1], w[e], w[e + 1], x[e], x[e + 1]);
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (l[e] > out && (w[e] || !by_weight)) atomicAdd(h + (int)(x[e] * weigh.kBinsPerOctave), by_weight ? w[e] : 1ull);
          return true;
        });
      }
      const int bin = find(sh, C, rank, target, share, above);
      if (bin < 0) return Cut{-INFINITY, 0u};
      // (the bin's values are inside these, whatever the roundings: octaves are off by less than 2^-11)
      const float m = sh.m, width = 1.0f / (Weigh::kBinsPerOctave * sh.ch), slack = 1.0f + 1e-5f;
      const float off = 2.5e-7f * fabsf(m) + 0x1p-11f / sh.ch;
      high = fminf(high, m - ((float)bin * width) / slack + off);
      const float lowest = m - ((float)(bin + 1) * width) * slack - off;
      // (no lower than a bound that all finite numbers are above; the last bin has no other)
      least = fmaxf(least, fmaxf(bin < kBins - 3 ? lowest : -INFINITY, -3.4028234663852886e38f));
      list(least, high, bin);
    }
    uint32_t top = order_key(high) >> KS;  // the highest key of the bins
    int shift = max(0, 32 - __clz(top - min(order_key(least) >> KS, top)) - kBinBits);
    uint32_t span = ~0u;  // keys of the bins, less one
#pragma unroll 1
    for (;;) {
      u64* h = bins();
      visit([&](float l) {
        const uint32_t d = top - (order_key(l) >> KS);
        if (l > out && d <= span) atomicAdd(h + (d >> shift), by_weight ? weight(l) : 1ull);
      });
      const int digit = find(sh, C, rank, target, 0, above);
      if (digit < 0) return Cut{-INFINITY, 0u};
      top -= (uint32_t)digit << shift;
      if (shift == 0) break;
      span = (1u << shift) - 1u;
      shift = max(0, shift - kBinBits);
    }
    // the bits below are those of a value of T: zeros, inverted where it is negative
    const uint32_t key = top << KS;
    const float at = key_value(key >> 31 ? key : key | ((1u << KS) - 1u));
    return Cut{at, by_weight ? times(target - above, weight(at)) : (uint32_t)(target - above)};
  }

  // Sums over what is above a cut, and the number of those at it: per part of a warp's run, per
  // warp, and per block in the letters.
  __device__ __noinline__ const Mail* sums(const Cut cut) {
    u64 s = 0;
    uint32_t n = 0;
    if (listed >= 0) {
#pragma unroll 1
      for (int i = lane; i < listed; i += 32) {
        const float l = sh.value[wp][i];
        if (l > cut.at) s += weight(l);
        n += l == cut.at;
      }
      s = warp_total(s);
      n = __reduce_add_sync(0xffffffffu, n);
    } else {
      const Row<T> row = this->row;
      const Weigh weigh(sh);
      u64 all = 0;
      uint32_t count = 0;
#pragma unroll 1
      for (int i = 0; row.first + i * row.part < row.end; ++i) {
        const int c0 = row.first + i * row.part, c1 = min(row.end, c0 + row.part);
        s = 0, n = 0;
        if (cut.at == -INFINITY) {  // all
          row.template for_pieces<2>(c0, c1, lane, [&](int, const float(&l)[VEC]) {
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
              u64 w0, w1;
              weigh.pair(l[e], l[e + 1], w0, w1);
              s += w0;
              s += w1;
            }
            return true;
          });
        } else {
          row.template for_pieces<1>(c0, c1, lane, [&](int, const float(&l)[VEC]) {
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
              u64 w0, w1;
              weigh.pair(l[e], l[e + 1], w0, w1);
              s += l[e] > cut.at ? w0 : 0;
              s += l[e + 1] > cut.at ? w1 : 0;
              n += (l[e] == cut.at) + (l[e + 1] == cut.at);
            }
            return true;
          });
        }
        s = warp_total(s);
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) sh.part_a[wp][i] = s, sh.part_b[wp][i] = n;
        all += s;
        count += n;
      }
      s = all, n = count;
    }
    return report(sh, C, rank, turns++ & 1, s, n);
  }
};

template <typename T>
__global__ void __launch_bounds__(kSampleThreads, 2) sample_rows(const __grid_constant__ SampleArgs a, int C) {
  constexpr int VEC = Row<T>::VEC;
  __shared__ SampleShared sh;
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  const int rank = blockIdx.x % C, r = blockIdx.x / C;
  if (C > 1) cg::this_cluster().barrier_arrive();  // every block runs before another writes to it

  // ---- the row's parameters; a row with one out of its range gets no token
  const float u = __ldg(a.u + r);
  const int top_k = a.top_k ? __ldg(a.top_k + r) : a.k0;
  u64 top_p = a.p0;
  bool invalid = !(u >= 0.0f && u < 1.0f), greedy = a.greedy;
  float tr = 1.0f, mr = 0.0f;
  if (a.temperature) {
    tr = __ldg(a.temperature + r);
    invalid = invalid || !(tr >= 0.0f && tr < INFINITY);
    greedy = greedy || tr == 0.0f;
    tr = fmaxf(fminf(tr, kHottest), kColdest);
  }
  if (a.top_p) {
    const float x = __ldg(a.top_p + r);
    invalid = invalid || !(x >= 0.0f);
    top_p = x >= 1.0f ? ~0ull : fraction(x);
    greedy = greedy || top_p == 0;
  }
  if (a.min_p) {
    mr = __ldg(a.min_p + r);
    invalid = invalid || !(mr >= 0.0f && mr <= 1.0f);
  }
  if (tid < 64) sh.powers[tid] = kPowers[tid];
  if (tid == 64) {
    sh.ch = a.ch, sh.cl = a.cl;
    if (a.temperature) {
      // log2(e) = 1.442695 + 1.9259630e-8 over the temperature, with the first quotient's remainder
      const float q = 1.44269502f / tr;
      sh.ch = q;
      sh.cl = (fmaf(-q, tr, 1.44269502f) + 1.92596303e-08f) / tr;
    }
  }
  if (tid == 96) {
    sh.rh = a.rh, sh.rl = a.rl;
    if (a.min_p) sh.rh = mr > 0.0f ? 0.0f : INFINITY, sh.rl = 0.0f;
    if ((a.min_p || a.temperature) && (a.min_p ? mr > 0.0f : a.rh < INFINITY)) {
      const double far = (a.min_p ? -log((double)mr) : (double)a.rh + a.rl) * (a.temperature ? (double)tr : a.t0);
      sh.rh = (float)far;
      sh.rl = (float)(far - (double)sh.rh);
    }
  }
  Sampler<T> t{sh, C, rank, lane, wp, {}, 0, -INFINITY, INFINITY, -1, -1};
  Row<T>& row = t.row;
  row.p = reinterpret_cast<const T*>(a.logits) + r * a.stride;
  row.V = a.V;
  row.lead = (int)(reinterpret_cast<uintptr_t>(row.p) & 15u) / (int)sizeof(T);
  {
    const int pieces = (row.lead + a.V + VEC - 1) / VEC, warps = C * kSampleWarps;
    const int each = ((pieces + warps - 1) / warps + 31) / 32;
    row.first = min(pieces, (rank * kSampleWarps + wp) * each * 32);
    row.end = min(pieces, row.first + each * 32);
    row.part = (each + kParts - 1) / kParts * 32;
  }

  // ---- the largest, of all warps' largest; a NaN anywhere comes first
  const float mine = row.largest(lane);
  const uint32_t key = __reduce_max_sync(0xffffffffu, mine != mine ? ~0u : order_key(mine));
  if (C > 1) {
    cg::this_cluster().barrier_wait();
    if (lane < C) cg::this_cluster().map_shared_rank(sh.tops, lane)[rank * kSampleWarps + wp] = key;
  } else if (lane == 0) {
    sh.tops[wp] = key;
  }
  meet(C);
  const int warps = C * kSampleWarps;
  uint32_t largest = 0u;
#pragma unroll 1
  for (int i = lane; i < warps; i += 32) largest = max(largest, sh.tops[i]);
  largest = __reduce_max_sync(0xffffffffu, largest);
  const float m = key_value(largest);
  const bool bad = !(fabsf(m) < INFINITY);
  if (bad || invalid) {
    if (rank == 0 && tid == 0) {
      a.token[r] = -1;
      if (a.logprob) a.logprob[r] = __uint_as_float(0x7fc00000u);
      if (a.status) atomicMin(a.status, invalid ? FOCUS_ERR_INVALID_ARG : FOCUS_ERR_NONFINITE);
    }
    return;
  }
  if (tid == 0) sh.m = m, Weigh::prepare(sh, m);

  // ---- one is left: the first of the largest
  if (greedy || top_k == 1 || a.V == 1) {
    int at = INT_MAX;
    if (__any_sync(0xffffffffu, key == largest))
      row.template for_pieces<2>(row.first, row.end, lane, [&](int i0, const float(&l)[VEC]) {
#pragma unroll
        for (int e = VEC - 1; e >= 0; --e)
          if (l[e] == m) at = min(at, i0 + e);
        return !__any_sync(0xffffffffu, at < INT_MAX);
      });
    at = __reduce_min_sync(0xffffffffu, at);
    // the first warp that has one, in the order of the runs, writes
    int first = warps;
#pragma unroll 1
    for (int i = lane; i < warps; i += 32) first = min(first, sh.tops[i] == largest ? i : warps);
    first = __reduce_min_sync(0xffffffffu, first);
    if (first == rank * kSampleWarps + wp && lane == 0) {
      a.token[r] = at;
      if (a.logprob) a.logprob[r] = 0.0f;
    }
    return;
  }

  // ---- what is left
  Cut cut{-INFINITY, 0u};
  if (top_k > 1 && top_k < a.V) {
    // The k-th largest of the warps' largest is no more than that of all: its rank among them
    if (tid == 0) sh.bound = 0u, sh.few = 0;
    __syncthreads();
    if (top_k <= warps && tid < warps) {
      const uint32_t x = sh.tops[tid];
      int before = 0;
#pragma unroll 8
      for (int i = 0; i < warps; ++i) before += (int)(sh.tops[i] > x) | ((int)(sh.tops[i] == x) & (int)(i < tid));
      if (before == top_k - 1) sh.bound = x;
    }
    __syncthreads();
    const float bound = sh.bound ? key_value(sh.bound) : -INFINITY;
    if (bound > -INFINITY) {
      if (t.choose_few(a, r, bound, top_k, top_p, u)) return;
      t.list(bound, m, -1);
    }
    cut = t.select(false, (u64)top_k, 0, -INFINITY);
    if (t.only >= 0) t.list(fmaxf(cut.at, -3.4028234663852886e38f), m, -1);  // (not that bin's, but all that are left)
  } else {
    __syncthreads();
  }
  const Mail* box;
  auto sum_of = [&]() { return warp_total(lane < C ? box[lane & (kMaxCluster - 1)].a : 0); };  // over the letters
  if (top_p != ~0ull) {
    // of the weights that top-k left
    if (cut.ties == 0) {
      cut = t.select(true, 0, top_p, -INFINITY);
      if (t.only >= 0) t.list(fmaxf(cut.at, -3.4028234663852886e38f), m, -1);
    } else {
      box = t.sums(cut);
      const u64 each = t.weight(cut.at), higher = sum_of(), target = share_of(top_p, higher + cut.ties * each);
      if (higher < target) {  // ties of the k-th value make up the rest
        if (each) cut.ties = min(cut.ties, times(target - higher, each));
      } else {
        cut = t.select(true, target, 0, cut.at);
      }
    }
  }
  const float low = least_of_min_p(sh);
  if (low > cut.at) cut = Cut{below(low), 0u};
  if (t.listed < 0 && cut.at > t.from) t.list(cut.at, m, -1);
  // ---- the draw
  box = t.sums(cut);
  const u64 tie_w = cut.ties ? t.weight(cut.at) : 0, total = sum_of() + cut.ties * tie_w;
  u64 target = __umul64hi(fraction(u), total);
  uint32_t ties = cut.ties;
  // the block, the warp, the part of its run in whose share of the sum the target lies
  const Mail its = box[lane & (kMaxCluster - 1)];
  if (part_of(lane < C ? its.a : 0, lane < C ? its.b : 0, tie_w, target, ties) != rank) return;
  const int w = lane & (kSampleWarps - 1);
  if (part_of(lane < kSampleWarps ? sh.warp_a[w] : 0, lane < kSampleWarps ? sh.warp_b[w] : 0, tie_w, target, ties) != wp) return;
  // Of this lane's N tokens l, the first at at(0): the token if the target lies in the warp's, else
  // what is left of it behind them.
  auto look = [&](auto& l, auto at) {
    constexpr int N = sizeof(l) / sizeof(float);
    u64 s = 0;
    uint32_t n = 0;
#pragma unroll 1
    for (int e = 0; e < N; ++e) {
      if (l[e] > cut.at) s += t.weight(l[e]);
      n += l[e] == cut.at;
    }
    const uint32_t n_upto = warp_upto(n, lane);
    uint32_t left = ties - min(ties, n_upto - n);
    s += min(left, n) * tie_w;
    const u64 upto = warp_upto(s);
    const unsigned hit = __ballot_sync(0xffffffffu, target < upto);
    if (hit && lane == __ffs(hit) - 1) {
      u64 rest = target - (upto - s);
#pragma unroll 1
      for (int e = 0; e < N; ++e) {
        u64 we = l[e] > cut.at ? t.weight(l[e]) : 0;
        if (l[e] == cut.at && left) we = tie_w, --left;
        if (rest < we) {
          put(a, r, sh, at(e), l[e], total);
          break;
        }
        rest -= we;
      }
    }
    target -= __shfl_sync(0xffffffffu, upto, 31);
    ties -= min(ties, __shfl_sync(0xffffffffu, n_upto, 31));
    return hit != 0;
  };
  if (t.listed >= 0) {
#pragma unroll 1
    for (int i0 = 0; i0 < t.listed; i0 += 32) {
      const int i = i0 + lane;
      float l[1] = {i < t.listed ? sh.value[wp][i] : -INFINITY};
      if (look(l, [&](int) { return sh.index[wp][i]; })) return;
    }
    return;
  }
  const bool has = lane < (row.end - row.first + row.part - 1) / row.part;
  const int q = lane & (kParts - 1);
  const int part = part_of(has ? sh.part_a[wp][q] : 0, has ? sh.part_b[wp][q] : 0, tie_w, target, ties);
  row.template for_pieces<1>(row.first + part * row.part, row.end, lane, [&](int i0, const float(&l)[VEC]) {
    return !look(l, [&](int e) { return i0 + e; });
  });
}

template <typename T>
cudaError_t launch(const SampleArgs& a, int rows, cudaStream_t s) {
  // Blocks of a row.  As many as are resident at once (two on an SM): 64 rows of 100003 with top_p take 64
  // us in 4 blocks each and 83 in 8, 16 chats' rows of 50000 59 in 2, 92 in 4.  More where a block would have
  // over 65536 tokens, whose passes wait for memory: 256 fp32 rows of 131072 with min_p take 127 us in one
  // block, 89 in 2, 82 in 4; 512 bf16 rows 135 in one, 133 in 2, 190 in 4.  As long as each warp has a
  // piece for each lane; 16 are more than clusters may have by default.
  int C = 1;
  while (C < kMaxCluster && ((int64_t)rows * 2 * C <= 2 * kSampleSms || a.V / C > 65536) &&
         a.V > C * kSampleThreads * Row<T>::VEC)
    C *= 2;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(sample_rows<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kSampleThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t rc = cudaLaunchKernelEx(&cfg, sample_rows<T>, a, C);
  return rc != cudaSuccess ? rc : cudaGetLastError();
}

}  // namespace

cudaError_t launch_sample(const focus_sample_params& p, const void* logits, const float* u, const float* temperature,
                          const int32_t* top_k, const float* top_p, const float* min_p, int32_t* token,
                          float* logprob, int32_t* status, cudaStream_t s) {
  SampleArgs a;
  a.logits = logits, a.stride = p.stride, a.u = u;
  a.temperature = temperature, a.top_k = top_k, a.top_p = top_p, a.min_p = min_p;
  a.k0 = p.top_k, a.t0 = std::max(std::min(p.temperature, (double)kHottest), (double)kColdest);
  a.greedy = (!temperature && p.temperature == 0.0) || (!top_p && p.top_p < 0x1p-64);
  const double c = temperature ? 1.0 : 1.4426950408889634074 / a.t0;
  a.ch = (float)c;
  a.cl = (float)(c - (double)a.ch);
  // min_p's distance, for temperature 1 where the rows have their own
  const double far = min_p || p.min_p == 0.0 ? INFINITY : -log(p.min_p) * (temperature ? 1.0 : a.t0);
  a.rh = (float)far;
  a.rl = far < INFINITY ? (float)(far - (double)a.rh) : 0.0f;
  a.p0 = top_p || p.top_p >= 1.0 ? ~0ull : (u64)(p.top_p * 0x1p64);
  a.V = p.V, a.token = token, a.logprob = logprob, a.status = status;
  return p.dtype == FOCUS_DTYPE_BF16  ? launch<bf16>(a, p.rows, s)
         : p.dtype == FOCUS_DTYPE_F16 ? launch<__half>(a, p.rows, s)
                                      : launch<float>(a, p.rows, s);
}

}  // namespace focus
