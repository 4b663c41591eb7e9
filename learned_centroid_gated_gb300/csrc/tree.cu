// Decode step for up to 64 drafted tokens per sequence over a cache in bf16 or in 8 bits,
// sequences of different lengths: attention on the same union set as the forward pass
// ("Why Attend to Everything? Focus is the Key", gist.science technical summary, section 2,
// "Core Architecture" and "Inference Efficiency (Top-k)": window keys with exact softmax
// plus distant keys that share a group), restricted among the drafted tokens to a token's
// ancestors in the draft tree.
//
// Memory-bound while the rows per KV head (T tokens x H / H_kv query heads) are few: the
// K and V rows that any drafted token may see are read once per 16 rows.
//   tree_split    one warp per slice of the work, KV head and group of 16 rows.  It lists
//                 the slice's keys that any of its rows sees, streams their rows through a
//                 shared-memory ring with 16-byte asynchronous copies, and keeps an online
//                 softmax per row; both products are m16n8k16 register-fragment MMAs.
//   tree_combine  merges a row's slices by their maxima: O, LSE.
// Measured, one token per sequence, 32 / 8 heads of 128: 32 sequences of up to 32K bf16 keys
// 175 us (6.1 TB/s), e4m3 110 us (5.0 TB/s), int8 121; 4 tokens (16 rows) over 128K keys, bf16 90 us,
// e4m3 85, int8 93; 4 sequences of up to 1000 keys (12 heads of 64) 8.7 us and 4.1 for the merge, of
// which the memory needs 0.8: the kernels' starts, the listing and dependent reads.  In bf16 the
// memory bounds it.  In 8 bits neither the memory (0.64 of its rate with 8 rows, 0.36 with 16) nor
// the issue slots (0.47, 0.41) are full: a warp's chain of conversion, scales and exponentials per
// tile, with 2.75 and 2 warps a scheduler to overlap, at 168 registers (D = 128: 152 bytes of
// them spilled) and 255.
#include <math.h>

#include <algorithm>

#include "tc_ptx.cuh"
#include "tree.cuh"
#include "warp_mma.cuh"

namespace focus {
namespace {

using namespace ptx;
using namespace wmma16;

constexpr int kTreeSms = 152;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPTop = 14.0f;  // 8-bit formats: log2 of the largest P times V scale

// Per-warp shared memory: a ring of tiles, each KT K rows, as many V rows and, in the 8-bit
// formats, their scales; per stage its keys' slots and masks; the listing.  8-bit tiles have
// 32 keys: the work per key that is not a product (reference, exponentials, listing) and its
// latency, not the memory, are what bounds them.
// bf16 rows are padded by 16 bytes (the eight rows of an ldmatrix phase start in different
// banks).  8-bit rows are read as 16-byte pieces (see below) and swizzled instead.
template <int D, int FMT, int NR>
struct TreeLayout {
  static constexpr bool B16 = FMT == FOCUS_CACHE_BF16;
  static constexpr int KT = B16 ? 16 : 32;                  // keys per tile
  static constexpr int STAGES = B16 ? (D == 128 ? 3 : 5) : (D == 128 ? 2 : 3);
  static constexpr int WARPS = B16 ? 8 : NR == 8 ? 11 : 8;  // per SM
  static constexpr int BLOCK = B16 && D == 128 ? 128 : 256;  // raw keys per listing step
  static constexpr int ROW = B16 ? 2 * D + 16 : D;
  static constexpr int OFF_SCALE = 2 * KT * ROW;
  static constexpr int OFF_KEY = OFF_SCALE + (B16 ? 0 : 2 * KT * 4);
  static constexpr int STAGE = OFF_KEY + 2 * KT * 4;
  static constexpr int OFF_IDX = STAGES * STAGE;
  static constexpr int OFF_MSK = OFF_IDX + BLOCK * 4;
  static constexpr int OFF_CNT = OFF_MSK + BLOCK * 4;
  static constexpr int BYTES = (OFF_CNT + STAGES * 4 + 15) / 16 * 16;
  static_assert(STAGE % 16 == 0 && ROW % 16 == 0, "16-byte aligned rows");
  static_assert(WARPS * (BYTES + 1024) <= 228 * 1024, "shared memory of an SM");
};

// Byte offset of 16-byte piece c of row r of a tile, 8-bit formats.  K is read by quads:
// lane (g, t4) takes piece t4 (+ 4) of row g; V by columns: lane (g, t4) takes piece g of
// rows 2 t4, 2 t4 + 1, .. (D = 128), half a piece with D = 64.  The XORs put the eight
// lanes of a phase into different banks.
template <int D>
__device__ __forceinline__ int k_piece(int r, int c) {
  return r * D + 16 * (D == 128 ? c ^ ((r & 1) << 2) : c);
}
template <int D>
__device__ __forceinline__ int v_piece(int r, int c) {
  if (D == 128) return r * D + 16 * (c ^ (2 * ((r >> 1) & 3)));
  const int p = (r & 16) | ((r & 15) >> 1) | ((r & 1) << 3);
  return p * D + 16 * (c ^ (((p >> 1) & 1) << 1));
}

// NR: rows per warp.  16 fill the MMA's M; O = P V has P as its row operand.  With up to 8
// the scores' upper half is empty, and O^T = V^T P^T takes the lane's own scores as its
// column operand: half the products and half the accumulators of NR = 16, and in 8 bits 11
// warps fit on an SM in place of 8 (4 rows: 32 e4m3 sequences 153 -> 118 us; up to 8 rows only
// this form is built, since NR = 16 had the upper half idle).
template <int D, int FMT, int NR, bool PRE>
__global__ void __launch_bounds__(32, (TreeLayout<D, FMT, NR>::WARPS))
tree_split(const __grid_constant__ TreeArgs a) {
  using L = TreeLayout<D, FMT, NR>;
  constexpr bool B16 = L::B16;
  constexpr int KT = L::KT, KH = KT / 16, KE = 4 * KH;  // keys of a tile, MMA steps, keys of a lane
  constexpr int RL = NR / 8;             // rows of a lane: g (and g + 8)
  constexpr int NB = NR == 8 ? D / 16 : D / 8;  // accumulator blocks
  constexpr int DB = D / 8;  // 8-bit formats: consecutive columns of a lane's V pieces
  extern __shared__ __align__(128) char smem[];
  const int lane = threadIdx.x, g = lane >> 2, t4 = lane & 3;
  int* idx = reinterpret_cast<int*>(smem + L::OFF_IDX);
  uint32_t* msk = reinterpret_cast<uint32_t*>(smem + L::OFF_MSK);
  int* cnt = reinterpret_cast<int*>(smem + L::OFF_CNT);
  const uint32_t ring = smem_u32(smem);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Rows of a partial tile beyond its keys keep older rows; zero them once so that they
  // are finite (their probabilities are exactly zero).
  for (int o = 16 * lane; o < L::STAGES * L::STAGE; o += 512)
    *reinterpret_cast<uint4*>(smem + o) = make_uint4(0u, 0u, 0u, 0u);

  const int64_t kvrow = (int64_t)a.H_kv * D;  // elements per slot
  constexpr int ES = B16 ? 2 : 1;

  const Slice slice = slice_of<PRE>(a, blockIdx.x, lane);
  for_segments<PRE>(a, slice, blockIdx.x, lane, [&](int64_t partial, int kvh, int rg, int b, int len, int js, int je) {
    // The rows: row x of the group is query head x % gq of drafted token x / gq.  With all
    // rows of one token its list of keys is exact and needs no test per element.
    const int r_end = min(a.rows - rg * NR, NR);
    const bool one_token = (rg * NR) / a.gq == (rg * NR + r_end - 1) / a.gq;
    const int rho = kvh / (a.H_kv / a.R);
    const uint32_t* M = a.mask + ((int64_t)cache_of<PRE>(b) * a.R + rho) * a.cap;

    // ---- this lane's rows, g and g + 8
    uint64_t word[RL];
    uint32_t mrow[RL];
    int near[RL];         // first position inside the window
    float fac[RL];        // logit (log2) = MMA result * fac (* K scale)
    uint32_t qa[D / 16][2 * RL];
#pragma unroll
    for (int e = 0; e < RL; ++e) {
      const int r = g + 8 * e;
      bool on = r < r_end;
      const int x = rg * NR + (on ? r : 0), t = x / a.gq, h = kvh * a.gq + x % a.gq;
      int64_t token = (int64_t)b * a.T + t;
      if constexpr (PRE) {
        const Drafted tok(a, b, t);
        on = on && tok.some;
        token = tok.x;
        word[e] = on ? tok.word : 0ull;
        near[e] = word[e] ? tok.near(a) : INT_MAX;
        mrow[e] = word[e] ? tok.groups(a, rho) : 0u;
      } else {
        word[e] = on ? tree_word(a, b, t) : 0ull;
        near[e] = word[e] ? len + __popcll(word[e]) - a.w : INT_MAX;
        mrow[e] = word[e] ? __ldg(M + len + t) : 0u;
      }
      fac[e] = a.sl2;
      const bf16* qr = a.q + (token * a.H + h) * D;
      if constexpr (B16) {
        const uint32_t* qw = reinterpret_cast<const uint32_t*>(qr);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          qa[c][e] = on ? __ldg(qw + 8 * c + t4) : 0u;
          qa[c][RL + e] = on ? __ldg(qw + 8 * c + 4 + t4) : 0u;
        }
      } else {
        // Step (c, i) multiplies columns 64 c + 16 t4 + 4 i .. + 3: the order of a
        // product's columns is free, and this one reads K in 16-byte pieces.
        float f[D / 4];
        float mx = 0.0f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t w = on ? __ldg(reinterpret_cast<const uint32_t*>(qr) + 32 * c + 8 * t4 + i) : 0u;
            f[16 * c + 2 * i] = __uint_as_float(w << 16);
            f[16 * c + 2 * i + 1] = __uint_as_float(w & 0xffff0000u);
            mx = fmaxf(mx, fmaxf(fabsf(f[16 * c + 2 * i]), fabsf(f[16 * c + 2 * i + 1])));
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        float up, down;
        row_unit(mx, up, down);
        fac[e] *= down;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          qa[c][e] = pack_f16(f[4 * c] * up, f[4 * c + 1] * up);
          qa[c][RL + e] = pack_f16(f[4 * c + 2] * up, f[4 * c + 3] * up);
        }
      }
    }
    // ---- what any row of the group sees
    const uint64_t any2 = word[0] | word[RL - 1];
    const uint32_t many = __reduce_or_sync(0xffffffffu, mrow[0] | mrow[RL - 1]);
    const int nearest = __reduce_min_sync(0xffffffffu, min(near[0], near[RL - 1]));
    const uint32_t wlo = __reduce_or_sync(0xffffffffu, (uint32_t)any2);
    const uint32_t whi = __reduce_or_sync(0xffffffffu, (uint32_t)(any2 >> 32));
    const uint64_t any_word = (uint64_t)whi << 32 | wlo;

    // ---- listing: keys of [js, je) in blocks, tiles issued from a block's list
    int jb = js, ncomp = 0, at = 0;
    constexpr int MW = L::BLOCK / 32;
    uint32_t mw[MW];
#pragma unroll
    for (int t = 0; t < MW; ++t) {
      const int j = jb + 32 * t + lane;
      mw[t] = j < je ? __ldg(M + j) : 0u;
    }
    const char* kb = reinterpret_cast<const char*>(a.kc) + ((int64_t)cache_of<PRE>(b) * a.cap * kvrow + (int64_t)kvh * D) * ES;
    const char* vb = reinterpret_cast<const char*>(a.vc) + ((int64_t)cache_of<PRE>(b) * a.cap * kvrow + (int64_t)kvh * D) * ES;
    const float* ksc = B16 ? nullptr : a.ks + ((int64_t)cache_of<PRE>(b) * a.H_kv + kvh) * a.cap;
    const float* vsc = B16 ? nullptr : a.vs + ((int64_t)cache_of<PRE>(b) * a.H_kv + kvh) * a.cap;

    auto issue = [&](int s) -> bool {
      while (at >= ncomp) {
        if (jb >= je) return false;
        ncomp = 0;
#pragma unroll
        for (int t = 0; t < MW; ++t) {
          const int j = jb + 32 * t + lane;
          bool ok = j < je;
          if (ok) {
            if (PRE || j < len) {
              ok = j >= nearest || (mw[t] & many) != 0u;
            } else {
              const int u = j - len;
              ok = (any_word >> u & 1ull) != 0ull;
              if (ok && one_token)  // the window among drafted tokens: by their depths
                ok = len + __popcll(tree_word(a, b, u)) - 1 >= nearest || (mw[t] & many) != 0u;
            }
          }
          const unsigned bal = __ballot_sync(0xffffffffu, ok);
          if (ok) {
            const int x = ncomp + __popc(bal & lanemask_lt());
            idx[x] = j;
            if (!one_token) msk[x] = mw[t];
          }
          ncomp += __popc(bal);
        }
        jb += L::BLOCK;
#pragma unroll
        for (int t = 0; t < MW; ++t) {  // the next block's words, in flight meanwhile
          const int j = jb + 32 * t + lane;
          mw[t] = j < je ? __ldg(M + j) : 0u;
        }
        at = 0;
        __syncwarp();
      }
      const int n = min(KT, ncomp - at);
      const uint32_t st = ring + s * L::STAGE;
      if (lane == 0) cnt[s] = n;
      if (!one_token && lane < n) {
        int* key = reinterpret_cast<int*>(smem + s * L::STAGE + L::OFF_KEY);
        key[lane] = idx[at + lane];
        key[KT + lane] = (int)msk[at + lane];
      }
      constexpr int CH = D * ES / 16, RPI = 32 / CH;  // 16-byte pieces per row, rows per instruction
      const int ch = lane % CH;
      for (int rr = lane / CH; rr < n; rr += RPI) {
        const int64_t off = (int64_t)idx[at + rr] * kvrow * ES + 16 * ch;
        if constexpr (B16) {
          cp_async16(st + rr * L::ROW + 16 * ch, kb + off);
          cp_async16(st + (KT + rr) * L::ROW + 16 * ch, vb + off);
        } else {
          cp_async16(st + k_piece<D>(rr, ch), kb + off);
          cp_async16(st + KT * D + v_piece<D>(rr, ch), vb + off);
        }
      }
      if constexpr (!B16) {
        if (lane < n) {
          cp_async4(st + L::OFF_SCALE + 4 * lane, ksc + idx[at + lane]);
          cp_async4(st + L::OFF_SCALE + 4 * (KT + lane), vsc + idx[at + lane]);
        }
      }
      cp_async_commit();
      at += n;
      return true;
    };

    // m: reference of the logits and of their sum l.  8-bit formats: mo is that of acc, that is of
    // P times V's scale.  The two are apart since V's scales may lie further from another than
    // fp32's exponents reach, and a key counts in l whatever its V row's size.
    float m[RL], mo[RL], l[RL], acc[NB][4];
#pragma unroll
    for (int r = 0; r < RL; ++r) m[r] = mo[r] = -INFINITY, l[r] = 0.0f;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;
    // Accumulator e's share of a number per row: NR = 8 has rows 2 t4, 2 t4 + 1 as columns
    // (their statistics sit in lanes 8 t4, 8 t4 + 4), NR = 16 has rows g, g + 8.
    auto of_rows = [&](const float(&x)[RL], float(&f)[4]) {
      if constexpr (NR == 8) {
        f[0] = f[2] = __shfl_sync(0xffffffffu, x[0], 8 * t4);
        f[1] = f[3] = __shfl_sync(0xffffffffu, x[0], 8 * t4 + 4);
      } else {
        f[0] = f[1] = x[0];
        f[2] = f[3] = x[RL - 1];
      }
    };
    __syncwarp();  // zeroed stages (and the last stretch's reads) before the first copy
    int issued = 0;  // one copy group per stage and per refill, empty or not
    for (int s = 0; s < L::STAGES; ++s) {
      if (issue(s)) ++issued;
      else cp_async_commit();
    }
    for (int t = 0; t < issued; ++t) {
      const int s = t % L::STAGES;
      cp_async_wait<L::STAGES - 1>();  // tile t's group has landed (this lane's copies)
      __syncwarp();                    // ... and every lane's
      const int n = cnt[s];
      const uint32_t st = ring + s * L::STAGE;
      float sc[2 * KH][4];  // scores of keys 8 i .. 8 i + 7
#pragma unroll
      for (int i = 0; i < 2 * KH; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[i][e] = 0.0f;
      if constexpr (B16) {
        const uint32_t ka = st + ((lane & 7) + ((lane >> 4) << 3)) * L::ROW + ((lane >> 3) & 1) * 16;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t r0, r1, r2, r3;
          ldsm_x4(ka + 32 * c, r0, r1, r2, r3);
          const uint32_t* A = qa[c];
          mma_bf16(sc[0], A[0], RL == 2 ? A[1] : 0u, A[RL], RL == 2 ? A[2 * RL - 1] : 0u, r0, r1);
          mma_bf16(sc[1], A[0], RL == 2 ? A[1] : 0u, A[RL], RL == 2 ? A[2 * RL - 1] : 0u, r2, r3);
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint4 x[2 * KH];
#pragma unroll
          for (int h = 0; h < 2 * KH; ++h) x[h] = lds128(st + k_piece<D>(g + 8 * h, 4 * c + t4));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t* A = qa[4 * c + i];
#pragma unroll
            for (int h = 0; h < 2 * KH; ++h) {
              uint32_t b0, b1;
              codes_f16x2<FMT>(i == 0 ? x[h].x : i == 1 ? x[h].y : i == 2 ? x[h].z : x[h].w, b0, b1);
              mma_f16(sc[h], A[0], RL == 2 ? A[1] : 0u, A[RL], RL == 2 ? A[2 * RL - 1] : 0u, b0, b1);
            }
          }
        }
      }
      // ---- logits (log2) of rows g, g + 8 and the lane's keys: 2 t4, 2 t4 + 1 of each eight
      float sx[RL][KE], vf[KE], lv[KE];
      const float* scale = reinterpret_cast<const float*>(smem + s * L::STAGE + L::OFF_SCALE);
#pragma unroll
      for (int e = 0; e < KE; ++e) {
        const int i = e >> 1, key = 8 * i + 2 * t4 + (e & 1);
        const float kf = B16 ? 1.0f : scale[key];
        if constexpr (!B16) vf[e] = scale[KT + key];
#pragma unroll
        for (int r = 0; r < RL; ++r) sx[r][e] = sc[i][2 * r + (e & 1)] * (kf * fac[r]);
      }
      if (!one_token || n < KT) {  // keys beyond the tile's, and those that a row does not see
        const int* keys = reinterpret_cast<const int*>(smem + s * L::STAGE + L::OFF_KEY);
        const bool drafts = !PRE && !one_token && keys[n - 1] >= len;  // slots ascend in a list
#pragma unroll
        for (int e = 0; e < KE; ++e) {
          const int key = 8 * (e >> 1) + 2 * t4 + (e & 1);
          bool see[RL];
          see[0] = see[RL - 1] = key < n;
          if (!B16 && key >= n) vf[e] = 0.0f;
          if (!one_token && key < n) {
            const int j = keys[key];
            const uint32_t mk = (uint32_t)keys[KT + key];
            int p = j;
            uint64_t bit = ~0ull;
            if (drafts && j >= len) {
              p = len + __popcll(tree_word(a, b, j - len)) - 1;
              bit = 1ull << (j - len);
            }
#pragma unroll
            for (int r = 0; r < RL; ++r)
              see[r] = (word[r] & bit) != 0ull && (p >= near[r] || (mk & mrow[r]) != 0u);
          }
#pragma unroll
          for (int r = 0; r < RL; ++r)
            if (!see[r]) sx[r][e] = -INFINITY;
        }
      }
      // ---- 8-bit formats: V's scales join P before it is rounded to fp16, and the reference
      // mo of a row is that of the product, which fp16 has to hold: its largest P vs is about
      // 2^14, so that what is smaller by up to 2^-38 still counts.  Scales within 2^4 of
      // another are bounded by one power of two, others (an outlier that a row may not even
      // see) measured key by key.
      float lift = 0.0f;
      bool wide = false;
      if constexpr (!B16) {
        const uint32_t u = lane < n ? __float_as_uint(fabsf(scale[KT + lane])) : 0u;
        const uint32_t top = __reduce_max_sync(0xffffffffu, u);
        const uint32_t low = __reduce_min_sync(0xffffffffu, u ? u : 0x7f800000u);
        wide = top >= 0x7f000000u || __uint_as_float(top) > 16.0f * __uint_as_float(low);
        lift = (float)max((int)(top >> 23) - 126, -80) - kPTop;
        if (wide) {
#pragma unroll
          for (int e = 0; e < KE; ++e) {
            if (!(fabsf(vf[e]) < INFINITY)) vf[e] = __uint_as_float(0x7fc00000u);
            lv[e] = __log2f(fmaxf(fabsf(vf[e]), kTinyScale)) - kPTop;
          }
        }
      }
      // P is rounded for the tensor core (bf16, as in the forward pass; in 8 bits times V's scale,
      // once, to fp16); l sums it unrounded.
      float corr[RL];  // of acc
      uint32_t pa[RL][2 * KH];
#pragma unroll
      for (int r = 0; r < RL; ++r) {
        float mt = -INFINITY, mv = -INFINITY;  // largest logit; 8-bit formats: with V's scale
        if (!B16 && wide) {
#pragma unroll
          for (int e = 0; e < KE; ++e) mv = fmaxf(mv, sx[r][e] + lv[e]);
          mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, 1));
          mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, 2));
        }
#pragma unroll
        for (int e = 0; e < KE; e += 2) mt = max3(mt, sx[r][e], sx[r][e + 1]);
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
        const float mn = fmaxf(m[r], mt);
        const float mu = mn == -INFINITY ? 0.0f : mn;  // a row without a key so far
        const float fl = ex2(m[r] - mu);
        float p[KE], sum = 0.0f;
#pragma unroll
        for (int e = 0; e < KE; ++e) p[e] = ex2(sx[r][e] - mu);
#pragma unroll
        for (int e = 0; e < KE; e += 2) sum += p[e] + p[e + 1];
        l[r] = l[r] * fl + sum;
        m[r] = mn;
        if constexpr (B16) {
          corr[r] = fl;
#pragma unroll
          for (int i = 0; i < 2 * KH; ++i) pa[r][i] = pack_bf16(p[2 * i], p[2 * i + 1]);
        } else {
          const float on = fmaxf(mo[r], wide ? mv : mt + lift);
          const float ou = on == -INFINITY ? 0.0f : on;
          corr[r] = ex2(mo[r] - ou);
          mo[r] = on;
          const float c = ex2(mu - ou);  // (2^-114 .. 2^94)
#pragma unroll
          for (int i = 0; i < 2 * KH; ++i) {
            float y0, y1;
            fmul2(y0, y1, p[2 * i], p[2 * i + 1], vf[2 * i], vf[2 * i + 1]);
            fmul2(y0, y1, y0, y1, c, c);
            pa[r][i] = pack_f16(y0, y1);
          }
        }
      }
      if (__any_sync(0xffffffffu, corr[0] != 1.0f || corr[RL - 1] != 1.0f)) {
        float f[4];
        of_rows(corr, f);
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] *= f[e];
      }
      if constexpr (B16) {
        const uint32_t va = st + (KT + (NR == 8 ? (lane & 7) + ((lane >> 4) << 3) : (lane & 15))) * L::ROW +
                            (NR == 8 ? (lane >> 3) & 1 : lane >> 4) * 16;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t r0, r1, r2, r3;
          ldsm_x4_t(va + 32 * i, r0, r1, r2, r3);
          if constexpr (NR == 8) {
            mma_bf16(acc[i], r0, r1, r2, r3, pa[0][0], pa[0][1]);
          } else {
            mma_bf16(acc[2 * i], pa[0][0], pa[RL - 1][0], pa[0][1], pa[RL - 1][1], r0, r1);
            mma_bf16(acc[2 * i + 1], pa[0][0], pa[RL - 1][0], pa[0][1], pa[RL - 1][1], r2, r3);
          }
        }
      } else {
        // keys 2 t4, 2 t4 + 1 and those + 8 of columns DB g .. DB g + DB - 1: byte i of a key
        // pair is what the MMA takes for column DB g + i of O, as column g of block i
        // (NR = 16) or as row g (+ 8) of block i / 2
#pragma unroll
        for (int h = 0; h < KH; ++h) {
          uint32_t vw[4][DB / 4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = 16 * h + 8 * (e >> 1) + 2 * t4 + (e & 1);
            if constexpr (D == 128) {
              const uint4 x = lds128(st + KT * D + v_piece<D>(key, g));
              vw[e][0] = x.x, vw[e][1] = x.y, vw[e][2] = x.z, vw[e][3] = x.w;
            } else {
              const uint2 x = lds64(st + KT * D + v_piece<D>(key, g >> 1) + 8 * (g & 1));
              vw[e][0] = x.x, vw[e][1] = x.y;
            }
          }
          const uint32_t p0 = pa[0][2 * h], p1 = pa[0][2 * h + 1], p2 = pa[RL - 1][2 * h], p3 = pa[RL - 1][2 * h + 1];
#pragma unroll
          for (int i = 0; i < DB / 4; ++i) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const uint32_t sel = hh ? 0x7362u : 0x5140u;
              uint32_t x0, x1, y0, y1;
              codes_f16x2<FMT>(__byte_perm(vw[0][i], vw[1][i], sel), x0, x1);
              codes_f16x2<FMT>(__byte_perm(vw[2][i], vw[3][i], sel), y0, y1);
              if constexpr (NR == 8) {
                mma_f16(acc[2 * i + hh], x0, x1, y0, y1, p0, p1);
              } else {
                const int blk = 4 * i + 2 * hh;
                mma_f16(acc[blk], p0, p2, p1, p3, x0, y0);
                mma_f16(acc[blk + 1], p0, p2, p1, p3, x1, y1);
              }
            }
          }
        }
      }
      __syncwarp();  // every lane is done with the stage
      if (issue(s)) ++issued;
      else cp_async_commit();
    }
    // ---- this segment's partial (8-bit formats: acc goes over to the reference of l)
    const int64_t slot = partial * NR;
    if constexpr (!B16) {
      float f[4], back[RL];
#pragma unroll
      for (int r = 0; r < RL; ++r) back[r] = ex2(mo[r] - m[r]);
      of_rows(back, f);
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] *= f[e];
    }
#pragma unroll
    for (int r = 0; r < RL; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (t4 == 0 && g + 8 * r < r_end) a.part_ml[slot + g + 8 * r] = make_float2(m[r], l[r]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if constexpr (NR == 8) {  // row 2 t4 + e
        if (2 * t4 + e >= r_end) continue;
        float* dst = a.part_acc + (slot + 2 * t4 + e) * D;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          if constexpr (B16) {
            dst[16 * i + g] = acc[i][e];
            dst[16 * i + g + 8] = acc[i][2 + e];
          } else {
            *reinterpret_cast<float2*>(dst + DB * g + 2 * i) = make_float2(acc[i][e], acc[i][2 + e]);
          }
        }
      } else {  // row g + 8 e
        if (g + 8 * e >= r_end) continue;
        float* dst = a.part_acc + (slot + g + 8 * e) * D;
        if constexpr (B16) {
#pragma unroll
          for (int i = 0; i < NB; ++i)
            *reinterpret_cast<float2*>(dst + 8 * i + 2 * t4) = make_float2(acc[i][2 * e], acc[i][2 * e + 1]);
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < NB; i += 4)
              *reinterpret_cast<float4*>(dst + DB * (2 * t4 + c) + i) =
                  make_float4(acc[i][2 * e + c], acc[i + 1][2 * e + c], acc[i + 2][2 * e + c], acc[i + 3][2 * e + c]);
        }
      }
    }
  });
  // (the own part's kernel, beside which this one runs, is done when this one is)
  if constexpr (PRE) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------------ combine --
template <int FMT>
__device__ __forceinline__ float cache_value(const void* x, int64_t at) {
  if constexpr (FMT == FOCUS_CACHE_BF16) return __bfloat162float(reinterpret_cast<const bf16*>(x)[at]);
  else if constexpr (FMT == FOCUS_CACHE_INT8) return (float)reinterpret_cast<const int8_t*>(x)[at];
  else {
    const __half_raw r = __nv_cvt_fp8_to_halfraw(reinterpret_cast<const __nv_fp8_storage_t*>(x)[at], __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&r));
  }
}

// Where the partials of row (t, h) of sequence b are.
template <bool PRE>
struct RowParts {
  int64_t ln, from, whole, part;
  Stretch s;
  int b, len, row, ns, first, last, n;  // slices first .. last may hold a part; n: partials to look at

  // Partial c of those to look at: its place, and its keys as [keys.x, keys.y).
  __device__ __forceinline__ bool find(const TreeArgs& a, int c, int64_t& slot, int2& keys) const {
    const int sl = first + c;
    const int64_t lo = slice_at(whole, ns, part, sl), hi = slice_at(whole, ns, part, sl + 1);
    keys = make_int2(units_before(a, s, lo - from) * kTreeUnit, units_before(a, s, hi - from) * kTreeUnit);
    if (keys.x >= keys.y) return false;  // no such partial
    slot = (sl + ln * a.B + b) * a.grp + row % a.grp;
    return true;
  }
  // (max, sum) of that partial; NaN where its slice gave up, so that nothing stale passes for a result.
  __device__ __forceinline__ float2 sums(const TreeArgs& a, int c, int64_t slot) const {
    const float2 x = a.part_ml[slot];
    if (a.flags && a.flags[first + c] != 0) return make_float2(__uint_as_float(0x7fc00000u), __uint_as_float(0x7fc00000u));
    return x;
  }
};

// All of a warp's lanes; total: all sequences' weight, bad: some length is out of range.
template <bool PRE>
__device__ __forceinline__ RowParts<PRE> row_parts(const TreeArgs& a, int b, int t, int h, int lane, int64_t& total, bool& bad) {
  RowParts<PRE> r;
  r.b = b, r.row = t * a.gq + h % a.gq;
  r.ln = (int64_t)(h / a.gq) * a.nrg + r.row / a.grp;
  total = 0, r.from = 0, bad = false;
  for (int x = lane; x < a.B; x += 32) {
    const int n = keys_of<PRE>(a, x);
    const int64_t wgt = stretch_of<PRE>(a, x, n).weight;
    bad = bad || !len_ok<PRE>(a, n);
    total += wgt;
    r.from += x < b ? wgt : 0;  // those before sequence b
  }
  total = warp_sum(total);
  r.from = warp_sum(r.from) + r.ln * total;
  bad = __any_sync(0xffffffffu, bad);
  r.len = keys_of<PRE>(a, b);
  r.s = stretch_of<PRE>(a, b, r.len);
  r.whole = total * a.H_kv * a.nrg;
  r.ns = slices_of<PRE>(a, r.whole);
  bool live = r.s.units > 0;
  if constexpr (PRE) live = live && Drafted(a, b, t).word != 0ull;
  else live = live && tree_word(a, b, t) != 0ull;
  r.part = quotient(r.whole, r.ns);  // a slice is `part` weights or one more
  r.first = live ? (int)max((int64_t)0, quotient(r.from, r.part + 1) - 1) : 0;
  r.last = live ? (int)min((int64_t)r.ns - 1, quotient(r.from + r.s.weight, r.part) + 1) : -1;
  r.n = r.last - r.first + 1;
  return r;
}

// All partials of a row: the prefix's or the only ones (a), behind them the own sequence's (o) of a batch
// behind a prefix.
template <bool PRE>
struct Parts {
  RowParts<PRE> p;
  RowParts<false> q;
  int n;       // partials to look at
  int tp, tq;  // the token's number in its run (or sequence), in its own sequence
  bool bad;   // some length is out of range
  int64_t total, total_q;

  // Token t of sequence b; over a prefix token b T + t of the batch's row.
  __device__ __forceinline__ Parts(const TreeArgs& a, const TreeArgs& o, int b, int t, int h, int lane) {
    const int x = PRE ? min(b * a.T + t, a.tokens - 1) : 0;
    bool placed = true;
    if (PRE && a.order) {
      const int at = __ldg(a.place + x);
      placed = at >= 0;
      b = max(at, 0) / a.T, t = max(at, 0) % a.T;
    }
    tp = t;
    p = row_parts<PRE>(a, b, t, h, lane, total, bad);
    if (!placed) p.n = 0;
    n = p.n;
    if constexpr (PRE) {
      tq = x % a.per;
      q = row_parts<false>(o, x / a.per, tq, h, lane, total_q, bad);
      n += q.n;
    }
  }
  // Partial c: the place of its sums in o.part_acc or a.part_acc (from a.part_acc), and its keys.
  template <int D>
  __device__ __forceinline__ bool find(const TreeArgs& a, const TreeArgs& o, int c, int64_t& slot, int64_t& place, int2& keys) const {
    if (!PRE || c < p.n) {
      if (!p.find(a, c, slot, keys)) return false;
      place = slot * D;
    } else {
      if (!q.find(o, c - p.n, slot, keys)) return false;
      place = slot * D + (o.part_acc - a.part_acc);
    }
    return true;
  }
  __device__ __forceinline__ float2 sums(const TreeArgs& a, const TreeArgs& o, int c, int64_t slot) const {
    return !PRE || c < p.n ? p.sums(a, c, slot) : q.sums(o, c - p.n, slot);
  }
  // The call's status, by one warp.
  __device__ __forceinline__ void put_status(const TreeArgs& a, const TreeArgs& o, int lane) const {
    int code = 0;
    if (a.flags && total > 0)
      for (int x = lane; x < p.ns; x += 32) code = min(code, a.flags[x]);
    if constexpr (PRE) {
      if (o.flags && total_q > 0)
        for (int x = lane; x < q.ns; x += 32) code = min(code, o.flags[x]);
    }
    code = __reduce_min_sync(0xffffffffu, code);
    if (lane == 0) *a.status = code ? code : bad ? FOCUS_ERR_BOUNDS : 0;
  }
};

// Shared memory of rows that are worked out again.
template <int NT>
struct Again {
  float weight[NT], x[NT];  // of partial results, of keys
  int key[NT];
  int64_t place[NT];
  int2 range[NT];
  unsigned bits[NT / 32], bad[NT / 32];
};

// Keys [js, je) of one row again, without the keys that it does not see: a thread per key
// lists NT keys, a warp per listed key takes its weight, NT / D groups of D threads sum the
// values, a key each at a time.  Returns the thread's share of column threadIdx.x % D.
template <int D, int FMT, int NT, bool PRE>
__device__ float keys_by_hand(const TreeArgs& a, const RowParts<PRE>& rp, int t, int h, float lse2, int js, int je, Again<NT>& sh) {
  constexpr int V = D / 32, NW = NT / 32, NG = NT / D, U = 4;
  const int b = rp.b, len = rp.len, kvh = h / a.gq, rho = kvh / (a.H_kv / a.R);
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, g = threadIdx.x / D, d = threadIdx.x % D;
  const uint32_t* M = a.mask + ((int64_t)cache_of<PRE>(b) * a.R + rho) * a.cap;
  uint64_t word;
  int near;
  uint32_t mrow;
  int64_t token = (int64_t)b * a.T + t;
  if constexpr (PRE) {
    const Drafted tok(a, b, t);
    word = tok.word, near = tok.near(a), mrow = tok.groups(a, rho), token = tok.x;
  } else {
    word = tree_word(a, b, t);
    near = len + __popcll(word) - a.w;
    mrow = M[len + t];
  }
  const bf16* q = a.q + (token * a.H + h) * D + V * lane;
  float qf[V];
#pragma unroll
  for (int v = 0; v < V; ++v) qf[v] = __bfloat162float(q[v]);
  float fac = a.sl2;
  if constexpr (FMT != FOCUS_CACHE_BF16) {  // (scaled as in the kernels: a large query times codes may pass fp32)
    float mx = 0.0f, up, down;
#pragma unroll
    for (int v = 0; v < V; ++v) mx = fmaxf(mx, fabsf(qf[v]));
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    row_unit(mx, up, down);
    fac *= down;
#pragma unroll
    for (int v = 0; v < V; ++v) qf[v] *= up;
  }
  const int64_t sc = ((int64_t)cache_of<PRE>(b) * a.H_kv + kvh) * a.cap;
  const int64_t row0 = ((int64_t)cache_of<PRE>(b) * a.cap * a.H_kv + kvh) * D;
  const int64_t kvrow = (int64_t)a.H_kv * D;
  float out = 0.0f;
  for (int j0 = js; j0 < je; j0 += NT) {
    const int j = j0 + threadIdx.x;
    bool see = j < je;
    if (see) {
      int p = j;
      if (!PRE && j >= len) {
        see = (word >> (j - len) & 1ull) != 0ull;
        p = len + __popcll(tree_word(a, b, j - len)) - 1;
      }
      see = see && (p >= near || (M[j] & mrow) != 0u);
    }
    const unsigned seen = __ballot_sync(0xffffffffu, see);
    if (lane == 0) sh.bits[wp] = seen;
    __syncthreads();
    int n = 0, at = 0;
    for (int i = 0; i < NW; ++i) {
      at += i < wp ? __popc(sh.bits[i]) : 0;
      n += __popc(sh.bits[i]);
    }
    if (see) sh.key[at + __popc(seen & lanemask_lt())] = j;
    __syncthreads();
    for (int i0 = wp; i0 < n; i0 += U * NW) {
      float x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        x[u] = 0.0f;
        if (i0 + u * NW < n) {
          const int64_t from = row0 + sh.key[i0 + u * NW] * kvrow + V * lane;
#pragma unroll
          for (int v = 0; v < V; ++v) x[u] += qf[v] * cache_value<FMT>(a.kc, from + v);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int o = 16; o; o >>= 1) x[u] += __shfl_xor_sync(0xffffffffu, x[u], o);
        if (lane == 0 && i0 + u * NW < n) {
          const int k = sh.key[i0 + u * NW];
          if constexpr (FMT != FOCUS_CACHE_BF16) x[u] *= a.ks[sc + k] * fac;
          else x[u] *= fac;
          x[u] = ex2(x[u] - lse2);
          if constexpr (FMT != FOCUS_CACHE_BF16) x[u] *= a.vs[sc + k];
          sh.x[i0 + u * NW] = x[u];
        }
      }
    }
    __syncthreads();
    float part = 0.0f;  // (a sum of its own per NT keys: no chain over a long sequence)
#pragma unroll 8
    for (int i = g; i < n; i += NG) part += sh.x[i] * cache_value<FMT>(a.vc, row0 + sh.key[i] * kvrow + d);
    out += part;
    __syncthreads();
  }
  return out;
}

// A row whose output came out not finite, again, by all of a block's threads: a NaN or an
// infinity in the V row of a key that it does not see, which other rows of the MMA do see, has
// met a zero weight there and spoilt the sum, or weights and values that fp32 holds had a
// product that it does not.  The partial results are merged again with weights that sum up to
// one, and those that are not finite are worked out again key by key: their part of the
// sequence, not all of it.  Returns column threadIdx.x of the output (threads below D).
// Measured, one such key that half of the tokens see behind 100000 keys: one token 0.07 -> 0.13
// ms, 16 drafts int8 0.15 -> 0.96 (bf16 0.12 -> 0.88), 64 drafts 0.22 -> 2.8 (0.18 -> 2.5); three
// in different slices, 16 drafts: 2.5.
template <int D, int FMT, int NT, bool PRE>
__device__ __noinline__ float row_again(const TreeArgs& a, const TreeArgs& o, const Parts<PRE>& rp, int h, float lse2, Again<NT>& sh) {
  constexpr int NG = NT / D, NW = NT / 32;
  const int tid = threadIdx.x, g = tid / D, d = tid % D;
  float acc = 0.0f;
  for (int base = 0; base < rp.n; base += NT) {
    const int c = base + tid;
    int64_t slot = 0, place = 0;
    int2 range = make_int2(0, 0);
    float w = 0.0f;
    if (c < rp.n && rp.template find<D>(a, o, c, slot, place, range)) {
      const float2 x = (!PRE || c < rp.p.n ? a : o).part_ml[slot];
      if (x.y != 0.0f) w = ex2(x.x - lse2);
    }
    sh.weight[tid] = w;
    sh.place[tid] = place;
    sh.range[tid] = range;
    if (tid < NW) sh.bad[tid] = 0u;
    __syncthreads();
    const int end = min(NT, rp.n - base);
    for (int i = g; i < end; i += NG) {
      if (sh.weight[i] == 0.0f) continue;
      const float p = a.part_acc[sh.place[i] + d];
      if (fabsf(p) < INFINITY) acc += sh.weight[i] * p;
      else atomicOr(&sh.bad[i >> 5], 1u << (i & 31));
    }
    __syncthreads();
    for (int i = 0; i < end; ++i) {
      if (!(sh.bad[i >> 5] >> (i & 31) & 1u)) continue;
      const bool mine = !(fabsf(a.part_acc[sh.place[i] + d]) < INFINITY);
      const int2 keys = sh.range[i];
      float x;
      if (!PRE || base + i < rp.p.n)
        x = keys_by_hand<D, FMT, NT>(a, rp.p, rp.tp, h, lse2, keys.x, min(keys.y, rp.p.len + drafts_of<PRE>(a)), sh);
      else
        x = keys_by_hand<D, FMT, NT>(o, rp.q, rp.tq, h, lse2, keys.x, min(keys.y, rp.q.len + o.T), sh);
      if (mine) acc += x;
    }
    __syncthreads();
  }
  // the groups' shares
  sh.weight[tid] = acc;
  __syncthreads();
  if (tid < D)
    for (int i = 1; i < NG; ++i) acc += sh.weight[i * D + tid];
  __syncthreads();
  return acc;
}

// Where the sum of a row of run b of a batch behind a prefix goes.
__device__ __forceinline__ int64_t lse_at(const TreeArgs& a, int b, int t, int h) {
  const int x = b * a.T + t;
  return ((int64_t)(x / a.per) * a.H + h) * a.per + x % a.per;
}

// Merge the partials of one row: grid (T * H, B), NT threads.  A pass takes NT of the
// slices that may hold a part of the row's sequence: a thread finds out whether its slice
// does, and its partial's (max, sum); with the largest maximum of all the weights are known,
// and NT / D groups of D threads sum the weighted partials, each a share of them, with no
// chain from one to the next (merging them pair by pair, a warp's share in order, took 46 us
// behind 128K tokens).  A programmatic dependent of the kernel that writes the partials.
template <int D, int FMT, int NT, bool PRE>
__global__ void __launch_bounds__(NT) tree_combine(const __grid_constant__ TreeArgs a, const __grid_constant__ TreeArgs o) {
  constexpr int NG = NT / D, NW = NT / 32, U = 8;
  __shared__ Again<NT> sh;
  __shared__ float sums[NG][D];
  __shared__ float red[2][NW];
  const int tid = threadIdx.x, wp = tid >> 5, lane = tid & 31, g = tid / D, d = tid % D;
  const int b = blockIdx.y, t = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const Parts<PRE> rp(a, o, b, t, h, lane);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && b == 0 && wp == 0) rp.put_status(a, o, lane);
  if (PRE && b * a.T + t >= a.tokens) return;
  float m = -INFINITY, l = 0.0f, acc = 0.0f;  // of all; this thread's shares
  for (int base = 0; base < rp.n; base += NT) {
    const int c = base + tid;
    float2 x = make_float2(-INFINITY, 0.0f);
    int64_t slot = 0, place = 0;
    int2 keys;
    if (c < rp.n && rp.template find<D>(a, o, c, slot, place, keys)) x = rp.sums(a, o, c, slot);
    const bool some = x.y != 0.0f;  // a key of the slice is seen
    float top = some ? x.x : -INFINITY;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) red[0][wp] = top;
    __syncthreads();
    for (int i = 0; i < NW; ++i) top = fmaxf(top, red[0][i]);
    // no maximum: nothing is seen, or all that is seen is NaN (a sum of NaN, which then makes
    // the row NaN); the same in every thread
    if (top == -INFINITY && !__syncthreads_or(some)) continue;
    const float mn = fmaxf(m, top), f = m == -INFINITY ? 0.0f : ex2(m - mn);
    const float w = some ? ex2(x.x - mn) : 0.0f;
    l = l * f + (some ? x.y * w : 0.0f);
    acc *= f;
    m = mn;
    sh.weight[tid] = w;
    sh.place[tid] = place;
    __syncthreads();
    const int end = min(NT, rp.n - base);
    if constexpr (NT == 128) {  // a thread has many to sum: U loads in flight
      for (int i0 = g; i0 < end; i0 += U * NG) {
        float y[U], p[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int at = i0 + i * NG;
          y[i] = at < end ? sh.weight[at] : 0.0f;
          p[i] = y[i] != 0.0f ? a.part_acc[sh.place[at] + d] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) acc += y[i] * p[i];
      }
    } else {
#pragma unroll 4
      for (int i = g; i < end; i += NG) {
        const float y = sh.weight[i];
        if (y != 0.0f) acc += y * a.part_acc[sh.place[i] + d];
      }
    }
    __syncthreads();
  }
  sums[g][d] = acc;
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) red[1][wp] = l;
  __syncthreads();
  float sum = 0.0f, out = 0.0f;
  for (int i = 0; i < NW; ++i) sum += red[1][i];
  if (tid < D)
    for (int i = 0; i < NG; ++i) out += sums[i][d];
  const bool empty = sum == 0.0f;
  const float lse2 = m + log2f(sum);
  out = empty ? 0.0f : out / sum;
  // (a sum that is not finite either has NaN of the row's own: the row is NaN)
  if (__syncthreads_or(tid < D && !(fabsf(out) < INFINITY)) && fabsf(lse2) < INFINITY)
    out = row_again<D, FMT, NT>(a, o, rp, h, lse2, sh);
  if (tid < D) a.o[(((int64_t)b * a.T + t) * a.H + h) * D + d] = __float2bfloat16_rn(out);
  if (tid == 0 && a.lse) a.lse[PRE ? lse_at(a, b, t, h) : ((int64_t)b * a.H + h) * a.T + t] = empty ? -INFINITY : lse2 * kLn2;
}

// The rows of a block of tree_combine_rows that came out not finite, one after another.  Out of
// line, so that the merge itself keeps its registers.
template <int D, int FMT, int NT, int R, bool PRE>
__device__ __noinline__ void rows_again(const TreeArgs& a, const TreeArgs& o, const int* again, const float* lse_of, Again<NT>& sh) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  for (int i = 0; i < NT / 32 * R; ++i) {
    if (!again[i]) continue;
    const int y = blockIdx.x * (NT / 32 * R) + i, t = y / a.H, h = y % a.H;
    const Parts<PRE> rp(a, o, b, t, h, lane);
    const float out = row_again<D, FMT, NT>(a, o, rp, h, lse_of[i], sh);
    if (threadIdx.x < D) a.o[(((int64_t)b * a.T + t) * a.H + h) * D + threadIdx.x] = __float2bfloat16_rn(out);
  }
}

// The same with a warp for R rows, for calls of many rows: grid (T * H / 8 R rounded up, B).  R > 1: query
// heads of one KV head (gq is a multiple of R), whose partials lie side by side: where they are is found
// once.  (That takes longer than the sums where sequences are short.)
template <int D, int FMT, int R, bool PRE>
__global__ void __launch_bounds__(256) tree_combine_rows(const __grid_constant__ TreeArgs a, const __grid_constant__ TreeArgs o) {
  constexpr int NT = 256, U = 8 / R, V = D / 32;  // V: columns of a lane
  using vec = std::conditional_t<V == 4, float4, float2>;
  __shared__ Again<NT> sh;
  __shared__ float lse_of[NT / 32 * R];
  const int wp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
  const int x = (blockIdx.x * 8 + wp) * R, t = min(x, a.T * a.H - 1) / a.H, h = x % a.H;
  const Parts<PRE> rp(a, o, b, t, h, lane);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (x == 0 && b == 0) rp.put_status(a, o, lane);
  const bool mine = x < a.T * a.H && (!PRE || b * a.T + t < a.tokens);
  float m[R], l[R], acc[R][V];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY, l[r] = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[r][v] = 0.0f;
  }
  for (int base = 0; mine && base < rp.n; base += 32) {
    float2 ml[R];
#pragma unroll
    for (int r = 0; r < R; ++r) ml[r] = make_float2(-INFINITY, 0.0f);
    int64_t slot = 0, place = 0;
    int2 keys;
    if (base + lane < rp.n && rp.template find<D>(a, o, base + lane, slot, place, keys)) {
#pragma unroll
      for (int r = 0; r < R; ++r) ml[r] = rp.sums(a, o, base + lane, slot + r);
    }
    float w[R];
    bool any = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool some = ml[r].y != 0.0f;  // a key of the slice is seen
      float top = some ? ml[r].x : -INFINITY;
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      w[r] = 0.0f;
      if (top == -INFINITY && !__any_sync(0xffffffffu, some)) continue;  // as above
      const float mn = fmaxf(m[r], top), f = m[r] == -INFINITY ? 0.0f : ex2(m[r] - mn);
      w[r] = some ? ex2(ml[r].x - mn) : 0.0f;
      l[r] = l[r] * f + (some ? ml[r].y * w[r] : 0.0f);
      m[r] = mn;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[r][v] *= f;
      any = true;
    }
    const int end = any ? min(32, rp.n - base) : 0;
    for (int i0 = 0; i0 < end; i0 += U) {  // U R loads in flight
      float y[U][R];
      vec p[U][R];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t from = __shfl_sync(0xffffffffu, place, i0 + i) + V * lane;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          y[i][r] = __shfl_sync(0xffffffffu, w[r], i0 + i);
          p[i][r] = vec{};
          if (y[i][r] != 0.0f) p[i][r] = *reinterpret_cast<const vec*>(a.part_acc + from + r * D);
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          acc[r][0] += y[i][r] * p[i][r].x, acc[r][1] += y[i][r] * p[i][r].y;
          if constexpr (V == 4) acc[r][2] += y[i][r] * p[i][r].z, acc[r][3] += y[i][r] * p[i][r].w;
        }
      }
    }
  }
  __shared__ int again[NT / 32 * R];
  bool some_odd = false;
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int o = 16; o; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
    const bool empty = l[r] == 0.0f;
    const float lse2 = m[r] + log2f(l[r]);
    bool odd = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      acc[r][v] = empty ? 0.0f : acc[r][v] / l[r];
      odd = odd || !(fabsf(acc[r][v]) < INFINITY);
    }
    if (mine) {
      bf16* to = a.o + (((int64_t)b * a.T + t) * a.H + h + r) * D + V * lane;
      if constexpr (V == 4)
        *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16(acc[r][0], acc[r][1]), pack_bf16(acc[r][2], acc[r][3]));
      else
        *reinterpret_cast<uint32_t*>(to) = pack_bf16(acc[r][0], acc[r][1]);
      if (lane == 0 && a.lse)
        a.lse[PRE ? lse_at(a, b, t, h + r) : ((int64_t)b * a.H + h + r) * a.T + t] = empty ? -INFINITY : lse2 * kLn2;
    }
    odd = __any_sync(0xffffffffu, odd && mine && fabsf(lse2) < INFINITY);  // (as above)
    if (lane == 0) again[wp * R + r] = odd, lse_of[wp * R + r] = lse2;
    some_odd = some_odd || odd;
  }
  if (!__syncthreads_or(some_odd)) return;
  // rows that are not finite, one after another, by all warps
  rows_again<D, FMT, NT, R, PRE>(a, o, again, lse_of, sh);
}

// ------------------------------------------------------------------------- launch --
constexpr int kTreeTcRows = 128;  // rows of a product of the tensor-core kernel (the MMA's M)

template <int NR>
int split_warps_of(int d_head, int format) {  // per SM
  constexpr int B = FOCUS_CACHE_BF16, E = FOCUS_CACHE_E4M3;
  return d_head == 64 ? (format == B ? TreeLayout<64, B, NR>::WARPS : TreeLayout<64, E, NR>::WARPS)
                      : (format == B ? TreeLayout<128, B, NR>::WARPS : TreeLayout<128, E, NR>::WARPS);
}
int split_warps(int d_head, int format, int rows) {
  return rows == 8 ? split_warps_of<8>(d_head, format) : split_warps_of<16>(d_head, format);
}

struct TreePlan {
  int gq, rows, grp, nrg, G, wfar;
  bool tc;
  size_t flags, ml, acc, total;  // offsets and size of the workspace
};

// share: of the keys that a sequence's drafted tokens may see (1: unknown)
TreePlan tree_plan(const focus_cache_params& p, bool force_tc = false, double share = 1.0) {
  TreePlan t;
  t.gq = p.H / p.H_kv;
  t.rows = p.T * t.gq;
  // Which kernel.  Up to 16 rows fill one warp's products.  With more, the one-warp kernel
  // reads the keys once per 16 rows, the tensor-core kernel once per 256, but it takes 12 us
  // more to set up and to merge.  Then 32 keys of a KV head cost it about 3.0 ns (5.5 with over 128 rows)
  // against 2.5 ns per 16 rows: With the merge, 64 rows per KV head over 2K bf16 keys take
  // 35 us against 26, over 16K 41 against 61, over 128K 126 against 334; 256 rows over 2K 36
  // against 43.  The lengths are not known here: the capacity stands for them.
  const double units = share * p.B * p.H_kv * ((p.cap + kTreeUnit - 1) / kTreeUnit);
  const int r16 = (t.rows + 15) / 16, r128 = (t.rows + 127) / 128;
  t.tc = force_tc || t.rows > 16 && 20e3 + units * (r128 == 1 ? 3.0 : 5.5 * ((r128 + 1) / 2)) < 8e3 + units * 2.5 * r16;
  t.grp = t.tc ? (t.rows > kTreeTcRows ? 2 * kTreeTcRows : kTreeTcRows) : t.rows > 8 ? 16 : 8;
  t.nrg = (t.rows + t.grp - 1) / t.grp;
  t.G = kTreeSms * (t.tc ? 1 : split_warps(p.d_head, p.format, t.grp));
  const int64_t lanes = (int64_t)p.H_kv * t.nrg;
  const int64_t most = lanes * p.B * (((int64_t)p.cap + kTreeUnit - 1) / kTreeUnit) * kTreeNear;
  t.G = (int)std::max<int64_t>(1, std::min<int64_t>(t.G, most / kTreeNear));
  // expected share of the far keys that some drafted token's mask meets (balance only)
  double miss = 1.0;
  for (int i = 0; i < p.top_k; ++i) miss *= std::max(0.0, (double)(p.K - p.top_k - i)) / (p.K - i);
  t.wfar = std::max(1, (int)std::lround(kTreeNear * (1.0 - pow(miss, p.T))));
  const size_t slots = (size_t)(t.G + lanes * p.B) * t.grp;
  t.flags = 256;
  t.ml = t.flags + align_up(sizeof(int32_t) * t.G, 256);
  t.acc = t.ml + align_up(sizeof(float2) * slots, 256);
  t.total = t.acc + align_up(sizeof(float) * slots * p.d_head, 256);
  return t;
}

// A kernel that may start when the one before it has (and waits for it itself where it needs it).
template <typename K, typename... A>
cudaError_t launch_beside(K* kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, int FMT, int NR, bool PRE>
cudaError_t launch_split(const TreeArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(tree_split<D, FMT, NR, PRE>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  });
  if (e != cudaSuccess) return e;
  constexpr size_t bytes = TreeLayout<D, FMT, NR>::BYTES;
  if (PRE) return launch_beside(tree_split<D, FMT, NR, PRE>, dim3((unsigned)a.G), 32, bytes, s, a);
  tree_split<D, FMT, NR, PRE><<<(unsigned)a.G, 32, bytes, s>>>(a);
  return cudaGetLastError();
}

// The merge of a's rows; o: as in Parts.
template <int D, int FMT, bool PRE>
cudaError_t launch_merge(const TreeArgs& a, const TreeArgs& o, cudaStream_t s) {
  // The merge, by its rows and by the partials of one, were all sequences alike.  Few rows with
  // many partials: many threads for a row (32 rows of 210: 10 us with 1024 threads, 33 with a
  // warp).  Many rows with few: 2048 of 19 take 8 us by warps, 12 by 128 threads, 41 by 512;
  // 512 of 38 take 13, 9.5 and 14; 256 of 38 take 15, 11 and 9.
  int64_t each = (int64_t)a.G / ((int64_t)a.H_kv * a.nrg * a.B);
  if (PRE) each += (int64_t)o.G / ((int64_t)o.H_kv * o.nrg * o.B);
  const int64_t rows = PRE ? (int64_t)a.tokens * a.H : (int64_t)a.T * a.H * a.B;
  auto by = [&](auto* kernel, int rows_each, int threads) {
    const int groups = PRE ? (a.tokens + a.T - 1) / a.T : a.B;
    return launch_beside(kernel, dim3((unsigned)((a.T * a.H + rows_each - 1) / rows_each), (unsigned)groups), threads, 0, s, a, o);
  };
  // Over a prefix, with two parts to be found: four rows to a warp from a block for each SM on.  The whole
  // call by one row and by four: 56832 rows 223 and 163 us, 34848 rows 146 and 88, 6992 rows 55 and 45, 5120
  // rows 289 and 278; but 3296 rows 140 and 145, 2048 rows 98 and 102.
  if constexpr (PRE) {
    if (each <= 32 && rows >= 32 * kTreeSms && a.gq % 4 == 0) return by(tree_combine_rows<D, FMT, 4, PRE>, 32, 256);
  }
  if (each <= 32 && rows >= 1536) return by(tree_combine_rows<D, FMT, 1, PRE>, 8, 256);
  if (each <= 64 && rows >= 512) return by(tree_combine<D, FMT, 128, PRE>, 1, 128);
  return each > 256 ? by(tree_combine<D, FMT, 1024, PRE>, 1, 1024)
         : each > 16 ? by(tree_combine<D, FMT, 512, PRE>, 1, 512)
                     : by(tree_combine<D, FMT, 128, PRE>, 1, 128);
}

template <int D, int FMT, bool PRE>
cudaError_t launch_parts(const TreeArgs& a, bool tc, cudaStream_t s) {
  return tc           ? launch_tree_tc(a, D, FMT, PRE, s)
         : a.grp == 8 ? launch_split<D, FMT, 8, PRE>(a, s)
                      : launch_split<D, FMT, 16, PRE>(a, s);
}

template <int D, int FMT>
cudaError_t launch_tree(const TreeArgs& a, bool tc, cudaStream_t s) {
  const cudaError_t e = launch_parts<D, FMT, false>(a, tc, s);
  return e != cudaSuccess ? e : launch_merge<D, FMT, false>(a, a, s);
}

}  // namespace

size_t tree_workspace_bytes(const focus_cache_params& p) { return tree_plan(p).total; }

namespace {

TreeArgs args_of(const focus_cache_params& p, const TreePlan& t, const bf16* q, const void* kc, const void* vc,
                 const float* ks, const float* vs, const uint32_t* mask, const int32_t* lens, const uint64_t* tree,
                 bf16* o, float* lse, char* ws, float scale) {
  TreeArgs a;
  a.q = q, a.kc = kc, a.vc = vc, a.ks = ks, a.vs = vs, a.mask = mask, a.lens = lens, a.tree = tree;
  a.part_ml = reinterpret_cast<float2*>(ws + t.ml);
  a.part_acc = reinterpret_cast<float*>(ws + t.acc);
  a.flags = t.tc ? reinterpret_cast<int32_t*>(ws + t.flags) : nullptr;
  a.o = o, a.lse = lse, a.status = reinterpret_cast<int32_t*>(ws);
  a.B = p.B, a.cap = p.cap, a.T = p.T, a.H = p.H, a.H_kv = p.H_kv, a.R = p.R, a.w = p.w;
  a.gq = t.gq, a.rows = t.rows, a.grp = t.grp, a.nrg = t.nrg;
  a.G = t.G, a.wfar = t.wfar, a.tma = 0;
  a.sl2 = scale * kLog2e;
  a.per = p.T;
  a.own_mask = nullptr, a.own_cap = a.plen = a.tokens = 0;
  a.order = nullptr, a.run_tokens = a.place = nullptr;
  return a;
}

}  // namespace

cudaError_t launch_decode_tree(const focus_cache_params& p, const bf16* q, const void* kc, const void* vc,
                               const float* ks, const float* vs, const uint32_t* mask,
                               const int32_t* lens, const uint64_t* tree, bf16* o, float* lse, char* ws,
                               float scale, cudaStream_t s) {
  const TreePlan t = tree_plan(p);
  const TreeArgs a = args_of(p, t, q, kc, vc, ks, vs, mask, lens, tree, o, lse, ws, scale);
  if (p.d_head == 64)
    return p.format == FOCUS_CACHE_BF16   ? launch_tree<64, FOCUS_CACHE_BF16>(a, t.tc, s)
           : p.format == FOCUS_CACHE_E4M3 ? launch_tree<64, FOCUS_CACHE_E4M3>(a, t.tc, s)
                                          : launch_tree<64, FOCUS_CACHE_INT8>(a, t.tc, s);
  return p.format == FOCUS_CACHE_BF16   ? launch_tree<128, FOCUS_CACHE_BF16>(a, t.tc, s)
         : p.format == FOCUS_CACHE_E4M3 ? launch_tree<128, FOCUS_CACHE_E4M3>(a, t.tc, s)
                                        : launch_tree<128, FOCUS_CACHE_INT8>(a, t.tc, s);
}

// ---------------------------------------------------------- a batch behind one prefix --
// Two parts and one merge.  The own keys go through decode_tree's kernels as they are (distances
// inside the own part do not know the prefix).  The prefix's keys go through the same kernels with
// the roles changed: up to 64 of the batch's tokens count as the drafted tokens of one sequence,
// each with its own window and groups, so that a K/V row is read once for all of them.  The
// prefix's kernel starts beside the own part's and takes the SMs as they become free; the merge
// takes the partial results of both.
//
// With one group a token, a run of tokens of one group sees a K-th of the far keys, and all of it.  Runs by
// group in place of the tokens' order then read (and multiply) the keys once in all, not once per run:
// 160 sequences behind 128K tokens, 4 groups, 508 -> 225 us.  One more kernel sorts them.
namespace {

constexpr int kSortThreads = 512;
constexpr int kSortRows = 128;         // rows of queries a KV head above which tokens are sorted,
constexpr int kSortRowsOfGroup = 16;   // that each group then has at least (on average),
constexpr int kSortKeysOfGroup = 2048; // and its far keys

// The tokens of the batch's row sorted by group, in runs of T places: a group's runs follow one another, and
// its tokens keep their order.  A token's group is the lowest bit of its mask (of routing head 0: there
// is one), no more than K of them: there are places for as many runs.  What a token sees goes by its
// whole mask, so other masks cost time alone.  One block; a pass counts, a pass places.
__global__ void __launch_bounds__(kSortThreads) sort_tokens(const __grid_constant__ TreeArgs a, int K, int4* order,
                                                             int32_t* run_tokens, int32_t* place) {
  constexpr int NW = kSortThreads / 32;
  __shared__ int count[33], first[33], warps[NW][33];
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  for (int i = tid; i < a.B * a.T; i += kSortThreads) order[i] = make_int4(-1, 0, 0, 0);
  for (int i = tid; i < a.B; i += kSortThreads) run_tokens[i] = 0;
  if (tid < 33) count[tid] = 0;
  __syncthreads();
  int4 entry;  // of the token looked at last
  int known = -1;
  auto group_of = [&](int x) {  // 32: no token
    const Drafted tok(a, x / a.T, x % a.T);  // (a.order is not set here: as they stand)
    known = x;
    if (!tok.word) return 32;
    const uint32_t m = tok.groups(a, 0);
    entry = make_int4(x, tok.near(a), (int)m, 0);
    return m ? min(__ffs(m), K) - 1 : 0;
  };
  int g = 32;
  for (int x0 = 0; x0 < a.tokens; x0 += kSortThreads)
    if (x0 + tid < a.tokens) atomicAdd(&count[g = group_of(x0 + tid)], 1);
  __syncthreads();
  if (tid == 0) {
    int run = 0;
    for (int g = 0; g < 32; ++g) {
      first[g] = run;
      run += (count[g] + a.T - 1) / a.T;
    }
    first[32] = run;
  }
  __syncthreads();
  if (tid < 32)
    for (int run = first[tid], n = count[tid]; n > 0; ++run, n -= a.T) run_tokens[run] = min(n, a.T);
  __syncthreads();
  if (tid < 33) count[tid] = 0;  // placed so far
  __syncthreads();
  for (int x0 = 0; x0 < a.tokens; x0 += kSortThreads) {
    for (int i = tid; i < NW * 33; i += kSortThreads) (&warps[0][0])[i] = 0;
    __syncthreads();
    const int x = x0 + tid;
    if (x != known) g = x < a.tokens ? group_of(x) : 32;
    const unsigned alike = __match_any_sync(0xffffffffu, g);
    const int before = __popc(alike & lanemask_lt());
    if (before == 0) warps[wp][g] = __popc(alike);
    __syncthreads();
    if (x < a.tokens) {
      int r = count[g] + before;
      for (int i = 0; i < wp; ++i) r += warps[i][g];
      const int at = g < 32 ? (first[g] + r / a.T) * a.T + r % a.T : -1;
      place[x] = at;
      if (at >= 0) order[at] = entry;
    }
    __syncthreads();
    if (tid < 33)
      for (int i = 0; i < NW; ++i) count[tid] += warps[i][tid];
    __syncthreads();
  }
}

struct SharedPlan {
  TreePlan own, pre;
  focus_cache_params run;  // the prefix as the kernels see it: runs of tokens as sequences
  bool sorted;
  size_t pre_at, order, run_tokens, place, total;
};

SharedPlan shared_plan(const focus_cache_params& p, int prefix_len) {
  SharedPlan s;
  s.own = tree_plan(p);
  s.run = p;
  const int64_t tokens = (int64_t)p.B * p.T;
  s.run.T = (int)std::min<int64_t>(tokens, FOCUS_MAX_DRAFT);
  s.run.B = (int)((tokens + s.run.T - 1) / s.run.T);
  s.run.cap = std::max(prefix_len, 1);
  // Sorted: one group a token, one routing head (heads with groups of their own would need runs of their own),
  // and fewer products for it.  Those are made for 128 rows at a time, used or not, and a run's rows come one
  // by one where the tokens are sorted, its listing reads the masks of all the prefix: so up to 128 rows of
  // all tokens are read at once as they stand, two groups save nothing, and many small ones only cost.
  // bf16, 32 query heads (8 KV heads unless said), not sorted / sorted, us of the whole call (160 tokens: with a
  // merge that took 10 longer on either side):
  //   tokens  groups | prefix 4096     8192       16384      65536
  //     32      4    |   37 / 44     41 / 53     57 / 59     98 / 110     128 rows
  //     64      2    |   47 / 52     54 / 60     69 / 75    136 / 151     two groups
  //     40      4    |   53 / 55     63 / 54     77 / 69    143 / 118
  //     64      4    |   47 / 46     53 / 49     70 / 58    136 / 108
  //     64      8    |   47 / 60     54 / 78     73 / 62    135 / 117
  //     64     32    |   48 / 71     54 / 106    69 / 132   138 / 222     8 rows a group
  //    160      4    |   68 / 74     84 / 82    119 / 93    302 / 169
  //    160     16    |   70 / 105    84 / 82    119 / 95    303 / 156
  //    160      4    |  108 / 99    147 / 117   223 / 145   682 / 329     32 KV heads
  // Runs have places for half as many tokens again as a group has on average.
  const int64_t rows = tokens * (p.H / p.H_kv);
  s.sorted = p.R == 1 && p.top_k == 1 && p.K > 2 && rows > kSortRows && rows >= (int64_t)kSortRowsOfGroup * p.K &&
             prefix_len >= kSortKeysOfGroup * p.K;
  if (s.sorted) {
    s.run.T = (int)std::min<int64_t>(s.run.T, std::max<int64_t>(4, (tokens * 3 / 2 + p.K - 1) / p.K));
    s.run.B = (int)((tokens + s.run.T - 1) / s.run.T) + p.K;
    s.pre = tree_plan(s.run, false, (double)std::max(p.K, s.run.B - p.K) / s.run.B / p.K);
    s.pre.wfar = std::max(1, (kTreeNear + p.K / 2) / p.K);
  } else {
    s.pre = tree_plan(s.run);
  }
  s.pre_at = align_up(s.own.total, 256);
  s.order = s.pre_at + align_up(s.pre.total, 256);
  s.run_tokens = s.order + (s.sorted ? align_up(sizeof(int4) * s.run.B * s.run.T, 256) : 0);
  s.place = s.run_tokens + (s.sorted ? align_up(sizeof(int32_t) * s.run.B, 256) : 0);
  s.total = s.place + (s.sorted ? align_up(sizeof(int32_t) * tokens, 256) : 0);
  return s;
}

template <int D, int FMT>
cudaError_t launch_shared(const TreeArgs& own, bool own_tc, const TreeArgs& pre, bool pre_tc, cudaStream_t s) {
  cudaError_t e = launch_parts<D, FMT, false>(own, own_tc, s);
  if (e == cudaSuccess) e = launch_parts<D, FMT, true>(pre, pre_tc, s);
  return e != cudaSuccess ? e : launch_merge<D, FMT, true>(pre, own, s);
}

}  // namespace

size_t shared_workspace_bytes(const focus_cache_params& p, int prefix_len) { return shared_plan(p, prefix_len).total; }

cudaError_t launch_decode_shared(const focus_cache_params& p, const bf16* q, int prefix_cap, int prefix_len, const void* pk,
                                 const void* pv, const float* pks, const float* pvs, const uint32_t* pmask, const void* kc,
                                 const void* vc, const float* ks, const float* vs, const uint32_t* mask, const int32_t* lens,
                                 const uint64_t* tree, bf16* o, float* lse, char* ws, float scale, cudaStream_t s) {
  const SharedPlan t = shared_plan(p, prefix_len);
  TreeArgs own = args_of(p, t.own, q, kc, vc, ks, vs, mask, lens, tree, o, lse, ws, scale);
  TreeArgs pre = args_of(t.run, t.pre, q, pk, pv, pks, pvs, pmask, lens, tree, o, lse, ws + t.pre_at, scale);
  pre.status = own.status;
  pre.cap = prefix_cap;
  pre.per = p.T;
  pre.own_mask = mask, pre.own_cap = p.cap, pre.plen = prefix_len, pre.tokens = p.B * p.T;
  if (t.sorted) {
    int4* order = reinterpret_cast<int4*>(ws + t.order);
    int32_t* run_tokens = reinterpret_cast<int32_t*>(ws + t.run_tokens);
    int32_t* place = reinterpret_cast<int32_t*>(ws + t.place);
    sort_tokens<<<1, kSortThreads, 0, s>>>(pre, p.K, order, run_tokens, place);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    pre.order = order, pre.run_tokens = run_tokens, pre.place = place;
  }
  constexpr int B = FOCUS_CACHE_BF16, E = FOCUS_CACHE_E4M3, I = FOCUS_CACHE_INT8;
  if (p.d_head == 64)
    return p.format == B   ? launch_shared<64, B>(own, t.own.tc, pre, t.pre.tc, s)
           : p.format == E ? launch_shared<64, E>(own, t.own.tc, pre, t.pre.tc, s)
                           : launch_shared<64, I>(own, t.own.tc, pre, t.pre.tc, s);
  return p.format == B   ? launch_shared<128, B>(own, t.own.tc, pre, t.pre.tc, s)
         : p.format == E ? launch_shared<128, E>(own, t.own.tc, pre, t.pre.tc, s)
                         : launch_shared<128, I>(own, t.own.tc, pre, t.pre.tc, s);
}

// Diagnostic launch of the tensor-core kernel on a small problem, one CTA: one loader warp keeps
// back its word that Q is there, the waits end after ~10 ms.  The MMA warp's wait runs out while the
// other roles stand at theirs, the loaders with all stages full: the CTA gives up, waits for its
// copies, frees its tensor memory and exits, and the merge makes every row NaN.
// o [T, 4, 128] bf16 and lse [4, T] are left at the returned offsets of ws.
size_t tree_selftest_bytes() { return 16u << 20; }
cudaError_t launch_tree_timeout_selftest(char* ws, int format, int T, size_t* o_at, size_t* lse_at, cudaStream_t s) {
  focus_cache_params p{};
  p.B = 1, p.cap = 2048, p.T = T, p.H = 4, p.H_kv = 1, p.d_head = 128;
  p.R = 1, p.K = 1, p.top_k = 1, p.w = 1 << 20, p.format = format;
  const TreePlan t = tree_plan(p, true);
  size_t at = t.total;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at += align_up(bytes, 256);
    return x;
  };
  const size_t kv = (size_t)p.cap * p.d_head * 2, rows = (size_t)T * p.H;
  const size_t q = take(rows * p.d_head * 2), k = take(kv), v = take(kv), ks = take(p.cap * 4), vs = take(p.cap * 4);
  const size_t mask = take(p.cap * 4), lens = take(4);
  *o_at = take(rows * p.d_head * 2), *lse_at = take(rows * 4);
  if (at > tree_selftest_bytes()) return cudaErrorInvalidValue;
  cudaError_t e = cudaMemsetAsync(ws, 0, at, s);
  if (e != cudaSuccess) return e;
  if ((e = cudaMemsetAsync(ws + lens + 1, 4, 1, s)) != cudaSuccess) return e;  // 1024 cached tokens
  const bool scales = format != FOCUS_CACHE_BF16;
  TreeArgs a = args_of(p, t, reinterpret_cast<bf16*>(ws + q), ws + k, ws + v, scales ? reinterpret_cast<float*>(ws + ks) : nullptr,
                       scales ? reinterpret_cast<float*>(ws + vs) : nullptr, reinterpret_cast<uint32_t*>(ws + mask),
                       reinterpret_cast<int32_t*>(ws + lens), nullptr, reinterpret_cast<bf16*>(ws + *o_at),
                       reinterpret_cast<float*>(ws + *lse_at), ws, 0.1f);
  a.G = 1;
  if ((e = launch_tree_tc_held(a, format, false, s)) != cudaSuccess) return e;
  return format == FOCUS_CACHE_BF16 ? launch_merge<128, FOCUS_CACHE_BF16, false>(a, a, s)
                                    : launch_merge<128, FOCUS_CACHE_INT8, false>(a, a, s);
}

// The same over a prefix of 1024 tokens, kSelftestSeqs sequences with 1024 of their own: the prefix's kernel
// or the own part's is the held one, the other works as always beside it; the merge reads both kernels' flags.
cudaError_t launch_shared_timeout_selftest(char* ws, int format, int T, bool hold_prefix, size_t* o_at, size_t* lse_at,
                                           cudaStream_t s) {
  focus_cache_params p{};
  p.B = kSelftestSeqs, p.cap = 2048, p.T = T, p.H = 4, p.H_kv = 1, p.d_head = 128;
  p.R = 1, p.K = 1, p.top_k = 1, p.w = 1 << 20, p.format = format;
  constexpr int kPrefix = 1024;
  focus_cache_params run = p;
  run.B = 1, run.T = p.B * T, run.cap = kPrefix;
  const TreePlan own_plan = tree_plan(p, true), plan = tree_plan(run, true);
  size_t at = align_up(own_plan.total, 256) + align_up(plan.total, 256);
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at += align_up(bytes, 256);
    return x;
  };
  const size_t kv = (size_t)p.cap * p.d_head * 2, rows = (size_t)p.B * T * p.H;
  const size_t q = take(rows * p.d_head * 2), k = take(p.B * kv), v = take(p.B * kv), ks = take(p.B * p.cap * 4), vs = take(p.B * p.cap * 4);
  const size_t mask = take(p.B * p.cap * 4), lens = take(p.B * 4);
  *o_at = take(rows * p.d_head * 2), *lse_at = take(rows * 4);
  if (run.T > FOCUS_MAX_DRAFT || at > tree_selftest_bytes()) return cudaErrorInvalidValue;
  cudaError_t e = cudaMemsetAsync(ws, 0, at, s);
  for (int b = 0; b < p.B && e == cudaSuccess; ++b) e = cudaMemsetAsync(ws + lens + 4 * b + 1, 4, 1, s);
  if (e != cudaSuccess) return e;
  auto args = [&](const focus_cache_params& x, const TreePlan& t, size_t from) {  // (the prefix: the first sequence's cache)
    const bool scales = format != FOCUS_CACHE_BF16;
    return args_of(x, t, reinterpret_cast<bf16*>(ws + q), ws + k, ws + v, scales ? reinterpret_cast<float*>(ws + ks) : nullptr,
                   scales ? reinterpret_cast<float*>(ws + vs) : nullptr, reinterpret_cast<uint32_t*>(ws + mask),
                   reinterpret_cast<int32_t*>(ws + lens), nullptr, reinterpret_cast<bf16*>(ws + *o_at),
                   reinterpret_cast<float*>(ws + *lse_at), ws + from, 0.1f);
  };
  TreeArgs own = args(p, own_plan, 0), pre = args(run, plan, align_up(own_plan.total, 256));
  pre.status = own.status, pre.per = T;
  pre.own_mask = own.mask, pre.own_cap = p.cap, pre.plen = kPrefix, pre.tokens = p.B * T;
  (hold_prefix ? pre : own).G = 1;
  e = hold_prefix ? launch_tree_tc(own, 128, format, false, s) : launch_tree_tc_held(own, format, false, s);
  if (e != cudaSuccess) return e;
  e = hold_prefix ? launch_tree_tc_held(pre, format, true, s) : launch_tree_tc(pre, 128, format, true, s);
  if (e != cudaSuccess) return e;
  return format == FOCUS_CACHE_BF16 ? launch_merge<128, FOCUS_CACHE_BF16, true>(pre, own, s)
                                    : launch_merge<128, FOCUS_CACHE_INT8, true>(pre, own, s);
}

}  // namespace focus
