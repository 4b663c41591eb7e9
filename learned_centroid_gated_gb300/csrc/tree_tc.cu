// Decode of drafted tokens over a cache, on the tensor cores: the kernel for more than 16
// rows (T tokens x H / H_kv query heads) per KV head.  The method, the slices and the last
// step (tree_combine) are those of tree.cu.
//
// Up to 128 rows share a K/V row that is read once: 4 d x 128 flops for 4 d bytes (bf16) is
// still below the tensor cores' balance, so the K/V stream has to stay the bound.  One CTA
// per SM takes a slice and works through its segments with
//   warps 8-11  list the keys that any row sees, and gather their K and V rows, 64 keys a
//               tile, with 16-byte asynchronous copies: bf16 rows straight into the
//               128-byte-swizzled operand tiles; 8-bit codes into a staging ring, whence
//               each thread turns the pieces that it copied itself into fp16 operands
//               (exact), so that no barrier stands between the copy and the conversion.
//   warp 12     issues the products: S = Q K^T (128 x 64, both operands in shared memory)
//               into one of four tensor-memory tiles, and O += P V with P read from tensor
//               memory.  It takes whichever is ready, the next S or the next P V.
//   warps 0-7   the softmax of a tile, a thread per row: warps 0-3 take even tiles, warps
//               4-7 odd ones, each with a maximum, a sum and an O of its own (two partial
//               results per segment), so that two tiles are in work at a time.
// The scales of 8-bit rows: K's multiplies the logits, V's multiplies P before it is rounded
// to fp16; the running reference of the exponentials is kept so that their product fits.
// Every wait is bounded; a wait that runs out raises FOCUS_ERR_TIMEOUT.
#include <math.h>

#include "tc_ptx.cuh"
#include "tree.cuh"
#include "warp_mma.cuh"

namespace focus {
namespace {

using namespace ptx;
using wmma16::cp_async16;
using wmma16::cp_async4;
using wmma16::cp_async_commit;
using wmma16::cp_async_wait;
using wmma16::lds128;
using wmma16::lanemask_lt;
using wmma16::pack_bf16;
using wmma16::pack_f16;

constexpr int kRows = 128;      // rows per CTA
constexpr int kTile = 64;       // keys per tile
constexpr int kScan = 512;      // raw keys per listing step (4 per loader lane)
constexpr int kList = 1024;     // entries of the list ring
constexpr int kMeta = 16;       // entries of the tile-metadata ring
constexpr int kSBuf = 4;        // tensor-memory tiles for S and P
constexpr int kThreads = 512;     // 16 warps; 13 work, the rest fill the last warpgroup
constexpr int kMmaWarp = 12, kLoadWarp = 8;

enum TileMode { kAll = 0, kMasks = 1, kEach = 2, kEnd = 3 };

struct alignas(16) TileMeta {  // an array of them is read in 16-byte pieces
  int pos[kTile];         // position of each key (a drafted key: its slot), -1 beyond the tile's keys
  uint32_t mask[kTile];
  float ks[kTile], vs[kTile];
  int mode, n;
  float vmax[2], vmin[2];  // V scales of each half: the largest, the least that is not 0
};

template <int D, int FMT>
struct Tc {
  static constexpr bool B16 = FMT == FOCUS_CACHE_BF16;
  static constexpr int BOXES = D / 64;
  static constexpr int STAGES = B16 ? (D == 128 ? 5 : 6) : 3;  // operand tiles
  static constexpr int RAW = B16 ? 0 : 4;                      // staging tiles of codes
  static constexpr int LAG = B16 ? (D == 128 ? 3 : 4) : 3;     // tiles whose copies are in flight
  static constexpr int QBOX = kRows * 128, KBOX = kTile * 128; // bytes of 64 columns
  static constexpr int KV = BOXES * KBOX;
  static constexpr int OFF_KV = BOXES * QBOX;
  static constexpr int OFF_RAW = OFF_KV + STAGES * 2 * KV;
  static constexpr int RAW_TILE = 2 * kTile * D;
  static constexpr int OFF_META = OFF_RAW + RAW * RAW_TILE;
  static constexpr int OFF_LIST = OFF_META + kMeta * (int)sizeof(TileMeta);
  static constexpr int OFF_DOWN = OFF_LIST + kList * 8;
  static constexpr int OFF_CNT = OFF_DOWN + 2 * kRows * 4;
  static constexpr int OFF_BAR = OFF_CNT + 2 * 4 * 4;
  static constexpr int BYTES = OFF_BAR + 8 * (2 * STAGES + 3 * kSBuf + 11) + 1024;
  // A metadata entry is written anew kMeta tiles later, when its tile has long been through
  // the products: a tile is issued once the one AHEAD before it is.
  static constexpr int AHEAD = B16 ? STAGES : RAW + STAGES;
  static_assert(AHEAD < kMeta, "a metadata entry outlives its tile");
  static_assert(LAG < STAGES || !B16, "copies in flight need stages of their own");
  static_assert(OFF_META % 16 == 0 && sizeof(TileMeta) % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
  static_assert(KV % 1024 == 0 && OFF_KV % 1024 == 0 && RAW_TILE % 16 == 0, "operand tiles start a swizzle period");
  static_assert(BYTES <= 232448, "shared memory of a CTA");
};

// Instruction descriptor, kind::f16 with fp16 operands (type code 0) and fp32 sums.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn_major) {
  return (1u << 4) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Registers: 512 threads launch with 128 each; the two softmax warpgroups take 152, the
// loaders and the last warpgroup keep 104 (2 x 152 + 2 x 104 = 4 x 128).
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 152;"); }
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 104;"); }

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ float4 lds_f4(const float* p) { return *reinterpret_cast<const float4*>(p); }

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1) tree_tc(const __grid_constant__ TreeArgs a) {
  using L = Tc<D, FMT>;
  constexpr bool B16 = L::B16;
  constexpr int S = L::STAGES, ES = B16 ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar = smem_u32(sm + L::OFF_BAR);
  const uint32_t b_full = bar, b_empty = bar + 8 * S;                     // + 8 * stage
  const uint32_t b_s = bar + 16 * S, b_p = b_s + 8 * kSBuf, b_pv = b_p + 8 * kSBuf;  // + 8 * S buffer
  const uint32_t b_q = b_pv + 8 * kSBuf, b_qfree = b_q + 8;               // Q tile there / read
  // O of a segment read: + 8 * (2 * warpgroup + (segment & 1)).  Two by turns, since a
  // warpgroup without a tile in the next segment may be done with that one too.
  const uint32_t b_epi = b_qfree + 8;
  const uint32_t b_drain = b_epi + 32, b_load = b_drain + 8;              // the loader warps' meetings
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(sm + L::OFF_BAR + 8 * (2 * S + 3 * kSBuf + 9));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::OFF_BAR + 8 * (2 * S + 3 * kSBuf + 10));
  TileMeta* meta = reinterpret_cast<TileMeta*>(sm + L::OFF_META);
  float* down = reinterpret_cast<float*>(sm + L::OFF_DOWN);  // [segment & 1][row]: 8-bit row units
  int* status = a.flags + blockIdx.x;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(b_full + 8 * i, 4);   // one arrival per loader warp
      mbar_init(b_empty + 8 * i, 1);
    }
    for (int i = 0; i < kSBuf; ++i) {
      mbar_init(b_s + 8 * i, 1);
      mbar_init(b_p + 8 * i, 4);      // one arrival per softmax warp
      mbar_init(b_pv + 8 * i, 1);
    }
    mbar_init(b_q, 4);
    mbar_init(b_qfree, 1);
    for (int i = 0; i < 4; ++i) mbar_init(b_epi + 8 * i, 4);
    mbar_init(b_drain, 1);
    mbar_init(b_load, 4);
    *abort_flag = 0;
    *status = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint32_t b, int phase) { return mbar_wait(b, phase & 1, abort_flag, status); };
  auto o_read = [&](int seg) {  // both warpgroups have read the O of segment seg
    const uint32_t b = b_epi + 8 * (seg & 1);
    return wait(b, seg >> 1) && wait(b + 16, seg >> 1);
  };

  if (warp >= kLoadWarp && warp < kMmaWarp) {
    // ------------------------------------------------------------------ loaders --
    fewer_registers();
    const int lt = tid - 32 * kLoadWarp, lw = lt >> 5;
    int* lidx = reinterpret_cast<int*>(sm + L::OFF_LIST);
    uint32_t* lmsk = reinterpret_cast<uint32_t*>(lidx + kList);
    int* cnt = reinterpret_cast<int*>(sm + L::OFF_CNT);  // [parity][warp]
    int t = 0;     // tiles, end marks among them
    int seg = 0, scans = 0, meets = 0;
    bool ok = true;
    // The loader warps meet: a barrier with a bounded wait.
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(b_load);
      ok = __all_sync(0xffffffffu, wait(b_load, meets++));
    };
    for_segments(a, blockIdx.x, lane, [&](int64_t, int kvh, int rg, int b, int len, int js, int je) {
      if (!ok) return;
      const int rho = kvh / (a.H_kv / a.R);
      const uint32_t* M = a.mask + ((int64_t)b * a.R + rho) * a.cap;
      const int rows = min(kRows, a.rows - rg * kRows);
      // ---- Q tile (the last segment's products have read the old one)
      if (seg > 0 && !(ok = __all_sync(0xffffffffu, wait(b_qfree, seg - 1)))) return;
      {
        const int x = rg * kRows + min(lt, rows - 1), tt = x / a.gq, h = kvh * a.gq + x % a.gq;
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (((int64_t)b * a.T + tt) * a.H + h) * D);
        const bool on = lt < rows;
        float up = 1.0f, dn = 1.0f;
        if constexpr (!B16) {
          float mx = 0.0f;
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = __ldg(src + c);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
          }
          row_unit(mx, up, dn);
        }
        down[(seg & 1) * kRows + lt] = dn;
        const uint32_t q0 = smem_u32(sm) + lt * 128;
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = on ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
          if constexpr (!B16) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_f16(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
          }
          sts128(q0 + (c / 8) * L::QBOX + (((c & 7) ^ (lt & 7)) << 4), w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_q);
      }
      // ---- what the rows see: four rows per lane
      uint32_t many = 0u, wlo = 0u, whi = 0u;
      int nearest = INT_MAX, farthest = INT_MIN;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int x = 32 * i + lane;
        if (x < rows) {
          const int tt = (rg * kRows + x) / a.gq;
          const uint64_t word = tree_word(a, b, tt);
          if (word) {
            many |= __ldg(M + len + tt);
            wlo |= (uint32_t)word;
            whi |= (uint32_t)(word >> 32);
            const int near = len + __popcll(word) - a.w;
            nearest = min(nearest, near);
            farthest = max(farthest, near);
          }
        }
      }
      many = __reduce_or_sync(0xffffffffu, many);
      const uint64_t any_word = (uint64_t)__reduce_or_sync(0xffffffffu, whi) << 32 | __reduce_or_sync(0xffffffffu, wlo);
      nearest = __reduce_min_sync(0xffffffffu, nearest);
      farthest = __reduce_max_sync(0xffffffffu, farthest);

      const int64_t kvrow = (int64_t)a.H_kv * D * ES;  // bytes per slot
      const int64_t base = ((int64_t)b * a.cap * a.H_kv + kvh) * D * ES;
      const char* kb = reinterpret_cast<const char*>(a.kc) + base;
      const char* vb = reinterpret_cast<const char*>(a.vc) + base;
      const float* ksc = B16 ? nullptr : a.ks + ((int64_t)b * a.H_kv + kvh) * a.cap;
      const float* vsc = B16 ? nullptr : a.vs + ((int64_t)b * a.H_kv + kvh) * a.cap;

      int jb = js, head = 0, tail = 0;
      constexpr int MW = kScan / 128;
      uint32_t mw[MW];
      auto load_masks = [&]() {
#pragma unroll
        for (int i = 0; i < MW; ++i) {
          const int j = jb + 32 * (MW * lw + i) + lane;
          mw[i] = j < je ? __ldg(M + j) : 0u;
        }
      };
      // Appends the keys of the next kScan that some row sees to the list, in order.
      auto scan = [&]() {
        unsigned bal[MW];
        int mine = 0;
#pragma unroll
        for (int i = 0; i < MW; ++i) {
          const int j = jb + 32 * (MW * lw + i) + lane;
          bool see = j < je;
          if (see) see = j < len ? j >= nearest || (mw[i] & many) != 0u : (any_word >> (j - len) & 1ull) != 0ull;
          bal[i] = __ballot_sync(0xffffffffu, see);
          mine += __popc(bal[i]);
        }
        int* c = cnt + 4 * (scans++ & 1);
        if (lane == 0) c[lw] = mine;
        meet();  // counts there
        if (!ok) return;
        int at = head, all = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          at += i < lw ? c[i] : 0;
          all += c[i];
        }
#pragma unroll
        for (int i = 0; i < MW; ++i) {
          if (bal[i] >> lane & 1u) {
            const int x = (at + __popc(bal[i] & lanemask_lt())) & (kList - 1);
            lidx[x] = jb + 32 * (MW * lw + i) + lane;
            lmsk[x] = mw[i];
          }
          at += __popc(bal[i]);
        }
        head += all;
        jb += kScan;
        load_masks();
        meet();  // entries there
      };
      // Starts the copies of the next tile (n keys of the list).
      auto issue = [&](int n) {
        TileMeta& me = meta[t & (kMeta - 1)];
        const int first = lidx[tail & (kList - 1)], last = lidx[(tail + n - 1) & (kList - 1)];
        if (lt < kTile) {
          const int x = (tail + lt) & (kList - 1);
          me.pos[lt] = lt < n ? lidx[x] : -1;
          me.mask[lt] = lt < n ? lmsk[x] : 0u;
        }
        if (lt == 0) {
          me.n = n;
          me.mode = n == kTile && last < len && first >= farthest ? kAll : last < min(nearest, len) ? kMasks : kEach;
        }
        constexpr int CH = D * ES / 16, RPI = 128 / CH;  // pieces per row, rows per pass
        const int ch = lt % CH;
        const uint32_t st = smem_u32(sm + (B16 ? L::OFF_KV + (t % S) * 2 * L::KV
                                               : L::OFF_RAW + (t % (B16 ? 1 : L::RAW)) * L::RAW_TILE));
#pragma unroll
        for (int r = lt / CH; r < kTile; r += RPI) {
          uint32_t dst = st;
          if constexpr (B16) dst += (ch / 8) * L::KBOX + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
          else dst += r * D + 16 * ch;
          constexpr int VOFF = B16 ? L::KV : kTile * D;
          if (r < n) {
            const int64_t off = (int64_t)lidx[(tail + r) & (kList - 1)] * kvrow + 16 * ch;
            cp_async16(dst, kb + off);
            cp_async16(dst + VOFF, vb + off);
          } else {  // no key: finite values under zero weights
            sts128(dst, 0u, 0u, 0u, 0u);
            sts128(dst + VOFF, 0u, 0u, 0u, 0u);
          }
        }
        if constexpr (!B16) {
          const int r = lt & (kTile - 1);
          float* dst = (lt < kTile ? me.ks : me.vs) + r;
          if (r < n) cp_async4(smem_u32(dst), (lt < kTile ? ksc : vsc) + lidx[(tail + r) & (kList - 1)]);
          else *dst = 0.0f;
        }
        tail += n;
      };
      // Hands tile x over, its copies (this thread's) having landed.
      auto finish = [&](int x, bool end) {
        if constexpr (!B16) {
          if (x >= S && !(ok = __all_sync(0xffffffffu, wait(b_empty + 8 * (x % S), x / S - 1)))) return;
          if (!end) {
            const uint32_t raw = smem_u32(sm + L::OFF_RAW + (x % (B16 ? 1 : L::RAW)) * L::RAW_TILE);
            const uint32_t st = smem_u32(sm + L::OFF_KV + (x % S) * 2 * L::KV);
            constexpr int CH = D / 16, RPI = 128 / CH;
            const int ch = lt % CH;
#pragma unroll 2
            for (int r = lt / CH; r < kTile; r += RPI) {
#pragma unroll
              for (int v = 0; v < 2; ++v) {
                const uint4 y = lds128(raw + v * kTile * D + r * D + 16 * ch);
                const uint32_t w[4] = {y.x, y.y, y.z, y.w};
                uint32_t h[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  h[2 * i] = codes_f16<FMT>(w[i]);
                  h[2 * i + 1] = codes_f16<FMT>(w[i] >> 16);
                }
                // 16 columns are two 16-byte chunks of the operand tile's row
                const uint32_t dst = st + v * L::KV + (ch / 4) * L::KBOX + r * 128;
                const int c = 2 * (ch & 3);
                sts128(dst + ((c ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
                sts128(dst + (((c + 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
              }
            }
            TileMeta& me = meta[x & (kMeta - 1)];
            if (lt >= kTile) {  // (an infinite scale reads as NaN: the row's maximum stays finite)
              const float y = me.vs[lt - kTile];
              const bool fine = fabsf(y) < INFINITY;
              if (!fine) me.vs[lt - kTile] = __uint_as_float(0x7fc00000u);
              const uint32_t u = fine ? __float_as_uint(fabsf(y)) : 0u;
              const uint32_t top = __reduce_max_sync(0xffffffffu, u);
              const uint32_t low = __reduce_min_sync(0xffffffffu, u ? u : 0x7f800000u);
              if (lane == 0) {
                me.vmax[lw - 2] = __uint_as_float(top);
                me.vmin[lw - 2] = __uint_as_float(low);
              }
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_full + 8 * (x % S));
      };
      load_masks();
      int landed = t;  // tiles handed over so far
      for (;;) {
        while (ok && head - tail < kTile && jb < je) scan();
        if (!ok) break;
        const int n = min(kTile, head - tail);
        if (n == 0) break;
        if constexpr (B16) {
          if (t >= S && !(ok = __all_sync(0xffffffffu, wait(b_empty + 8 * (t % S), t / S - 1)))) break;
        }
        issue(n);
        cp_async_commit();
        ++t;
        if (t - landed > L::LAG) {
          cp_async_wait<L::LAG>();
          finish(landed++, false);
          if (!ok) break;
        }
      }
      cp_async_wait<0>();
      while (ok && landed < t) finish(landed++, false);
      for (int e = 0; ok && e < 2; ++e) {  // an end mark for each softmax warpgroup
        if constexpr (B16) {
          if (t >= S && !(ok = __all_sync(0xffffffffu, wait(b_empty + 8 * (t % S), t / S - 1)))) break;
        }
        if (lt == 0) meta[t & (kMeta - 1)].mode = kEnd;
        finish(t++, true);
      }
      ++seg;
      if (ok) meet();  // the list starts anew
    });
    cp_async_wait<0>();
  } else if (warp >= kMmaWarp) {
    fewer_registers();
    // ---------------------------------------------------------------- MMA issue --
    if (warp == kMmaWarp) {
    constexpr uint32_t IS = B16 ? idesc_bf16(kRows, kTile, 0) : idesc_f16(kRows, kTile, 0);
    constexpr uint32_t IPV = B16 ? idesc_bf16(kRows, D, 1) : idesc_f16(kRows, D, 1);
    int t = 0, c = 0, seg = 0;  // tiles with end marks, products, segments
    bool ok = true;
    for_segments(a, blockIdx.x, lane, [&](int64_t, int, int, int, int, int, int) {
      if (lane == 0 && ok) {
        ok = wait(b_q, seg);
        tc_fence_after();
        int ts = t, cs = c, cp = c;
        bool ended = false, fresh[2] = {true, true};
        long long t0 = clock64();
        while (ok && !(ended && cp == cs)) {
          bool some = false;
          if (!ended && cs < cp + kSBuf && mbar_try_wait(b_full + 8 * (ts % S), (ts / S) & 1)) {
            some = true;
            if (meta[ts & (kMeta - 1)].mode == kEnd) {
              ended = true;
            } else {
              tc_fence_after();
              const uint64_t da = sw128_desc(smem_u32(sm), 16, 1024);
              const uint64_t db = sw128_desc(smem_u32(sm + L::OFF_KV + (ts % S) * 2 * L::KV), 16, 1024);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                umma_ss(tmem + (cs % kSBuf) * kTile, da + (((kk / 4) * L::QBOX + (kk % 4) * 32) >> 4),
                        db + (((kk / 4) * L::KBOX + (kk % 4) * 32) >> 4), IS, kk > 0);
              umma_commit(b_s + 8 * (cs % kSBuf));
              ++cs;
              ++ts;
            }
          }
          if (cp < cs && mbar_try_wait(b_p + 8 * (cp % kSBuf), (cp / kSBuf) & 1)) {
            some = true;
            tc_fence_after();
            const int wg = cp & 1, st = (t + cp - c) % S;
            const uint64_t dv = sw128_desc(smem_u32(sm + L::OFF_KV + st * 2 * L::KV + L::KV), L::KBOX, 1024);
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              umma_ts(tmem + kSBuf * kTile + wg * 128, tmem + (cp % kSBuf) * kTile + 8 * kk, dv + ((kk * 2048) >> 4),
                      IPV, !fresh[wg] || kk > 0 ? 1u : 0u);
            fresh[wg] = false;
            umma_commit(b_pv + 8 * (cp % kSBuf));
            umma_commit(b_empty + 8 * st);
            ++cp;
          }
          if (some) {
            t0 = clock64();
          } else if (*abort_flag) {
            ok = false;
          } else if (clock64() - t0 > kTimeoutCycles) {
            *abort_flag = 1;
            raise_status(status, FOCUS_ERR_TIMEOUT);
            ok = false;
          }
        }
        umma_commit(b_qfree);
        // The end marks' stages go back once both warpgroups have read them (and O): the
        // loaders cannot lap a warpgroup that still waits for its mark.
        if (ok && (ok = wait(b_full + 8 * ((ts + 1) % S), (ts + 1) / S) && o_read(seg))) {
          mbar_arrive(b_empty + 8 * (ts % S));
          mbar_arrive(b_empty + 8 * ((ts + 1) % S));
          t = ts + 2;
          c = cs;
        }
        ++seg;
      }
      __syncwarp();
    });
    if (lane == 0) {
      umma_commit(b_drain);  // every product issued above completes before TMEM is released
      mbar_drain(b_drain, 0);
    }
    __syncwarp();
    }
  } else {
    // ------------------------------------------------------------------ softmax --
    more_registers();
    const int wg = warp >> 2, r = (warp & 3) * 32 + lane;  // warpgroup; row = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + lane_off + kSBuf * kTile + wg * 128;
    // sums of exponentials up to which a tile keeps the reference: far inside fp32 (bf16 P
    // has its exponents); in fp16 P times the V scale stays below 2^15
    constexpr float kSumCap = B16 ? 1.8446744e19f : 32768.0f;
    constexpr float kTop = B16 ? 0.0f : 7.0f;  // log2 of the largest weight when m is set
    int t = wg, c = wg, seg = 0;
    bool ok = true;
    for_segments(a, blockIdx.x, lane, [&](int64_t partial, int kvh, int rg, int b, int len, int, int) {
      if (!ok) return;
      const int rho = kvh / (a.H_kv / a.R);
      const uint32_t* M = a.mask + ((int64_t)b * a.R + rho) * a.cap;
      const int x = rg * kRows + r, tt = min(x, a.rows - 1) / a.gq;
      const bool on = x < a.rows;
      const uint64_t word = on ? tree_word(a, b, tt) : 0ull;
      const uint32_t mrow = word ? __ldg(M + len + tt) : 0u;
      const int near = word ? len + __popcll(word) - a.w : INT_MAX;
      float m = -INFINITY, l = 0.0f, fac = a.sl2;
      const int c0 = c;
      for (;; t += 2, c += 2) {
        const TileMeta& me = meta[t & (kMeta - 1)];
        ok = __all_sync(0xffffffffu, wait(b_full + 8 * (t % S), t / S));
        if (!ok) return;
        const int mode = me.mode;
        if (mode == kEnd) break;
        if (c == c0) fac = a.sl2 * (B16 ? 1.0f : down[(seg & 1) * kRows + r]);
        ok = __all_sync(0xffffffffu, wait(b_s + 8 * (c % kSBuf), c / kSBuf));
        if (!ok) return;
        tc_fence_after();
        const uint32_t tS = tmem + lane_off + (c % kSBuf) * kTile;
        uint32_t x0[32], x1[32];
        tmem_ld32(tS, x0);
        tmem_ld32(tS + 32, x1);
        tmem_ld_wait(x0);
        tie32(x1);
        float vtop = 1.0f;
        bool wide = false;
        if constexpr (!B16) {
          vtop = fmaxf(fmaxf(me.vmax[0], me.vmax[1]), kTinyScale);
          wide = vtop > 16.0f * fminf(me.vmin[0], me.vmin[1]);
          auto by_k = [&](uint32_t(&xx)[32], int cb) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 s = lds_f4(me.ks + cb + i);
              float y0, y1;
              fmul2(y0, y1, __uint_as_float(xx[i]), __uint_as_float(xx[i + 1]), s.x, s.y);
              xx[i] = __float_as_uint(y0), xx[i + 1] = __float_as_uint(y1);
              fmul2(y0, y1, __uint_as_float(xx[i + 2]), __uint_as_float(xx[i + 3]), s.z, s.w);
              xx[i + 2] = __float_as_uint(y0), xx[i + 3] = __float_as_uint(y1);
            }
          };
          by_k(x0, 0);
          by_k(x1, 32);
        }
        // ---- keys that this row does not see
        constexpr uint32_t kNeg = 0xff800000u;
        if (mode == kMasks) {
          auto drop = [&](uint32_t(&xx)[32], int cb) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const uint4 k4 = *reinterpret_cast<const uint4*>(me.mask + cb + i);
              xx[i] = (k4.x & mrow) ? xx[i] : kNeg;
              xx[i + 1] = (k4.y & mrow) ? xx[i + 1] : kNeg;
              xx[i + 2] = (k4.z & mrow) ? xx[i + 2] : kNeg;
              xx[i + 3] = (k4.w & mrow) ? xx[i + 3] : kNeg;
            }
          };
          drop(x0, 0);
          drop(x1, 32);
        } else if (mode == kEach) {
          uint64_t see = 0ull;
          const int n = me.n;
          for (int i = 0; i < n; ++i) {
            int p = me.pos[i];
            bool s = true;
            if (p >= len) {
              s = (word >> (p - len) & 1ull) != 0ull;
              p = len + __popcll(tree_word(a, b, p - len)) - 1;
            }
            if (s && (p >= near || (me.mask[i] & mrow) != 0u)) see |= 1ull << i;
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (!((uint32_t)see >> i & 1u)) x0[i] = kNeg;
            if (!((uint32_t)(see >> 32) >> i & 1u)) x1[i] = kNeg;
          }
        }
        // ---- exponentials against the row's reference m, which moves only when a tile's
        // sum passes the cap or while the row has seen no key.  8-bit formats: m is the
        // reference of P times V's scale, which is what fp16 has to hold; a tile whose scales
        // are far apart (an outlier that this row may not even see) is measured key by key.
        float f = 1.0f;        // what O has to be multiplied by
        const bool seen = m != -INFINITY;  // without a key so far O is zero
        auto refer = [&](float mx) {
          if (mx > m) {
            if (seen) f = ex2(m - mx);
            l *= f;
            m = mx;
          }
        };
        auto take_max = [&]() {
          float mm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; ++i)
            mm[i & 3] = max3(mm[i & 3], __uint_as_float(x0[i]), __uint_as_float(x1[i]));
          float mx = fmaxf(fmaxf(mm[0], mm[1]), fmaxf(mm[2], mm[3])) * fac;
          if constexpr (!B16) mx += log2f(vtop) - kTop;
          refer(mx);
        };
        if (wide) {
          if constexpr (!B16) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              mx = fmaxf(mx, __uint_as_float(x0[i]) * fac + __log2f(fmaxf(fabsf(me.vs[i]), kTinyScale)));
              mx = fmaxf(mx, __uint_as_float(x1[i]) * fac + __log2f(fmaxf(fabsf(me.vs[32 + i]), kTinyScale)));
            }
            if (mx - kTop > m + 7.0f || m == -INFINITY) refer(mx - kTop);
          }
        } else if (__any_sync(0xffffffffu, m == -INFINITY)) {
          take_max();
        }
        float la, lb;
        auto emit_all = [&]() {
          const float nms = m == -INFINITY ? 0.0f : -m;
          la = 0.0f;
          lb = 0.0f;
          auto emit = [&](uint32_t(&xx)[32], int k) {  // P over its S, which is in registers
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              float y[4];
              ffma2(y[0], y[1], __uint_as_float(xx[2 * i]), __uint_as_float(xx[2 * i + 1]), fac, fac, nms, nms);
              ffma2(y[2], y[3], __uint_as_float(xx[2 * i + 2]), __uint_as_float(xx[2 * i + 3]), fac, fac, nms, nms);
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = ex2(y[e]);
              fadd2(la, lb, la, lb, y[0], y[1]);
              fadd2(la, lb, la, lb, y[2], y[3]);
              if constexpr (B16) {
                pk[i] = pack_bf16(y[0], y[1]);
                pk[i + 1] = pack_bf16(y[2], y[3]);
              } else {
                const float4 s = lds_f4(me.vs + 32 * k + 2 * i);
                fmul2(y[0], y[1], y[0], y[1], s.x, s.y);
                fmul2(y[2], y[3], y[2], y[3], s.z, s.w);
                pk[i] = pack_f16(y[0], y[1]);
                pk[i + 1] = pack_f16(y[2], y[3]);
              }
            }
            tmem_st16(tS + 16 * k, pk);
          };
          emit(x0, 0);
          emit(x1, 1);
        };
        emit_all();
        if (!wide && __any_sync(0xffffffffu, !((la + lb) * vtop <= kSumCap))) {
          take_max();
          emit_all();
        }
        l += la + lb;
        if (__any_sync(0xffffffffu, f != 1.0f) && c > c0) {
          // O of this warpgroup's earlier tiles follows the reference
          ok = __all_sync(0xffffffffu, wait(b_pv + 8 * ((c - 2) % kSBuf), (c - 2) / kSBuf));
          if (!ok) return;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            uint32_t y[32];
            tmem_ld32(tO + 32 * k, y);
            tmem_ld_wait(y);
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
            tmem_st32(tO + 32 * k, y);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_p + 8 * (c % kSBuf));
      }
      t += 2;  // the end mark
      // ---- this segment's partial
      const bool some = c > c0;
      if (some) {
        ok = __all_sync(0xffffffffu, wait(b_pv + 8 * ((c - 2) % kSBuf), (c - 2) / kSBuf));
        if (!ok) return;
        tc_fence_after();
      }
      const int64_t slot = (partial * kTreeTcParts + wg) * kRows + r;
      if (on) a.part_ml[slot] = make_float2(m, some ? l : 0.0f);
      if (some) {
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint32_t y[32];
          tmem_ld32(tO + 32 * k, y);
          tmem_ld_wait(y);
          if (on) {
            float4* dst = reinterpret_cast<float4*>(a.part_acc + slot * D + 32 * k);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i] = make_float4(__uint_as_float(y[4 * i]), __uint_as_float(y[4 * i + 1]),
                                   __uint_as_float(y[4 * i + 2]), __uint_as_float(y[4 * i + 3]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_epi + 8 * (2 * wg + (seg & 1)));
      ++seg;
    });
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int FMT>
cudaError_t launch(const TreeArgs& a, cudaStream_t s) {
  using L = Tc<D, FMT>;
  cudaError_t e = cudaFuncSetAttribute(tree_tc<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  if (e != cudaSuccess) return e;
  tree_tc<D, FMT><<<(unsigned)a.G, kThreads, L::BYTES, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_tc(const TreeArgs& a, int d_head, int format, cudaStream_t s) {
  if (d_head == 64)
    return format == FOCUS_CACHE_BF16   ? launch<64, FOCUS_CACHE_BF16>(a, s)
           : format == FOCUS_CACHE_E4M3 ? launch<64, FOCUS_CACHE_E4M3>(a, s)
                                        : launch<64, FOCUS_CACHE_INT8>(a, s);
  return format == FOCUS_CACHE_BF16   ? launch<128, FOCUS_CACHE_BF16>(a, s)
         : format == FOCUS_CACHE_E4M3 ? launch<128, FOCUS_CACHE_E4M3>(a, s)
                                      : launch<128, FOCUS_CACHE_INT8>(a, s);
}

}  // namespace focus
