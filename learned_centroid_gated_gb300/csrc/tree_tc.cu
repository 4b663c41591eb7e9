// Decode of drafted tokens over a cache, on the tensor cores: the kernel for many rows
// (T tokens x H / H_kv query heads) per KV head.  The method, the slices and the last step
// (tree_combine) are those of tree.cu.
//
// Up to 256 rows share a K/V row that is read once: at most 4 d x 256 flops for 4 d bytes
// (bf16), about the balance of the tensor cores and the memory, so the K/V stream has to
// stay the bound.  One CTA per SM takes a slice and works through its segments with
//   loader warps   list the keys that any row sees and bring their K and V rows, 64 keys a
//               tile: 64 consecutive keys by TMA, others row by row with 16-byte asynchronous
//               copies.  bf16 rows go straight into the 128-byte-swizzled operand tiles;
//               8-bit codes into a staging ring, whence the loaders turn them into fp16
//               operands (exact).
//   warp 12     issues the products: S = Q K^T (both operands in shared memory) into tensor
//               memory, and O += P V with P read from tensor memory.  It takes whichever is
//               ready.  An MMA costs its issuer about 75 cycles however narrow it is, so
//               where both row halves use a tile (256 rows, bf16) S is made for two tiles at
//               once (N = 128) and the products follow a fixed order: 1.46 -> 1.20 ms for 64
//               tokens behind a million.
//   warps 13-15 (readers) take the tiles in turn and work out which key each drafted token
//               sees, as one 64-bit word per token, and bring the scales of 8-bit rows.
//   softmax warps   a thread per row.  More than 128 rows (NT = 2): two warpgroups, each with
//               128 rows of every tile, and four loader warps.  Up to 128 (NT = 1): one
//               warpgroup, and eight loader warps, since the codes' conversion, not the
//               softmax, is the longer chain (64 rows over 128K int8 keys: 158 us with two
//               softmax warpgroups by turns and four loader warps, 141 so; bf16 114 and 117).
// Measured: 64 drafts of 32 / 8 heads over a million bf16 keys 1.20 ms, 3.4 TB/s and 0.88
// PFLOP/s (the products alone would take 0.53 ms at the peak rate); 16 drafts over 128K keys
// 117 us bf16 (4.6 TB/s), 144 us int8 (1.9 TB/s); 64 drafts over 128K 179 and 236 us.  What bounds
// it: with 256 rows nothing is full (of 2700 cycles a tile the issuer is busy 1200, the tensor
// pipe a third, DRAM 0.38): a half's S, softmax and P V follow one another, since P lies over S and
// its next S waits for its last P V.  With fewer rows and int8 the softmax warps' instructions
// (1800 cycles of a tile's 2500, its bytes 740); with bf16 the bytes' 1400 and the softmax's 1200
// of 2000, partly in turn.  8-bit codes cost the conversion and the scales on top, so that they
// save less time than bytes.
// The roles' loops share the instruction cache: the code is kept short rather than unrolled
// (the conversion's loop unrolled by 4: 157 -> 172 us, by 2 the least).
// The scales of 8-bit rows: K's multiplies the logits; V's multiplies P, and the reference of
// the exponentials is that of the product, which is what fp16 has to hold.  P times V's scale is
// an fp32 product and is rounded once (as fp16 times an fp16 scale, three roundings, it took the
// same time: 64 rows over 128K int8 keys 147 us both).
// Every wait is bounded; a wait that runs out raises FOCUS_ERR_TIMEOUT.
#include <cuda.h>
#include <math.h>

#include <mutex>

#include "tc_ptx.cuh"
#include "tree.cuh"
#include "warp_mma.cuh"

namespace focus {
namespace {

using namespace ptx;
using wmma16::cp_async16;
using wmma16::cp_async_commit;
using wmma16::cp_async_wait;
using wmma16::lds128;
using wmma16::lanemask_lt;
using wmma16::pack_bf16;
using wmma16::pack_f16;

constexpr int kRows = 128;      // rows of a product (the MMA's M)
constexpr int kTile = 64;       // keys per tile
constexpr int kSBuf = 4;        // tensor-memory tiles for S and P
constexpr int kMeta = 8;        // entries of the tile-metadata ring
constexpr int kOrders = 16;     // entries of the ring of orders
constexpr int kScan = 256;      // raw keys per listing step
constexpr int kList = 1024;     // entries of the list ring
constexpr int kThreads = 512;
constexpr int kMmaWarp = 12, kReadWarp = 13, kReaders = 3;

// What the softmax has to know of a tile, from a reader.
template <bool B16>
struct alignas(16) TileMeta;
template <>
struct alignas(16) TileMeta<true> {
  uint64_t see[FOCUS_MAX_DRAFT];  // [token of the row group]: its keys of the tile
  int end;                        // no tile: the segment's end
};
template <>
struct alignas(16) TileMeta<false> {
  uint64_t see[FOCUS_MAX_DRAFT];
  int end;
  int wide;                       // V scales differ by more than 2^4, or are above 2^kFarGap
  float lv, unit;                 // V scales are below 2^lv; 2^-lv
  float ks[kTile], vs[kTile];     // scales
};

// What the readers and the MMA warp have to know of a tile, from a loader: its place in the
// list and its keys, or kEnd where it is none but the segment's end.
struct Order {
  int tail, n;
};
constexpr int kEnd = -1;
constexpr float kFarGap = 60.0f;  // log2

template <int D, int FMT, int NT>
struct Tc {
  static constexpr bool B16 = FMT == FOCUS_CACHE_BF16;
  static constexpr bool PAIR = B16 && NT == 2;  // S of two tiles at once
  static constexpr int LOAD_WARP = 4 * NT, LW = kMmaWarp - LOAD_WARP;  // first loader warp; loader warps
  using Meta = TileMeta<B16>;
  static constexpr int BOXES = D / 64;
  // operand tiles; staging tiles of codes; tiles whose copies (row by row) are in flight
  static constexpr int STAGES = B16 ? (D == 128 ? (NT == 1 ? 5 : 4) : 6) : 3;
  static constexpr int RAW = B16 ? 0 : (D == 128 && NT == 2 ? 3 : 4);
  static constexpr int LAG = B16 ? STAGES - 2 : RAW - 1;
  static constexpr int SLOTS = B16 ? STAGES : RAW;                      // tiles that copies go to
  static constexpr int QBOX = kRows * 128, KBOX = kTile * 128;          // bytes of 64 columns
  static constexpr int QT = BOXES * QBOX, KV = BOXES * KBOX;
  static constexpr int RAW_TILE = 2 * kTile * D;
  static constexpr int OFF_KV = NT * QT;
  static constexpr int OFF_RAW = OFF_KV + STAGES * 2 * KV;
  static constexpr int OFF_META = OFF_RAW + RAW * RAW_TILE;
  static constexpr int OFF_ORDER = OFF_META + kMeta * (int)sizeof(Meta);
  static constexpr int OFF_LIST = OFF_ORDER + kOrders * (int)sizeof(Order);
  static constexpr int OFF_DOWN = OFF_LIST + kList * 4;
  static constexpr int OFF_SETS = OFF_DOWN + (B16 ? 0 : 2 * NT * kRows * 4);
  static constexpr int OFF_CNT = OFF_SETS + 3 * 32 * 8;
  static constexpr int OFF_BAR = OFF_CNT + 2 * 8 * 4;
  static constexpr int BARS = 2 * STAGES + 3 * kSBuf + 8 + 2 * SLOTS + kMeta + kOrders;
  static constexpr int OFF_SLICE = OFF_BAR + 8 * (BARS + 2);
  static constexpr int BYTES = OFF_SLICE + (int)sizeof(Slice) + 1024;
  // K rows of a stage: box stride and, of a pair, its tiles one behind the other
  static constexpr int KSTEP = PAIR ? 2 * KBOX : KBOX;
  __host__ __device__ static constexpr int k_at(int stage) {
    return OFF_KV + (PAIR ? (stage >> 1) * 4 * KV + (stage & 1) * KBOX : stage * 2 * KV);
  }
  __host__ __device__ static constexpr int v_at(int stage) {
    return OFF_KV + (PAIR ? (stage >> 1) * 4 * KV + 2 * KV + (stage & 1) * KV : stage * 2 * KV + KV);
  }
  // An entry of the metadata ring is written anew kMeta tiles later, when its tile has long
  // been through the products: a tile is issued once the one AHEAD before it is.  So the
  // readers are never kMeta tiles behind either, which is what the list holds on to (with
  // less than a tile left over and a listing step ahead), and the orders twice over.
  static constexpr int AHEAD = B16 ? STAGES : RAW + STAGES;
  static_assert(AHEAD < kMeta && kMeta * kTile + kTile + kScan <= kList && kOrders >= 2 * kMeta, "rings");
  static_assert(!PAIR || STAGES % 2 == 0, "pairs of stages");
  static_assert(OFF_META % 16 == 0 && sizeof(Meta) % 16 == 0 && OFF_CNT % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
  static_assert(KV % 1024 == 0 && OFF_KV % 1024 == 0 && RAW_TILE % 128 == 0, "operand tiles start a swizzle period");
  static_assert(BYTES <= 232448, "shared memory of a CTA");
};

// Instruction descriptor, kind::f16 with fp16 operands (type code 0) and fp32 sums.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn_major) {
  return (1u << 4) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Registers: 512 threads launch with 128 each; the loaders and the last warpgroup keep 104, the
// softmax takes what that leaves: 152 in each of two warpgroups, or 200 in one
// (2 x 152 + 2 x 104 = 200 + 3 x 104 = 4 x 128).
template <int NT>
__device__ __forceinline__ void more_registers() {
  if constexpr (NT == 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
  else asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
}
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 104;"); }

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// HOLD: the self-test's form, in which a loader warp keeps back its word that Q is there and the
// waits end after about 10 ms.  (A limit read at run time cost the others 1%.)
template <int D, int FMT, int NT, bool HOLD>
__global__ void __launch_bounds__(kThreads, 1)
tree_tc(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap map_k,
        const __grid_constant__ CUtensorMap map_v) {
  using L = Tc<D, FMT, NT>;
  using Meta = typename L::Meta;
  constexpr bool B16 = L::B16;
  constexpr int S = L::STAGES, ES = B16 ? 2 : 1;
  constexpr int LW = L::LW;
  constexpr long long kLimit = HOLD ? 20000000LL : kTimeoutCycles;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (stays a shared-memory pointer to the compiler)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar = smem_u32(sm + L::OFF_BAR);
  const uint32_t b_full = bar, b_empty = bar + 8 * S;                     // + 8 * stage
  const uint32_t b_s = bar + 16 * S, b_p = b_s + 8 * kSBuf, b_pv = b_p + 8 * kSBuf;  // + 8 * S buffer
  const uint32_t b_q = b_pv + 8 * kSBuf, b_qfree = b_q + 8;               // Q tile there / read
  // O of a segment read: + 8 * (2 * warpgroup + (segment & 1)).  Two by turns, since a
  // warpgroup without a tile in the next segment may be done with that one too.
  const uint32_t b_epi = b_qfree + 8;
  const uint32_t b_drain = b_epi + 32, b_load = b_drain + 8;              // the loader warps' meetings
  const uint32_t b_tma = b_load + 8, b_raw = b_tma + 8 * L::SLOTS;        // + 8 * slot: TMA there / codes read
  const uint32_t b_meta = b_raw + 8 * L::SLOTS, b_order = b_meta + 8 * kMeta;  // + 8 * entry: written
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(sm + L::OFF_BAR + 8 * L::BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::OFF_BAR + 8 * (L::BARS + 1));
  Meta* meta = reinterpret_cast<Meta*>(sm + L::OFF_META);
  Order* orders = reinterpret_cast<Order*>(sm + L::OFF_ORDER);
  int* lidx = reinterpret_cast<int*>(sm + L::OFF_LIST);
  float* down = reinterpret_cast<float*>(sm + L::OFF_DOWN);  // [segment & 1][row]: 8-bit row units
  int* status = a.flags + blockIdx.x;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  volatile Slice& slice = *reinterpret_cast<volatile Slice*>(sm + L::OFF_SLICE);
  if (warp == 0) {
    const Slice mine = slice_of(a, blockIdx.x, lane);
    if (lane == 0) {
      slice.W = mine.W, slice.lo = mine.lo, slice.hi = mine.hi;
      slice.ln = mine.ln;
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < S; ++i) {
      mbar_init(b_full + 8 * i, LW);  // one arrival per loader warp
      mbar_init(b_empty + 8 * i, 1);
    }
    for (int i = 0; i < kSBuf; ++i) {
      mbar_init(b_s + 8 * i, 1);
      mbar_init(b_p + 8 * i, 4);      // one arrival per softmax warp
      mbar_init(b_pv + 8 * i, 1);
    }
    mbar_init(b_q, LW);
    mbar_init(b_qfree, 1);
    for (int i = 0; i < 4; ++i) mbar_init(b_epi + 8 * i, 4);
    mbar_init(b_drain, 1);
    mbar_init(b_load, LW);
    for (int i = 0; i < L::SLOTS; ++i) {
      mbar_init(b_tma + 8 * i, 1);
      mbar_init(b_raw + 8 * i, LW);
    }
    for (int i = 0; i < kMeta; ++i) mbar_init(b_meta + 8 * i, 1);
    for (int i = 0; i < kOrders; ++i) mbar_init(b_order + 8 * i, 1);
    *abort_flag = 0;
    *status = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint32_t b, int phase) { return mbar_wait(b, phase & 1, abort_flag, status, kLimit); };
  auto wait_all = [&](uint32_t b, int phase) { return __all_sync(0xffffffffu, wait(b, phase)) != 0; };
  auto o_read = [&](int seg) {  // the softmax warps have read the O of segment seg
    const uint32_t b = b_epi + 8 * (seg & 1);
    return wait(b, seg >> 1) && (NT == 1 || wait(b + 16, seg >> 1));
  };

  if (warp >= L::LOAD_WARP && warp < kMmaWarp) {
    // ------------------------------------------------------------------ loaders --
    fewer_registers();
    const int lt = tid - 32 * L::LOAD_WARP, lw = lt >> 5;
    int* cnt = reinterpret_cast<int*>(sm + L::OFF_CNT);  // [parity][warp]
    int t = 0;     // tiles, an end mark per segment among them
    int seg = 0, scans = 0, meets = 0;
    // by slot: the tile in it comes by TMA; TMA copies so far (their parity; whether any)
    uint32_t by_tma = 0u, tma_odd = 0u, tma_any = 0u;
    bool ok = true;
    // The loader warps meet: a barrier with a bounded wait.
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(b_load);
      ok = wait_all(b_load, meets++);
    };
    for_segments(a, slice, blockIdx.x, lane, [&](int64_t, int kvh, int rg, int b, int len, int js, int je) {
      if (!ok) return;
      const int rho = kvh / (a.H_kv / a.R);
      const uint32_t* M = a.mask + ((int64_t)b * a.R + rho) * a.cap;
      const int row0 = rg * NT * kRows, rows = min(NT * kRows, a.rows - row0);
      const int tok0 = row0 / a.gq, ntok = (row0 + rows - 1) / a.gq - tok0 + 1;
      // ---- Q tiles (the last segment's products have read the old ones)
      if (seg > 0 && !(ok = wait_all(b_qfree, seg - 1))) return;
#pragma unroll 1
      for (int rt = 0; rt < NT; ++rt) {
        constexpr int HALVES = LW / 4, CQ = D / 8 / HALVES;  // threads per row, 16-byte chunks of each
        const int qr = lt % kRows, y = rt * kRows + qr, from = HALVES == 1 ? 0 : lt / kRows * CQ;
        const bool on = y < rows;
        const int x = row0 + (on ? y : 0), tt = x / a.gq, h = kvh * a.gq + x % a.gq;
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (((int64_t)b * a.T + tt) * a.H + h) * D);
        float up = 1.0f;
        if constexpr (!B16) {
          float mx = 0.0f, dn;
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = __ldg(src + c);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
          }
          row_unit(mx, up, dn);
          if (from == 0) down[((seg & 1) * NT + rt) * kRows + qr] = dn;
        }
        const uint32_t q0 = smem_u32(sm) + rt * L::QT + qr * 128;
#pragma unroll 4
        for (int i = 0; i < CQ; ++i) {
          const int c = from + i;
          const uint4 v = on ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
          if constexpr (!B16) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pack_f16(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xffff0000u) * up);
          }
          sts128(q0 + (c / 8) * L::QBOX + (((c & 7) ^ (qr & 7)) << 4), w[0], w[1], w[2], w[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && !(HOLD && lw == 0)) mbar_arrive(b_q);
      // ---- what the tokens see, taken together
      uint32_t many = 0u, wlo = 0u, whi = 0u;
      int nearest = INT_MAX;
      for (int i = lane; i < ntok; i += 32) {
        const uint64_t word = tree_word(a, b, tok0 + i);
        if (word) {
          many |= __ldg(M + len + tok0 + i);
          wlo |= (uint32_t)word;
          whi |= (uint32_t)(word >> 32);
          nearest = min(nearest, len + __popcll(word) - a.w);
        }
      }
      many = __reduce_or_sync(0xffffffffu, many);
      const uint64_t any_word = (uint64_t)__reduce_or_sync(0xffffffffu, whi) << 32 | __reduce_or_sync(0xffffffffu, wlo);
      nearest = __reduce_min_sync(0xffffffffu, nearest);

      const int64_t kvrow = (int64_t)a.H_kv * D * ES;  // bytes per slot
      const int64_t base = ((int64_t)b * a.cap * a.H_kv + kvh) * D * ES;
      const char* kb = reinterpret_cast<const char*>(a.kc) + base;
      const char* vb = reinterpret_cast<const char*>(a.vc) + base;

      int jb = js, head = 0, tail = 0;
      constexpr int MW = kScan / (32 * LW);
      uint32_t mw[MW];
      auto load_masks = [&]() {
#pragma unroll
        for (int i = 0; i < MW; ++i) {
          const int j = jb + 32 * (MW * lw + i) + lane;
          mw[i] = j < je ? __ldg(M + j) : 0u;
        }
      };
      // Appends the keys of the next SCAN that some row sees to the list, in order.  bf16: where
      // three quarters of them are seen all are listed, since 64 keys in a row come by TMA,
      // which costs less than leaving a quarter out (128K keys of which 0.66, 0.74 and 0.88 are
      // seen: 113, 130 and 129 us without the rest, 116, 116 and 116 with it).  Codes are half
      // the bytes, and each key has a conversion: the rest stays out (117, 140 and 141 us
      // against 142, 141 and 141).
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
        int* c = cnt + 8 * (scans++ & 1);
        if (lane == 0) c[lw] = mine;
        meet();  // counts there
        if (!ok) return;
        int all = 0, at = head;
#pragma unroll
        for (int i = 0; i < LW; ++i) {
          const int n = c[i];
          all += n;
          at += i < lw ? n : 0;
        }
        if (B16 && jb + kScan <= min(len, je) && 4 * all >= 3 * kScan) {
          all = kScan;
          at = head + 32 * MW * lw;
#pragma unroll
          for (int i = 0; i < MW; ++i) bal[i] = ~0u;
        }
#pragma unroll
        for (int i = 0; i < MW; ++i) {
          if (bal[i] >> lane & 1u) {
            const int x = (at + __popc(bal[i] & lanemask_lt())) & (kList - 1);
            lidx[x] = jb + 32 * (MW * lw + i) + lane;
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
        const int sl = t % L::SLOTS;
        const int first = lidx[tail & (kList - 1)], last = lidx[(tail + n - 1) & (kList - 1)];
        const bool run = a.tma && n == kTile && last - first == kTile - 1;
        const uint32_t kst = smem_u32(sm + (B16 ? L::k_at(sl) : L::OFF_RAW + sl * L::RAW_TILE));
        const uint32_t vst = smem_u32(sm + (B16 ? L::v_at(sl) : L::OFF_RAW + sl * L::RAW_TILE + kTile * D));
        by_tma = (by_tma & ~(1u << sl)) | (uint32_t)run << sl;
        if (lt == 0) {
          orders[t & (kOrders - 1)] = Order{tail, n};
          mbar_arrive(b_order + 8 * (t & (kOrders - 1)));
        }
        if (run) {
          if (lt == 0) {
            if (!B16 && t >= L::SLOTS && !wait(b_raw + 8 * sl, t / L::SLOTS - 1)) ok = false;
            if (ok) {
              // bf16: on the stage's own barrier, as this warp's arrival; codes: on the slot's
              const uint32_t bt = B16 ? b_full + 8 * sl : b_tma + 8 * sl;
              mbar_expect_tx(bt, 2 * kTile * D * ES);
              const int z = b * a.cap + first;
              if constexpr (B16) {
#pragma unroll
                for (int bx = 0; bx < L::BOXES; ++bx) {
                  tma_load_3d(kst + bx * L::KSTEP, &map_k, 64 * bx, kvh, z, bt);
                  tma_load_3d(vst + bx * L::KBOX, &map_v, 64 * bx, kvh, z, bt);
                }
              } else {
                tma_load_3d(kst, &map_k, 0, kvh, z, bt);
                tma_load_3d(vst, &map_v, 0, kvh, z, bt);
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
          if (!ok) return;
          tma_odd ^= 1u << sl;
          tma_any |= 1u << sl;
          if (B16 && lane == 0 && lw > 0) mbar_arrive(b_full + 8 * sl);
        } else {
          constexpr int CH = D * ES / 16, RPI = 32 * LW / CH;  // pieces per row, rows per pass
          const int ch = lt % CH;
#pragma unroll 4
          for (int r = lt / CH; r < kTile; r += RPI) {
            const int in = B16 ? r * 128 + (((ch & 7) ^ (r & 7)) << 4) : r * D + 16 * ch;
            const uint32_t kd = kst + in + (B16 ? (ch / 8) * L::KSTEP : 0), vd = vst + in + (B16 ? (ch / 8) * L::KBOX : 0);
            if (r < n) {
              const int64_t off = (int64_t)lidx[(tail + r) & (kList - 1)] * kvrow + 16 * ch;
              cp_async16(kd, kb + off);
              cp_async16(vd, vb + off);
            } else {  // no key: finite values under zero weights
              sts128(kd, 0u, 0u, 0u, 0u);
              sts128(vd, 0u, 0u, 0u, 0u);
            }
          }
        }
        tail += n;
      };
      // Hands tile x over, its copies (the TMA's, or this thread's own) having landed.
      auto finish = [&](int x, bool end) {
        const int sl = x % L::SLOTS;
        const bool run = !end && (by_tma >> sl & 1u);
        if (B16 && run) return;
        if (run && !(ok = wait_all(b_tma + 8 * sl, (tma_odd >> sl & 1u) ^ 1u))) return;
        if constexpr (!B16) {
          if (x >= S && !(ok = wait_all(b_empty + 8 * (x % S), x / S - 1))) return;
          if (!end) {
            const uint32_t raw = smem_u32(sm + L::OFF_RAW + sl * L::RAW_TILE);
            constexpr int CH = D / 16, RPI = 32 * LW / CH;
            // (16 columns are two 16-byte chunks of the operand tile's row; lanes of the second
            // box store theirs in the other order, so that eight lanes meet all banks)
            const int ch = lt % CH, c = 2 * (ch & 3), second = (ch / 4) & 1;
#pragma unroll 2
            for (int r = lt / CH; r < kTile; r += RPI) {
              const uint4 y0 = lds128(raw + r * D + 16 * ch), y1 = lds128(raw + kTile * D + r * D + 16 * ch);
#pragma unroll
              for (int v = 0; v < 2; ++v) {
                const uint4 y = v ? y1 : y0;
                const uint32_t w[4] = {second ? y.z : y.x, second ? y.w : y.y, second ? y.x : y.z, second ? y.y : y.w};
                uint32_t h[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) codes_f16x2<FMT>(w[i], h[2 * i], h[2 * i + 1]);
                const uint32_t dst = smem_u32(sm + (v ? L::v_at(x % S) : L::k_at(x % S))) + (ch / 4) * L::KBOX + r * 128;
                sts128(dst + (((c + second) ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
                sts128(dst + (((c + 1 - second) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
              }
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(b_full + 8 * (x % S));
          if constexpr (!B16) mbar_arrive(b_raw + 8 * sl);
        }
      };
      load_masks();
      int landed = t;  // tiles handed over so far
      while (ok) {
        while (ok && head - tail < kTile && jb < je) scan();
        const int n = min(kTile, head - tail);
        if (!ok || n == 0) break;
        if constexpr (B16) {
          if (t >= S && !(ok = wait_all(b_empty + 8 * (t % S), t / S - 1))) break;
        }
        issue(n);
        cp_async_commit();
        if (!ok) break;
        ++t;
        if (t - landed > L::LAG) {
          cp_async_wait<L::LAG>();
          finish(landed++, false);
        }
      }
      cp_async_wait<0>();
      while (ok && landed < t) finish(landed++, false);
      if constexpr (B16) {
        if (ok && t >= S) ok = wait_all(b_empty + 8 * (t % S), t / S - 1);
      }
      if (ok) {
        if (lt == 0) {
          orders[t & (kOrders - 1)] = Order{0, kEnd};
          mbar_arrive(b_order + 8 * (t & (kOrders - 1)));
        }
        finish(t++, true);
      }
      ++seg;
      if (ok) meet();  // the list starts anew
    });
    cp_async_wait<0>();
    // No CTA exits with a copy in flight, whoever gives up and when: the last TMA of each slot lands
    // first (codes' copies have been waited for, unless this warp gave up).
    if (lt == 0 && (B16 || *abort_flag))
      for (int i = 0; i < L::SLOTS; ++i) {
        if (!(tma_any >> i & 1u)) continue;
        if constexpr (B16) mbar_drain(b_full + 8 * i, (uint32_t)((t - 1 - i) / S & 1));
        else mbar_drain(b_tma + 8 * i, (tma_odd >> i & 1u) ^ 1u);
      }
    __syncwarp();
  } else if (warp >= kMmaWarp) {
    fewer_registers();
    if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- MMA issue --
      constexpr uint32_t IS = B16 ? idesc_bf16(kRows, L::PAIR ? 2 * kTile : kTile, 0) : idesc_f16(kRows, kTile, 0);
      constexpr uint32_t IPV = B16 ? idesc_bf16(kRows, D, 1) : idesc_f16(kRows, D, 1);
      int t = 0, c = 0, seg = 0;  // tiles with end marks, products, segments
      uint32_t p_par = 0u;        // pairs: by P tile, parity of its next P
      bool ok = true;
      auto s_product = [&](uint32_t dst, int rt, int stage) {
        const uint64_t da = sw128_desc(smem_u32(sm + rt * L::QT), 16, 1024);
        const uint64_t db = sw128_desc(smem_u32(sm + L::k_at(stage)), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss(dst, da + (((kk / 4) * L::QBOX + (kk % 4) * 32) >> 4), db + (((kk / 4) * L::KSTEP + (kk % 4) * 32) >> 4), IS,
                  kk > 0);
      };
      auto pv_product = [&](int wg, int buf, int stage, bool add) {
        const uint64_t dv = sw128_desc(smem_u32(sm + L::v_at(stage)), L::KBOX, 1024);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          umma_ts(tmem + kSBuf * kTile + wg * 128, tmem + buf * kTile + 8 * kk, dv + ((kk * 2048) >> 4), IPV,
                  add || kk > 0 ? 1u : 0u);
      };
      for_segments(a, slice, blockIdx.x, lane, [&](int64_t, int, int, int, int, int, int) {
        if (lane == 0 && ok) {
          ok = wait(b_q, seg);
          tc_fence_after();
          bool ended = false;
          uint32_t fresh = 0u;  // by warpgroup: O has a product of this segment
          long long t0 = clock64();
          bool some = false;
          auto idle = [&]() {  // bounds the wait of a round without work
            if (some) {
              t0 = clock64();
            } else if (*abort_flag) {
              ok = false;
            } else if (clock64() - t0 > kLimit) {
              *abort_flag = 1;
              raise_status(status, FOCUS_ERR_TIMEOUT);
              ok = false;
            }
            some = false;
          };
          // Tile x, or the end mark in its place, is there.
          auto arrived = [&](int x) {
            if (!mbar_test_wait(b_full + 8 * (x % S), (x / S) & 1)) return false;
            ended = orders[x & (kOrders - 1)].n == kEnd;
            return true;
          };
          int ts = t;  // tiles looked at; at the end, the end mark
          if constexpr (L::PAIR) {
            // The S of a unit, the tiles of a pair of stages, is made at once for a row half rt
            // when both tiles (or the end) are there and the half's last P V are issued; what
            // a segment's odd start or end leaves out of it is not read.  The two halves
            // alternate: while one's softmax works the tensor core has the other's products.
            bool ready = false;  // the next unit's tiles are there
            int nb = t;          // its first tile
            auto look = [&](bool block) {
              const int up = (nb | 1) + 1;
              while (!ended && ts < up) {
                if (block) {
                  if (!(ok = wait(b_full + 8 * (ts % S), ts / S))) break;
                  ended = orders[ts & (kOrders - 1)].n == kEnd;
                } else if (!arrived(ts)) {
                  return;
                }
                if (!ended) ++ts;
              }
              ready = ok && nb < ts;
            };
            auto make_s = [&](int rt) {
              tc_fence_after();
              s_product(tmem + rt * 2 * kTile, rt, (nb & ~1) % S);
              umma_commit(b_s + 8 * rt);
            };
            if (ok) look(true);
            if (ready) {
              make_s(0);
              make_s(1);
            }
            while (ready) {
              const int cb = nb, ce = min((nb | 1) + 1, ts);  // the unit whose S are made
              bool made[2] = {false, false};
              nb = ce;
              ready = false;
#pragma unroll
              for (int rt = 0; rt < 2; ++rt) {
                for (int x = cb; ok && x < ce; ++x) {
                  const int buf = 2 * rt + (x & 1);
                  if (!(ok = wait(b_p + 8 * buf, p_par >> buf))) break;
                  p_par ^= 1u << buf;
                  tc_fence_after();
                  pv_product(rt, buf, x % S, fresh >> rt & 1u);
                  fresh |= 1u << rt;
                  umma_commit(b_pv + 8 * buf);
                  if (rt == 1) umma_commit(b_empty + 8 * (x % S));
                }
                if (!ready) look(false);
                if (ready) {
                  make_s(rt);
                  made[rt] = true;
                }
              }
              if (!ready) look(true);
              if (ready) {
                if (!made[0]) make_s(0);
                if (!made[1]) make_s(1);
              }
            }
          } else {
            int cs = c, cp = c;
            int have = -1;  // the tile whose rows are there
            while (ok && !(ended && cp == cs)) {
              const bool begun = NT == 2 && ((cs - c) & 1);  // this tile's second product
              if (!ended && cs < cp + kSBuf && have != ts && arrived(ts)) {
                some = true;
                have = ts;
              }
              if (!ended && cs < cp + kSBuf && have == ts) {
                some = true;
                tc_fence_after();
                s_product(tmem + (cs % kSBuf) * kTile, begun, ts % S);
                umma_commit(b_s + 8 * (cs % kSBuf));
                ++cs;
                if (NT == 1 || begun) ++ts;
              }
              if (cp < cs && mbar_test_wait(b_p + 8 * (cp % kSBuf), (cp / kSBuf) & 1)) {
                some = true;
                tc_fence_after();
                const int wg = NT == 1 ? 0 : cp & 1, st = (t + (cp - c) / NT) % S;
                pv_product(wg, cp % kSBuf, st, fresh >> wg & 1u);
                fresh |= 1u << wg;
                umma_commit(b_pv + 8 * (cp % kSBuf));
                if (NT == 1 || ((cp - c) & 1)) umma_commit(b_empty + 8 * st);
                ++cp;
              }
              idle();
            }
            c = cs;
          }
          umma_commit(b_qfree);
          // The end mark's stage goes back once the softmax warps have read it (and O): the
          // loaders cannot lap a warpgroup that still waits for the mark.
          if (ok && (ok = wait(b_full + 8 * (ts % S), ts / S) && o_read(seg))) {
            mbar_arrive(b_empty + 8 * (ts % S));
            t = ts + 1;
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
    } else {
      // ------------------------------------------------------------------ readers --
      const int me_no = warp - kReadWarp;
      uint64_t* sets = reinterpret_cast<uint64_t*>(sm + L::OFF_SETS) + 32 * me_no;  // [group]: keys of a tile
      int t = 0;  // tiles, end marks among them
      bool ok = true;
      for_segments(a, slice, blockIdx.x, lane, [&](int64_t, int kvh, int rg, int b, int len, int, int) {
        if (!ok) return;
        const int rho = kvh / (a.H_kv / a.R);
        const uint32_t* M = a.mask + ((int64_t)b * a.R + rho) * a.cap;
        const int row0 = rg * NT * kRows, rows = min(NT * kRows, a.rows - row0);
        const int tok0 = row0 / a.gq, ntok = (row0 + rows - 1) / a.gq - tok0 + 1;
        // this lane's two tokens: ancestors, groups, first position inside the window
        uint64_t word[2];
        uint32_t grp[2];
        int near[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = 32 * e + lane;
          word[e] = i < ntok ? tree_word(a, b, tok0 + i) : 0ull;
          grp[e] = word[e] ? __ldg(M + len + tok0 + i) : 0u;
          near[e] = word[e] ? len + __popcll(word[e]) - a.w : INT_MAX;
        }
        const uint32_t many = __reduce_or_sync(0xffffffffu, grp[0] | grp[1]);
        const int nearest = __reduce_min_sync(0xffffffffu, min(near[0], near[1]));
        const int farthest =
            __reduce_max_sync(0xffffffffu, max(word[0] ? near[0] : INT_MIN, word[1] ? near[1] : INT_MIN));
        const float* ksc = B16 ? nullptr : a.ks + ((int64_t)b * a.H_kv + kvh) * a.cap;
        const float* vsc = B16 ? nullptr : a.vs + ((int64_t)b * a.H_kv + kvh) * a.cap;
        for (bool ended = false; !ended; ++t) {
          if (!(ok = wait_all(b_order + 8 * (t & (kOrders - 1)), t / kOrders))) return;
          const Order o = orders[t & (kOrders - 1)];
          const bool mine = t % kReaders == me_no;
          Meta& me = meta[t & (kMeta - 1)];
          if (o.n == kEnd) {
            ended = true;
            if (mine && lane == 0) me.end = 1;
          } else if (mine) {
            const int n = o.n;
            const int first = lidx[o.tail & (kList - 1)], last = lidx[(o.tail + n - 1) & (kList - 1)];
            int j[2];
            uint32_t mk[2], valid[2];
            float ks[2], vs[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = 32 * e + lane;
              j[e] = r < n ? lidx[(o.tail + r) & (kList - 1)] : 0;
              mk[e] = r < n ? __ldg(M + j[e]) : 0u;
              valid[e] = n >= 32 * e + 32 ? ~0u : n > 32 * e ? (1u << (n - 32 * e)) - 1u : 0u;
              if constexpr (!B16) {
                ks[e] = r < n ? __ldg(ksc + j[e]) : 0.0f;
                vs[e] = r < n ? __ldg(vsc + j[e]) : 0.0f;
              }
            }
            if (last < min(nearest, len)) {
              // before every window and the drafted tokens: for each group some token has, the
              // tile's keys that have it; a token sees the union of its groups' keys
              for (uint32_t g = many; g; g &= g - 1) {
                const int at = __ffs(g) - 1;
                const unsigned s0 = __ballot_sync(0xffffffffu, mk[0] >> at & 1u), s1 = __ballot_sync(0xffffffffu, mk[1] >> at & 1u);
                if (lane == 0) sets[at] = (uint64_t)s1 << 32 | s0;
              }
              __syncwarp();
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint64_t w = 0ull;
                for (uint32_t g = grp[e]; g; g &= g - 1) w |= sets[__ffs(g) - 1];
                if (32 * e + lane < ntok) me.see[32 * e + lane] = w;
              }
              __syncwarp();
            } else if (first >= farthest && last < len) {  // inside every window
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (32 * e + lane < ntok) me.see[32 * e + lane] = word[e] ? (uint64_t)valid[1] << 32 | valid[0] : 0ull;
            } else {
              uint64_t bit[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                bit[e] = valid[e] >> lane & 1u ? ~0ull : 0ull;
                if (bit[e] && j[e] >= len) {  // a drafted key: its token's bit, its position
                  bit[e] = 1ull << (j[e] - len);
                  j[e] = len + __popcll(tree_word(a, b, j[e] - len)) - 1;
                }
              }
              for (int i = 0; i < ntok; ++i) {
                const uint64_t w = __shfl_sync(0xffffffffu, i < 32 ? word[0] : word[1], i & 31);
                const uint32_t g = __shfl_sync(0xffffffffu, i < 32 ? grp[0] : grp[1], i & 31);
                const int from = __shfl_sync(0xffffffffu, i < 32 ? near[0] : near[1], i & 31);
                const unsigned s0 = __ballot_sync(0xffffffffu, (w & bit[0]) != 0ull && (j[0] >= from || (mk[0] & g) != 0u));
                const unsigned s1 = __ballot_sync(0xffffffffu, (w & bit[1]) != 0ull && (j[1] >= from || (mk[1] & g) != 0u));
                if (lane == 0) me.see[i] = (uint64_t)s1 << 32 | s0;
              }
            }
            if constexpr (!B16) {  // scales (an infinite one of V reads as NaN)
              uint32_t top = 0u, low = 0x7f800000u;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t u = __float_as_uint(fabsf(vs[e]));
                if (u >= 0x7f800000u) {
                  vs[e] = __uint_as_float(0x7fc00000u);
                } else {
                  top = max(top, u);
                  if (u) low = min(low, u);
                }
              }
              top = __reduce_max_sync(0xffffffffu, top);
              low = __reduce_min_sync(0xffffffffu, low);
              const int ex = max((int)(top >> 23) - 126, -80);  // scales are below 2^ex
              const float unit = __uint_as_float((uint32_t)(127 - min(ex, 126)) << 23);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                me.ks[32 * e + lane] = ks[e];
                me.vs[32 * e + lane] = vs[e];
              }
              if (lane == 0) {
                me.wide = ex > (int)kFarGap || __uint_as_float(top) > 16.0f * __uint_as_float(low);
                me.lv = (float)ex;
                me.unit = unit;
              }
            }
            if (lane == 0) me.end = 0;
          }
          __syncwarp();
          if (mine && lane == 0) mbar_arrive(b_meta + 8 * (t & (kMeta - 1)));
        }
      });
    }
  } else {
    // ------------------------------------------------------------------ softmax --
    more_registers<NT>();
    const int wg = warp >> 2, r = (warp & 3) * 32 + lane;  // warpgroup; row = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + lane_off + kSBuf * kTile + wg * 128;
    // A tile keeps the row's reference while its exponentials sum up to no more than the cap:
    // far inside fp32 (bf16 P has its exponents), or what fp16 holds of them times V's scale.
    constexpr float kSumCap = B16 ? 1.8446744e19f : 32768.0f;
    constexpr float kTop = B16 ? 0.0f : 7.0f;  // log2 of the largest weight when m is set
    constexpr float kLogitCap = 1.8446744e19f;   // 8-bit formats: a tile's share of l, before its reference follows
    int t = 0, c = wg, seg = 0;  // tiles with end marks, products, segments
    // pairs: parities of the next S of this warpgroup, and of the P V of its two P tiles
    uint32_t s_par = 0u, pv_par = 0u;
    bool ok = true;
    for_segments(a, slice, blockIdx.x, lane, [&](int64_t partial, int, int rg, int b, int, int, int) {
      if (!ok) return;
      const int row0 = rg * NT * kRows, x = row0 + (NT == 2 ? wg * kRows : 0) + r;
      const bool on = x < a.rows;
      const int tt = min(x, a.rows - 1) / a.gq, ti = tt - row0 / a.gq;  // token; its place in the row group
      const bool alive = on && tree_word(a, b, tt) != 0ull;
      // a row that is no token sees nothing: its reference need not be looked for
      // 8-bit formats: m is the reference of O, that is of P times V's scale; the sum l has one of
      // its own, ml, of the logits alone, since V's scales may lie further apart than fp32's
      // exponents reach and a key counts in l whatever its V row's size.  The exponentials are
      // taken against m, or ml while m is far above it (the scales are large), and multiplied by
      // back = 2^(ml - m) for P then; gap = 2^(ref - ml) brings their sums to l.
      float m = alive ? -INFINITY : 0.0f, l = 0.0f, fac = a.sl2;
      float ml = m, ref = m, gap = 0.0f, back = 1.0f, most = INFINITY;  // most: kLogitCap / gap
      bool far = false;  // some row of the warp is far
      const int c0 = c;
      // This warpgroup's last product P V (that of tile t - 1) is done.
      auto pv_done = [&]() {
        if constexpr (L::PAIR) {
          const int at = (t - 1) & 1;  // (its bit was turned when its P was handed over)
          return wait_all(b_pv + 8 * (2 * wg + at), (pv_par >> at & 1u) ^ 1u);
        } else {
          return wait_all(b_pv + 8 * ((c - NT) % kSBuf), (c - NT) / kSBuf);
        }
      };
      for (;; ++t, c += NT) {
        const Meta& me = meta[t & (kMeta - 1)];
        if (!(ok = wait_all(b_meta + 8 * (t & (kMeta - 1)), t / kMeta))) return;
        if (me.end) break;
        if (!B16 && c == c0) fac = a.sl2 * down[((seg & 1) * NT + (NT == 2 ? wg : 0)) * kRows + r];
        const uint64_t see = alive ? me.see[ti] : 0ull;
        const int buf = L::PAIR ? 2 * wg + (t & 1) : c % kSBuf;
        if constexpr (L::PAIR) {
          if (c == c0 || !(t & 1)) {  // a new pair's S
            if (!(ok = wait_all(b_s + 8 * wg, s_par))) return;
            s_par ^= 1u;
          }
        } else {
          if (!(ok = wait_all(b_s + 8 * buf, c / kSBuf))) return;
        }
        tc_fence_after();
        const uint32_t tS = tmem + lane_off + buf * kTile;
        uint32_t x0[32], x1[32];
        tmem_ld32(tS, x0);
        tmem_ld32(tS + 32, x1);
        tmem_ld_wait(x0);
        tie32(x1);
        float lv = 0.0f, unit = 1.0f;
        bool wide = false;
        if constexpr (!B16) {
          lv = me.lv;
          unit = me.unit;
          wide = far || me.wide != 0;
          auto by_k = [&](uint32_t(&xx)[32], int cb) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 s = *reinterpret_cast<const float4*>(me.ks + cb + i);
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
        if (!__all_sync(0xffffffffu, see == ~0ull)) {  // keys that this row does not see
          constexpr uint32_t kNeg = 0xff800000u;
          const uint32_t s0 = (uint32_t)see, s1 = (uint32_t)(see >> 32);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            x0[i] = s0 >> i & 1u ? x0[i] : kNeg;
            x1[i] = s1 >> i & 1u ? x1[i] : kNeg;
          }
        }
        // ---- exponentials against the row's reference m, which moves only when a tile's
        // sum passes the cap or while the row has seen no key.  8-bit formats: V's scales are
        // below 2^lv in this tile; a tile whose scales are far apart (an outlier that this row
        // may not even see) is measured key by key, and so are all while some row is far.
        float f = 1.0f;                    // what O has to be multiplied by
        const bool seen = m != -INFINITY;  // without a key so far O is zero
        float la, lb;
        auto take_max = [&]() {
          float mm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; ++i)
            mm[i & 3] = max3(mm[i & 3], __uint_as_float(x0[i]), __uint_as_float(x1[i]));
          const float top = fmaxf(fmaxf(mm[0], mm[1]), fmaxf(mm[2], mm[3])) * fac;
          float mx = top + lv;
          if constexpr (!B16) {
            if (wide) {
              mx = -INFINITY;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                mx = fmaxf(mx, __uint_as_float(x0[i]) * fac + __log2f(fmaxf(fabsf(me.vs[i]), kTinyScale)));
                mx = fmaxf(mx, __uint_as_float(x1[i]) * fac + __log2f(fmaxf(fabsf(me.vs[32 + i]), kTinyScale)));
              }
            }
          }
          if (mx - kTop > m + (wide ? 7.0f : 0.0f)) {  // (key by key, fp16 has room for another 2^7)
            mx -= kTop;
            if (seen) f = ex2(m - mx);
            if (B16) l *= f;
            m = mx;
          }
          if constexpr (!B16) {
            if (top > ml) {
              l *= ex2(ml - top);
              ml = top;
            }
            const bool mine = m - ml > kFarGap;
            far = __any_sync(0xffffffffu, mine);
            ref = mine ? ml : m;
            back = mine ? ex2(ml - m) : 1.0f;
            gap = m == -INFINITY ? 0.0f : ex2(ref - ml);
            most = kLogitCap / gap;
          } else {
            ref = m;
          }
        };
        auto emit_all = [&]() {
          const float nms = m == -INFINITY ? 0.0f : -ref;
          la = 0.0f;
          lb = 0.0f;
          auto emit = [&](uint32_t(&xx)[32], int k) {  // P over its S, which is in registers
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              float y[8];
#pragma unroll
              for (int e = 0; e < 8; e += 2)
                ffma2(y[e], y[e + 1], __uint_as_float(xx[2 * i + e]), __uint_as_float(xx[2 * i + e + 1]), fac, fac,
                      nms, nms);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = ex2(y[e]);
#pragma unroll
              for (int e = 0; e < 8; e += 2) fadd2(la, lb, la, lb, y[e], y[e + 1]);
              if constexpr (B16) {
#pragma unroll
                for (int e = 0; e < 4; ++e) pk[i + e] = pack_bf16(y[2 * e], y[2 * e + 1]);
              } else {
#pragma unroll
                for (int e = 0; e < 8; e += 4) {  // times V's scale in fp32, rounded once
                  const float4 s = *reinterpret_cast<const float4*>(me.vs + 32 * k + 2 * i + e);
                  fmul2(y[e], y[e + 1], y[e], y[e + 1], s.x, s.y);
                  fmul2(y[e + 2], y[e + 3], y[e + 2], y[e + 3], s.z, s.w);
                }
                if (far) {
#pragma unroll
                  for (int e = 0; e < 8; e += 2) fmul2(y[e], y[e + 1], y[e], y[e + 1], back, back);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) pk[i + e] = pack_f16(y[2 * e], y[2 * e + 1]);
              }
            }
            tmem_st16(tS + 16 * k, pk);
          };
          emit(x0, 0);
          emit(x1, 1);
        };
        // (a loop, so that the code is there once: the warps' instructions share a cache)
        bool again = wide || __any_sync(0xffffffffu, m == -INFINITY);
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
          if (again) take_max();
          emit_all();
          const float cap = B16 ? kSumCap : wide ? INFINITY : fminf(kSumCap * unit, most);
          again = pass == 0 && __any_sync(0xffffffffu, !(la + lb <= cap));
          if (!again) break;
        }
        l += B16 ? la + lb : (la + lb) * gap;
        if (__any_sync(0xffffffffu, f != 1.0f) && c > c0) {
          // O of this warpgroup's earlier products follows the reference
          if (!(ok = pv_done())) return;
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
        if (lane == 0) mbar_arrive(b_p + 8 * buf);
        if (L::PAIR) pv_par ^= 1u << (t & 1);
      }
      // ---- this segment's partial
      const bool some = c > c0;
      if (some) {
        if (!(ok = pv_done())) return;
        tc_fence_after();
      }
      ++t;  // the end mark
      const int64_t slot = (partial * NT + wg) * kRows + r;
      if (on) a.part_ml[slot] = make_float2(B16 ? m : ml, some ? l : 0.0f);
      if (some) {
        // (8-bit formats: O goes over to the reference that the merge knows, that of l)
        const float to_l = B16 ? 1.0f : ex2(m - ml);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint32_t y[32];
          tmem_ld32(tO + 32 * k, y);
          tmem_ld_wait(y);
          if (on) {
            float4* dst = reinterpret_cast<float4*>(a.part_acc + slot * D + 32 * k);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float4 z = make_float4(__uint_as_float(y[4 * i]), __uint_as_float(y[4 * i + 1]),
                                     __uint_as_float(y[4 * i + 2]), __uint_as_float(y[4 * i + 3]));
              if constexpr (!B16) z.x *= to_l, z.y *= to_l, z.z *= to_l, z.w *= to_l;
              dst[i] = z;
            }
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

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
  static EncodeTiled fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(p);
  });
  return fn;
}

// Tensor map of a cache, [B * cap, H_kv, D]; box: kTile slots of one head, 64 bf16 columns in
// the operand tiles' swizzle, or a whole row of codes.
bool make_map(CUtensorMap* m, const void* base, const TreeArgs& a, int D, bool b16) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t es = b16 ? 2 : 1;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.H_kv, (cuuint64_t)a.B * a.cap};
  const cuuint64_t strides[2] = {(cuuint64_t)D * es, (cuuint64_t)a.H_kv * D * es};
  const cuuint32_t box[3] = {(cuuint32_t)(b16 ? 64 : D), 1, kTile}, step[3] = {1, 1, 1};
  return fn(m, b16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base),
            dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            b16 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int FMT, int NT, bool HOLD>
cudaError_t launch(TreeArgs a, cudaStream_t s) {
  using L = Tc<D, FMT, NT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(tree_tc<D, FMT, NT, HOLD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Tc<D, FMT, NT>::BYTES);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap mk{}, mv{};
  // a TMA coordinate is 32 bits; beyond that (or without the encoder) rows come one by one
  a.tma = (int64_t)a.B * a.cap < INT32_MAX && make_map(&mk, a.kc, a, D, L::B16) && make_map(&mv, a.vc, a, D, L::B16);
  tree_tc<D, FMT, NT, HOLD><<<(unsigned)a.G, kThreads, L::BYTES, s>>>(a, mk, mv);
  return cudaGetLastError();
}

template <int D, int FMT>
cudaError_t launch_nt(const TreeArgs& a, cudaStream_t s) {
  return a.grp == kRows ? launch<D, FMT, 1, false>(a, s) : launch<D, FMT, 2, false>(a, s);
}

}  // namespace

cudaError_t launch_tree_tc(const TreeArgs& a, int d_head, int format, cudaStream_t s) {
  if (d_head == 64)
    return format == FOCUS_CACHE_BF16   ? launch_nt<64, FOCUS_CACHE_BF16>(a, s)
           : format == FOCUS_CACHE_E4M3 ? launch_nt<64, FOCUS_CACHE_E4M3>(a, s)
                                        : launch_nt<64, FOCUS_CACHE_INT8>(a, s);
  return format == FOCUS_CACHE_BF16   ? launch_nt<128, FOCUS_CACHE_BF16>(a, s)
         : format == FOCUS_CACHE_E4M3 ? launch_nt<128, FOCUS_CACHE_E4M3>(a, s)
                                      : launch_nt<128, FOCUS_CACHE_INT8>(a, s);
}

cudaError_t launch_tree_tc_held(const TreeArgs& a, int format, cudaStream_t s) {
  constexpr int B = FOCUS_CACHE_BF16, I = FOCUS_CACHE_INT8;
  if (format == B) return a.grp == kRows ? launch<128, B, 1, true>(a, s) : launch<128, B, 2, true>(a, s);
  return a.grp == kRows ? launch<128, I, 1, true>(a, s) : launch<128, I, 2, true>(a, s);
}

}  // namespace focus
