// Acceptance of drafted tokens: the path of a draft tree that the chosen tokens follow, and its
// rows moved together in the cache.
//
// A drafted token u is right when it is the first child of its parent whose token is the one
// chosen there (and not negative), and accepted when it and all its ancestors but the root are right: no walk, one
// test of 64-bit words per token (a thread each), so that a tree of depth 64 takes no longer than
// one of depth 2.  The accepted tokens are a chain 0 = u_0 < u_1 < .., and row u_i moves from slot
// len + u_i to slot len + i: never upwards, so one thread that takes a 16-byte column of all rows
// in order, some at a time, reads every source before it is written over.
// Latency-bound: two dependent loads, the words' tests, the rows' loads.  Measured: 32 chains of 5 over
// e4m3, 8 KV heads of 128, 4.2 us; 16 trees of 64 over bf16, 32 KV heads, 6.2 us (the memory needs 0.2).
// A cluster of blocks shares a sequence's columns; its barrier stands between the blocks' reading the
// length and its new value, which may be the same word.
#include <cooperative_groups.h>

#include <algorithm>

#include "tree.cuh"

namespace focus {
namespace {

namespace cg = cooperative_groups;

constexpr int kAcceptThreads = 256;

struct AcceptArgs {
  const int32_t *draft, *chosen;
  const uint64_t* tree;
  char *kc, *vc;
  float *ks, *vs;
  uint32_t* mask;
  const int32_t* lens;
  int32_t *lens_out, *count, *path, *next, *status;
  int cap, T, H_kv, R, blocks;
  int row;  // 16-byte pieces of a slot's keys
};

// Moves column x of the rows path[from ..] behind `base`; `step` elements from a slot to the next.
template <typename X>
__device__ __forceinline__ void move(X* x, int64_t step, const int* path, int from, int n) {
  constexpr int U = 8;
  for (int i0 = from; i0 < n; i0 += U) {
    X y[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i0 + i < n) y[i] = x[path[i0 + i] * step];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i0 + i < n) x[(i0 + i) * step] = y[i];
  }
}

__global__ void __launch_bounds__(kAcceptThreads) accept_path(const __grid_constant__ AcceptArgs a) {
  __shared__ uint64_t words[FOCUS_MAX_DRAFT];
  __shared__ int chosen[FOCUS_MAX_DRAFT], parents[FOCUS_MAX_DRAFT], path[FOCUS_MAX_DRAFT];
  __shared__ unsigned bits[3][2];  // right but for twins, right, accepted: a word of each of two warps
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  const int b = blockIdx.x / a.blocks, rank = blockIdx.x % a.blocks;
  const int len = a.lens[b];
  const bool fits = len >= 0 && len <= a.cap - a.T;
  if (a.blocks > 1) cg::this_cluster().barrier_arrive();
  const bool token = tid < a.T;
  const uint64_t all = a.T == 64 ? ~0ull : (1ull << a.T) - 1;
  uint64_t word = 0;
  int draft = 0;
  if (token) {
    const int64_t at = (int64_t)b * a.T + tid;
    word = fits ? (a.tree ? a.tree[at] : (2ull << tid) - 1) & all : 0ull;
    words[tid] = word;
    chosen[tid] = a.chosen[at];
    draft = a.draft[at];
  }
  __syncthreads();
  if (tid < FOCUS_MAX_DRAFT) {
    const uint64_t above = word & ((1ull << tid) - 1);
    const int parent = above ? 63 - __clzll(above) : -1;
    parents[tid] = parent;
    // (a word that is not its parent's and its own bit is of no token of the tree; a negative token is none:
    // the choice of a row without one, a place that the draft left empty)
    const bool right = token && (parent >= 0 ? word == (words[parent] | 1ull << tid) && draft >= 0 && draft == chosen[parent]
                                             : tid == 0 && word == 1ull);
    const unsigned w = __ballot_sync(0xffffffffu, right);
    if (lane == 0) bits[0][wp] = w;
  }
  __syncthreads();
  if (tid < FOCUS_MAX_DRAFT) {
    const uint64_t likely = (uint64_t)bits[0][1] << 32 | bits[0][0];
    bool right = likely >> tid & 1ull;
    if (right && tid > 0)
      for (uint64_t x = likely & ((1ull << tid) - 1) & ~1ull; x && right; x &= x - 1) right = parents[__ffsll(x) - 1] != parents[tid];
    const unsigned w = __ballot_sync(0xffffffffu, right);
    if (lane == 0) bits[1][wp] = w;
  }
  __syncthreads();
  if (tid < FOCUS_MAX_DRAFT) {
    const uint64_t right = (uint64_t)bits[1][1] << 32 | bits[1][0];
    // (a word need not have its own token's bit, where it is of no tree)
    const unsigned w = __ballot_sync(0xffffffffu, (right >> tid & 1ull) != 0ull && (word & ~right) == 0ull);
    if (lane == 0) bits[2][wp] = w;
  }
  __syncthreads();
  const uint64_t taken = (uint64_t)bits[2][1] << 32 | bits[2][0];
  const int n = __popcll(taken);
  if (token && (taken >> tid & 1ull)) path[__popcll(taken & ((1ull << tid) - 1))] = tid;
  __syncthreads();
  // rows that stay: u_i = i, up to the first token that is not accepted
  const int from = ~taken ? __ffsll(~taken) - 1 : 64;
  if (n > from) {
    const int pieces = 2 * a.row, scales = a.ks ? 2 * a.H_kv : 0;
    for (int c = rank * kAcceptThreads + tid; c < pieces + scales + a.R; c += a.blocks * kAcceptThreads) {
      if (c < pieces) {
        uint4* x = reinterpret_cast<uint4*>(c < a.row ? a.kc : a.vc) + ((int64_t)b * a.cap + len) * a.row + (c < a.row ? c : c - a.row);
        move(x, a.row, path, from, n);
      } else if (c < pieces + scales) {
        const int s = c - pieces, h = s < a.H_kv ? s : s - a.H_kv;
        move((s < a.H_kv ? a.ks : a.vs) + ((int64_t)b * a.H_kv + h) * a.cap + len, 1, path, from, n);
      } else {
        move(a.mask + ((int64_t)b * a.R + c - pieces - scales) * a.cap + len, 1, path, from, n);
      }
    }
  }
  if (a.blocks > 1) cg::this_cluster().barrier_wait();
  if (rank != 0) return;
  if (token) a.path[(int64_t)b * a.T + tid] = tid < n ? path[tid] : -1;
  if (tid == 0) {
    a.count[b] = n;
    a.next[b] = n ? chosen[path[n - 1]] : -1;
    a.lens_out[b] = len + n;
    if (!fits && a.status) raise_status(a.status, FOCUS_ERR_BOUNDS);
  }
}

}  // namespace

cudaError_t launch_tree_accept(const focus_cache_params& p, const int32_t* draft, const int32_t* chosen,
                               const uint64_t* tree, void* kc, void* vc, float* ks, float* vs, uint32_t* mask,
                               const int32_t* lens, int32_t* lens_out, int32_t* count, int32_t* path, int32_t* next,
                               int32_t* status, cudaStream_t s) {
  AcceptArgs a;
  a.draft = draft, a.chosen = chosen, a.tree = tree;
  a.kc = (char*)kc, a.vc = (char*)vc, a.ks = ks, a.vs = vs, a.mask = mask;
  a.lens = lens, a.lens_out = lens_out, a.count = count, a.path = path, a.next = next, a.status = status;
  a.cap = p.cap, a.T = p.T, a.H_kv = p.H_kv, a.R = p.R;
  a.row = p.H_kv * p.d_head * (p.format == FOCUS_CACHE_BF16 ? 2 : 1) / 16;
  // a column for each thread, eight blocks at most
  const int columns = 2 * a.row + (ks ? 2 * p.H_kv : 0) + p.R;
  a.blocks = p.T == 1 ? 1 : std::min(8, (columns + kAcceptThreads - 1) / kAcceptThreads);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * a.blocks));
  cfg.blockDim = dim3(kAcceptThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, accept_path, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace focus
