// mk_cache.cu -- moving rows of the decoder's cache: accepted drafts, forks and beams.
//
// Both kernels only copy, in place, 16 bytes per thread and access; their bound is memory.  Rows
// are head_dim 16-bit values; a plane is one (layer, K|V, sequence, KV head).
#include <cuda_runtime.h>

#include "mk_internal.h"
#include "mk_ptx.cuh"

namespace mk {
namespace cache {

constexpr int kThreads = 256;
constexpr int kMaxNodes = MK_MAX_TREE_NODES;

struct Params {
  uint4* base;
  int64_t layer, kv, seq, head;  // strides in 16-byte pieces; a row is `row` pieces
  int layers, B, hkv, max_seq, row;
  const int32_t *path, *n_path, *src, *lens;
  int32_t* new_lens;
  int n;
};

// ---- commit: row len + path[j] to row len + j ----
// path[j] >= j and both grow, so a row is never written before a later copy has read it as long
// as the copies of a plane go in order: a warp takes a plane's 32 / row copies at a time, several
// such groups' loads before their stores.  Rows of 256 bytes far apart: 16 sequences' paths through
// 64-node trees (32 layers, 32 heads of 128) take 13 us, the rate of a plain copy; one sequence's
// (8 heads) 2.4 us.  Six blocks per SM, all resident at once, read the path once each: with a block for
// every 8 planes, eight groups in flight and so three blocks per SM it took 23 us.
constexpr int kCommitBlocks = 6;
__global__ void __launch_bounds__(kThreads, kCommitBlocks) commit(const Params P) {
  griddep_wait();
  __shared__ int16_t path[kMaxNodes];
  __shared__ int s_count, s_first;
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = min(max(P.lens[b], 0), P.max_seq);
  if (warp == 0) {
    // the path counts up to the first entry that is out of order, out of range or behind the cache
    const int want = min(max(P.n_path[b], 0), P.n), room = min(P.n, P.max_seq - len);
    int count = 0, first = kMaxNodes;
    for (int j0 = 0; j0 < want; j0 += 32) {
      const int j = j0 + lane;
      const int x = j < want ? P.path[(int64_t)b * P.n + j] : -1;
      int before = __shfl_up_sync(0xffffffffu, x, 1);
      if (lane == 0) before = j0 ? (int)path[j0 - 1] : -1;
      const uint32_t ok = __ballot_sync(0xffffffffu, j < want && x > before && x < room);
      if (j < want) path[j] = (int16_t)x;
      __syncwarp();
      const int good = ~ok ? __ffs(~ok) - 1 : 32;  // entries in order from j0 on
      const uint32_t moved = __ballot_sync(0xffffffffu, lane < good && x != j);
      if (moved && first == kMaxNodes) first = j0 + __ffs(moved) - 1;
      count = j0 + good;
      if (good < 32) break;
    }
    if (lane == 0) {
      s_count = count, s_first = first;
      if (blockIdx.x == 0) P.new_lens[b] = len + count;
    }
  }
  __syncthreads();
  const int count = s_count, first = s_first;  // copies first .. count - 1 move something
  const int per = 32 / P.row, r = lane / P.row, c = lane - r * P.row;
  const int planes = P.layers * 2 * P.hkv;
  constexpr int kDeep = 4;
  for (int x = blockIdx.x * (kThreads / 32) + warp; x < planes; x += gridDim.x * (kThreads / 32)) {
    const int h = x % P.hkv, lk = x / P.hkv;
    uint4* p = P.base + (lk >> 1) * P.layer + (lk & 1) * P.kv + b * P.seq + h * P.head + (int64_t)len * P.row + c;
    for (int j0 = first; j0 < count; j0 += per * kDeep) {
      uint4 v[kDeep];
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const int j = j0 + k * per + r;
        if (j < count) v[k] = p[path[j] * P.row];
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const int j = j0 + k * per + r;
        if (j < count) p[j * P.row] = v[k];
      }
      __syncwarp();
    }
  }
}

// ---- reorder: sequence b takes the rows of sequence src[b] ----
// A thread takes one 16-byte place of every sequence: it loads it from every sequence that
// another one takes over, then stores, so that any map works in place (swaps, cycles, forks) and
// a row that several sequences take is read once.  8 beams of 1001 rows (32 layers, 8 heads of 128)
// take 240 to 250 us, the rate of a plain copy; a prompt of 39 rows forked to 4 answers 7 us.
constexpr int kB = MK_MAX_BATCH;

// V: what a thread takes of a place (16 bytes, or 8 where many sequences are read: the values of
// all of them are in registers at once, and fewer registers keep four blocks on an SM).
// N: sequences read at most; U: places of a thread in flight.
template <typename V, int N, int U>
__device__ __forceinline__ void move_places(const Params& P, V* p, int64_t at, int64_t step, int64_t end, int distinct,
                                            const int* from, const int* upto, const uint32_t* to) {
  constexpr int kPer = sizeof(uint4) / sizeof(V);
  const int64_t seq = P.seq * kPer;
  for (; at < end * kPer; at += step * U) {
    V v[U][N];
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int y = 0; y < N; ++y) {
        const int64_t a = at + k * step;
        if (y < distinct && a < (int64_t)upto[y] * kPer) v[k][y] = p[from[y] * seq + a];
      }
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int y = 0; y < N; ++y) {
        const int64_t a = at + k * step;
        if (y < distinct && a < (int64_t)upto[y] * kPer)
          for (uint32_t set = to[y]; set; set &= set - 1) p[(__ffs(set) - 1) * seq + a] = v[k][y];
      }
  }
}

__global__ void __launch_bounds__(kThreads, 3) reorder(const Params P) {
  griddep_wait();
  __shared__ int from[kB], upto[kB];   // sequences to read, and how many pieces of each
  __shared__ uint32_t to[kB];          // the sequences that take them
  __shared__ int s_distinct, s_most;
  const int tid = threadIdx.x;
  if (tid < 32) {
    const int b = tid;
    int src = b < P.B ? P.src[b] : -1;
    if (src < 0 || src >= P.B) src = b;  // keeps its rows
    const int len = b < P.B ? min(max(P.lens[src], 0), P.max_seq) : 0;
    const uint32_t same = __match_any_sync(0xffffffffu, b < P.B ? src : 64 + b);  // who takes what I take
    const uint32_t moves = __ballot_sync(0xffffffffu, b < P.B && src != b);
    const bool lead = b < P.B && (same & moves) && b == __ffs(same) - 1;
    const uint32_t leads = __ballot_sync(0xffffffffu, lead);
    if (lead) {
      const int y = __popc(leads & ((1u << b) - 1));
      from[y] = src, upto[y] = len * P.row, to[y] = same & moves;
    }
    int most = (same & moves) ? len * P.row : 0;
    for (int off = 16; off; off >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
    if (tid == 0) s_distinct = __popc(leads), s_most = most;
    // every block reads lens and only the first writes new_lens: they may not be one array
    if (blockIdx.x == 0 && blockIdx.y == 0 && b < P.B) P.new_lens[b] = len;
  }
  __syncthreads();
  const int distinct = s_distinct, most = s_most;
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int x = blockIdx.y; x < P.layers * 2 * P.hkv; x += gridDim.y) {
    const int h = x % P.hkv, lk = x / P.hkv;
    uint4* p = P.base + (lk >> 1) * P.layer + (lk & 1) * P.kv + h * P.head;
    const int64_t at = (int64_t)blockIdx.x * kThreads + tid;
    if (distinct == 1)
      move_places<uint4, 1, 4>(P, p, at, step, most, distinct, from, upto, to);
    else if (distinct <= 4)
      move_places<uint4, 4, 1>(P, p, at, step, most, distinct, from, upto, to);
    else if (distinct <= 8)
      move_places<uint4, 8, 1>(P, p, at, step, most, distinct, from, upto, to);
    else
      move_places<uint2, kB, 1>(P, reinterpret_cast<uint2*>(p), at, step, most, distinct, from, upto, to);
  }
}

static Params params(const mk_cache_shape& s, void* cache, const int32_t* lens, int32_t* new_lens) {
  Params P = {};
  P.base = static_cast<uint4*>(cache);
  P.layers = s.n_layers, P.B = s.B, P.hkv = s.n_kv_heads, P.max_seq = s.max_seq, P.row = s.head_dim / 8;
  P.head = (int64_t)s.max_seq * P.row, P.seq = P.head * s.n_kv_heads, P.kv = P.seq * s.max_batch, P.layer = P.kv * 2;
  P.lens = lens, P.new_lens = new_lens;
  return P;
}

}  // namespace cache

static int n_sms_now() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

int cache_commit(const mk_cache_shape& s, void* cache, const int32_t* path, int n, const int32_t* n_path,
                 const int32_t* lens, int32_t* new_lens, cudaStream_t stream, std::string* err) {
  cache::Params P = cache::params(s, cache, lens, new_lens);
  P.path = path, P.n_path = n_path, P.n = n;
  const int planes = s.n_layers * 2 * s.n_kv_heads, warps = cache::kThreads / 32;
  const int all = (planes + warps - 1) / warps, want = (cache::kCommitBlocks * n_sms_now() + s.B - 1) / s.B;
  const cudaError_t e = launch_early(cache::commit, dim3(all < want ? all : want, s.B), cache::kThreads, stream, P);
  if (e != cudaSuccess) {
    *err = std::string("cache commit launch: ") + cudaGetErrorString(e);
    return MK_ERR_CUDA;
  }
  return MK_OK;
}

int cache_reorder(const mk_cache_shape& s, void* cache, const int32_t* src, const int32_t* lens, int32_t* new_lens,
                  cudaStream_t stream, std::string* err) {
  cache::Params P = cache::params(s, cache, lens, new_lens);
  P.src = src;
  const int planes = s.n_layers * 2 * s.n_kv_heads;
  // about eight blocks per SM, along the rows first where there are few planes
  const int64_t pieces = (int64_t)s.max_seq * P.row;
  const int y = planes < 65535 ? planes : 65535, want = (8 * n_sms_now() + y - 1) / y;
  const int64_t most = (pieces + cache::kThreads - 1) / cache::kThreads;
  const cudaError_t e = launch_early(cache::reorder, dim3((unsigned)(want < most ? want : most), y), cache::kThreads, stream, P);
  if (e != cudaSuccess) {
    *err = std::string("cache reorder launch: ") + cudaGetErrorString(e);
    return MK_ERR_CUDA;
  }
  return MK_OK;
}

}  // namespace mk
