// mk_tree_attention.cu -- attention of a tree of drafted tokens over a KV cache.
//
// Formula.  Sequence b has len rows in the cache and nn drafted nodes behind them, node i at row
// len + i; A(i) is node i with its ancestors.  For query head h of node i (KV head h / G):
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j),  j in {0..len-1} + {len + a : a in A(i)}.
//
// Mapping.  The G query heads of a KV head and the nodes share their keys, so they are the rows
// of one matrix product: a row tile is 128 rows (floor(128 / G) nodes x G heads) and both
// products run on the tensor cores (M = 128, fp32 accumulators in TMEM): S = Q K^T over 64-key
// tiles, O += P V with P as the TMEM operand.  K tiles are K-major, V tiles MN-major, both as TMA
// writes them with the 128-byte swizzle.  128 rows cost the same as 1: a tile (128 values per key)
// takes the tensor cores about 0.2 us, while its 32 KB take an SM's share of HBM 0.7 us.
//
// A block holds one row tile; two blocks share an SM, so that one's start, end and softmax run
// beside the other's loads and products.  (Two row tiles per block that share every key tile, one
// block per SM, read L2 half as often and were slower: 156 us against 140 for 8 x 256 nodes, both
// with 128-key tiles.)  Four
// warps do the softmax, one issues the loads, one the products, and two helpers prepare the tree:
// the ancestor bits of every node, and V tiles that end the sequence.
//
// Bound.  With few rows per key memory: 16 sequences x 13 nodes over up to 1280 rows (32 KV heads of
// 128) take 42 to 48 us by their lengths, 4.2 to 4.8 TB/s.  With many the chain of a tile, scores -
// softmax - P - product: 8 x 256 nodes over 4096 rows (32 / 4 heads of 64) take 132 us, 550 TFLOP/s, with
// the exponential unit busy for less than half of the time and the tensor cores for a third; 4 x 64 nodes
// over up to 32768 rows (32 / 8 heads of 128, fp16) 118 to 150 us, 610 to 770 TFLOP/s, by their lengths
// and by the clock that the power limit leaves.  5 nodes over 551 rows: 7.5 us, 1 node 7.2, of which the
// loads' and the cluster's latencies are nearly all.
//
// The keys of a (sequence, KV head, row tile) unit are split over a thread-block cluster, whose
// blocks merge their partial results through distributed shared memory: no workspace, no
// atomics, a fixed order of summation.
//
// Precision.  S, the softmax statistics and O are fp32.  P is rounded to the inputs' 16-bit type
// for the second product (relative 2^-8 / 2^-11, the size of the output's own rounding).  The
// maximum that P is taken against is only moved when it grows by more than 2^8; fp16 takes P
// times 2^7, so that small weights stay clear of fp16's subnormals (largest 2^15).  With fp32 q and o
// (WIDE) q and P each enter their product as two 16-bit parts, the value's rounding and what that
// left over, so that both products see 16 (bf16) or 22 (fp16) bits of them.  That is twice the products,
// and with heads of 128 one block per SM, whose chain nothing overlaps then: the cases above take 71,
// 164, 273 and 8.6 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "mk_internal.h"
#include "mk_ptx.cuh"

namespace mk {
namespace tree {

constexpr int kKeys = 64;         // keys per tile
constexpr int kRows = 128;        // rows per row tile
constexpr int kMaxNodes = MK_MAX_TREE_NODES;
constexpr int kAncStride = kMaxNodes / 32 + 1;  // odd: rows fall on different banks
constexpr int kMaxCluster = 16;

constexpr int kSoft = 4;          // softmax warps; then loads, products, two helpers
constexpr int kTmaWarp = 4, kMmaWarp = 5, kHelper = 6;
constexpr int kThreads = 256;

template <int D, bool WIDE>
struct Geo {
  static constexpr int kTile = kKeys * D * 2;      // bytes of a K or V tile
  static constexpr int kQTile = kRows * D * 2;
  static constexpr int kStages = 4 * (128 / D);
  static constexpr int kQ = kQTile * (WIDE ? 2 : 1);  // high parts, then low parts
  static constexpr int kData = kQ + kStages * kTile;
  static constexpr int kOStride = D + 4;           // floats: 16-byte rows, no bank conflicts
  // Behind the partial O's (over Q and the ring): a warp's 32 rows x 32 columns on their way out
  static constexpr int kStageStride = 36;
  static constexpr int kStageAt = (kRows + kMaxCluster) * kOStride * 4;
  static_assert(kStageAt + kSoft * 32 * kStageStride * 4 <= kData, "partial O's and stages fit over Q and the ring");
  // Tensor memory: S of even and odd tiles at 0 and 64 (over each, P; its low parts 32 columns on),
  // O at 128.  Shared memory bounds the blocks per SM to 512 / kCols: one more would wait for tensor memory
  // while its cluster's other blocks hold theirs.
  static constexpr uint32_t kCols = 256;
  static_assert(kData > 76 * 1024, "at most two blocks per SM");
};

struct Params {
  const void* q;  // 16-bit values, or fp32 (WIDE), as o
  const uint16_t* v;
  void* o;
  const int32_t *parents, *n_nodes, *lens;
  int64_t q_seq, q_node, q_head, o_seq, o_node, o_head, v_seq, v_head, v_row;
  int n, hkv, G, max_seq;
  int nt;        // nodes per row tile
  int units;     // row tiles per (sequence, KV head)
  uint32_t inv_g;  // r / G = r * inv_g >> 16 for r < 256
  float c;       // |scale| * log2(e)
  uint32_t negate; // scale < 0: the product takes -Q (a bit of the instruction descriptor)
  uint64_t timeout_ns;
  int drop_block;  // test hook: the block that issues no loads (-1: none)
};

struct Ctl {
  uint64_t full[8], empty[8], s_full[2], p_full[2], o_done, o_full, q_full, mma_done, anc_full;
  uint32_t tmem, abort;
  uint32_t bad_v;  // infinite or NaN values among the drafts that this block saw
  // Counters that only grow, for roles that may be more than one step apart (an mbarrier's parity
  // cannot tell two steps from none): V tiles to clean that were issued; each helper's shares done.
  // (One count of both helpers' shares would not do: they do not wait for each other, so two shares
  // may be one helper's of two tiles.)
  uint32_t v_issued, v_clean[2];
  uint32_t bad_any;  // some block of the cluster has bad_v set
  // (maximum, sum) of every row that this block finishes from every block of the cluster
  float2 stat[kRows + kMaxCluster];
  uint32_t anc[kMaxNodes * kAncStride];
};

__device__ uint32_t g_err;  // first wait that ran out since the last status call

// Wait for a barrier phase, for at most timeout_ns; false when time ran out here or elsewhere.
__device__ bool wait_slow(uint64_t* bar, uint32_t parity, uint64_t timeout_ns, Ctl& S, bool quiet) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_test(bar, parity)) {
    if (!quiet && *reinterpret_cast<volatile uint32_t*>(&S.abort)) return false;
    if (globaltimer_ns() - t0 > timeout_ns) {
      *reinterpret_cast<volatile uint32_t*>(&S.abort) = 1;
      atomicExch(&g_err, 1u);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const Params& P, Ctl& S) {
  if (mbar_test(bar, parity)) return true;
  return wait_slow(bar, parity, P.timeout_ns, S, false);
}

// For a whole warp: every lane gets the same answer, as the warp-wide tcgen05 forms need.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const Params& P, Ctl& S) {
  return __all_sync(0xffffffffu, wait(bar, parity, P, S));
}

// Wait until a growing counter has reached `value`, with the same limit.
__device__ __forceinline__ bool wait_count(const uint32_t* at, uint32_t value, const Params& P, Ctl& S) {
  if ((int32_t)(ld_acquire_cta_shared(at) - value) >= 0) return true;
  const uint64_t t0 = globaltimer_ns();
  while ((int32_t)(ld_acquire_cta_shared(at) - value) < 0) {
    __nanosleep(40);
    if (*reinterpret_cast<volatile uint32_t*>(&S.abort)) return false;
    if (globaltimer_ns() - t0 > P.timeout_ns) {
      *reinterpret_cast<volatile uint32_t*>(&S.abort) = 1;
      atomicExch(&g_err, 1u);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_count_warp(const uint32_t* at, uint32_t value, const Params& P, Ctl& S) {
  return __all_sync(0xffffffffu, wait_count(at, value, P, S));
}
// Whether the helpers found infinite or NaN values among the drafts of this block's tiles, all of
// which they have cleaned by now (their counts make what they stored before visible).
__device__ __forceinline__ bool found_bad_v(const Ctl& S) {
  ld_acquire_cta_shared(&S.v_clean[0]);
  ld_acquire_cta_shared(&S.v_clean[1]);
  return S.bad_v != 0;
}
__device__ __forceinline__ void count_up(uint32_t* at) {
  asm volatile("red.release.cta.shared::cta.add.u32 [%0], 1;" ::"r"(smem_u32(at)) : "memory");
}

__device__ __forceinline__ void tma_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

// Shared-memory matrix descriptor with the 128-byte swizzle; sbo: bytes between 8-row groups,
// lbo (MN-major only): bytes between the 64-element halves.
__device__ __forceinline__ uint64_t desc128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

// The products are issued by one thread, but the whole warp walks the loop around them: the waits
// and the descriptors are the same for every lane then and stay in uniform registers.  (In a loop
// of one lane each instruction cost about 80 cycles to issue, more than it runs.)
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
// D[tmem] (+)= A[tmem] . B[smem desc], one thread.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accum)
      : "memory");
}

#define MK_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), \
                    "=r"(v[i + 6]), "=r"(v[i + 7])
#define MK_U8(v, i) "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]), \
                    "+r"(v[i + 6]), "+r"(v[i + 7])
#define MK_I8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), \
                    "r"(v[i + 6]), "r"(v[i + 7])
#define MK_LIST32                                                                                                \
  "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, " \
  "%23, %24, %25, %26, %27, %28, %29, %30, %31}"

// 32 columns of this thread's TMEM lane; valid after tmem_wait_ld on the same registers.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " MK_LIST32 ", [%32];"
               : MK_R8(r, 0), MK_R8(r, 8), MK_R8(r, 16), MK_R8(r, 24)
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Ties the registers to the wait before: nothing that uses them moves above it.
__device__ __forceinline__ void tmem_use32(uint32_t* r) {
  asm volatile("" : MK_U8(r, 0), MK_U8(r, 8), MK_U8(r, 16), MK_U8(r, 24)::"memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], " MK_LIST32 ";" ::MK_I8(r, 0), MK_I8(r, 8), MK_I8(r, 16),
      MK_I8(r, 24), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <bool FP16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (FP16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Whether a 16-bit value is infinite or NaN; its value; two values as their 16-bit roundings and
// the roundings of what those left over.
template <bool FP16>
__device__ __forceinline__ bool nonfinite16(uint32_t h) {
  constexpr uint32_t e = FP16 ? 0x7c00u : 0x7f80u;
  return (h & e) == e;
}
template <bool FP16>
__device__ __forceinline__ float value16(uint16_t h) {
  if constexpr (FP16) return __half2float(__ushort_as_half(h));
  return __uint_as_float((uint32_t)h << 16);
}

template <bool FP16>
__device__ __forceinline__ void split16(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack16<FP16>(x, y);
  lo = pack16<FP16>(x - value16<FP16>((uint16_t)hi), y - value16<FP16>((uint16_t)(hi >> 16)));
}

// Stores to a peer block's shared memory.
__device__ __forceinline__ void st_peer_f2(uint32_t addr, float x, float y) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void st_peer_v4(uint32_t addr, const uint4& x) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w)
               : "memory");
}

// Bits rel0 .. rel0 + 31 of what a node sees: every row before its drafts (rel < 0), then its
// ancestor bits; nothing behind the last node (the bits there are zero).
__device__ __forceinline__ uint32_t visible32(const uint32_t* anc, int rel0) {
  if (rel0 <= -32) return 0xffffffffu;
  if (rel0 < 0) return (anc[0] << -rel0) | ((1u << -rel0) - 1u);
  const int w = rel0 >> 5;
  if (w >= kMaxNodes / 32) return 0;
  const uint32_t hi = w + 1 < kMaxNodes / 32 ? anc[w + 1] : 0u;
  return __funnelshift_r(anc[w], hi, rel0 & 31);
}

// Loads run K two tiles ahead of V: K 0, K 1, V 0, K 2, V 1, ..: where K and V of tile j come, of T tiles.
__device__ __forceinline__ int k_index(int j) { return j < 2 ? j : 2 * j - 1; }
__device__ __forceinline__ int v_index(int j, int T) { return j + min(T, j + 2); }

// Ancestor bits (self included) of nodes 0..nn-1, one warp, 32 nodes at a time.  Within the block
// of 32 by doubling: a node takes over the bits of the node it points at, and then points where
// that one points.  What it points at then lies in an earlier block, whose bits are complete.
// `next`: the parent of node `lane`.
__device__ __forceinline__ void ancestors(const int32_t* parents, int next, int nn, uint32_t* anc, int lane) {
  for (int base = 0; base < nn; base += 32) {
    const int i = base + lane;
    int up = next;
    next = i + 32 < nn ? parents[i + 32] : -1;
    bool live = i < nn && up >= -1 && up < i;  // else not a tree's: the node sees nothing
    uint32_t own = live ? 1u << lane : 0u;
    if (!live) up = -1;
    while (__any_sync(0xffffffffu, up >= base)) {
      const int src = up >= base ? up - base : lane;
      const uint32_t bits = __shfl_sync(0xffffffffu, own, src);
      const int further = __shfl_sync(0xffffffffu, up, src);
      const bool ok = __shfl_sync(0xffffffffu, (int)live, src);
      if (up >= base) {
        own |= bits, up = further;
        if (!ok) live = false, own = 0, up = -1;
      }
    }
    uint32_t* mine = anc + i * kAncStride;
    if (up >= 0 && !(anc[up * kAncStride + (up >> 5)] >> (up & 31) & 1)) live = false;
#pragma unroll
    for (int k = 0; k < kMaxNodes / 32; ++k) {
      uint32_t w = live && up >= 0 && k * 32 < base ? anc[up * kAncStride + k] : 0u;
      if (k * 32 == base && live) w = own;
      mine[k] = w;
    }
    __syncwarp();
  }
}

// Whether a node's parents are a tree's (its own bit is set then).
__device__ __forceinline__ bool alive(const Ctl& S, int node) {
  return S.anc[node * kAncStride + (node >> 5)] >> (node & 31) & 1;
}

template <bool WIDE>
using Out = typename std::conditional<WIDE, float, uint16_t>::type;

// Infinite and NaN values of drafts that the node sees, added to n output values at `out`.
template <bool FP16, bool WIDE>
__device__ __noinline__ void add_nonfinite(const Params& P, const Ctl& S, int b, int h, int len, int node, int col,
                                           int n, Out<WIDE>* out) {
  if (!alive(S, node)) return;
  for (int a = 0; a <= node; ++a) {
    if (!(S.anc[node * kAncStride + (a >> 5)] >> (a & 31) & 1)) continue;
    const uint16_t* val = P.v + (int64_t)b * P.v_seq + (int64_t)h * P.v_head + (int64_t)(len + a) * P.v_row + col;
    for (int x = 0; x < n; ++x) {
      if (!nonfinite16<FP16>(val[x])) continue;
      if constexpr (WIDE)
        out[x] += value16<FP16>(val[x]);
      else
        out[x] = (uint16_t)pack16<FP16>(value16<FP16>(out[x]) + value16<FP16>(val[x]), 0.f);
    }
  }
}

// Output rows that this block finishes: row r's partial results, weighted, from the C blocks (they
// lie in this block's shared memory: part p of its x-th row at row p * per + x).  The loops are kept
// rolled: this runs once, and its instructions come from memory.
template <int D, bool FP16, bool WIDE>
__device__ __forceinline__ void merge(const Params& P, const Ctl& S, const float* parts, int b, int h, int first,
                                      int rows, int per, int rank, int C, int len, int warp, int lane) {
  using Ge = Geo<D, WIDE>;
  constexpr int kLanes = D / 4, kPer = 32 / kLanes;  // lanes per row, rows per warp side by side
  const int sub = lane / kLanes, in = lane % kLanes, col = in * 4;
  const int r0 = rank * per, r1 = min(rows, r0 + per);
#pragma unroll 1
  for (int base = r0 + warp * kPer; base < r1; base += kThreads / 32 * kPer) {
    const int r = min(base + sub, r1 - 1);
    // lane p of the row's group holds part p's weight (C <= 16 <= kLanes)
    const float2 st = S.stat[(r - r0) * C + (in & (C - 1))];
    float mx = st.x;
    for (int off = C / 2; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    // a part that saw no key has no O to read
    float f = st.x == -INFINITY && st.y == 0.f ? 0.f : mx == -INFINITY ? 1.f : ex2((st.x - mx) * P.c);
    float sum = st.y * f;
    for (int off = C / 2; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const int local = (int)(r * P.inv_g >> 16), g = r - local * P.G, node = first + local;
    // (a node that sees rows and has no weight for any has scores of -infinity only: 0 / 0)
    const bool live = alive(S, node);
    const float none = live && sum == 0.f ? __int_as_float(0x7fffffff) : 0.f;
    f = sum == 0.f || !live ? 0.f : __fdividef(f, sum);
    const float* src = parts + (r - r0) * Ge::kOStride + col;
    float acc[4] = {none, none, none, none};
#pragma unroll 4
    for (int p = 0; p < C; ++p) {
      const float fp = __shfl_sync(0xffffffffu, f, p, kLanes);
      const float4 v = *reinterpret_cast<const float4*>(src + p * per * Ge::kOStride);
      if (fp != 0.f) {
        acc[0] = fmaf(fp, v.x, acc[0]);
        acc[1] = fmaf(fp, v.y, acc[1]);
        acc[2] = fmaf(fp, v.z, acc[2]);
        acc[3] = fmaf(fp, v.w, acc[3]);
      }
    }
    if (base + sub >= r1) continue;
    Out<WIDE>* out = static_cast<Out<WIDE>*>(P.o) + (int64_t)b * P.o_seq + (int64_t)node * P.o_node +
                     (int64_t)(h * P.G + g) * P.o_head + col;
    if constexpr (WIDE)
      *reinterpret_cast<float4*>(out) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    else
      *reinterpret_cast<uint2*>(out) = make_uint2(pack16<FP16>(acc[0], acc[1]), pack16<FP16>(acc[2], acc[3]));
    if (S.bad_any) add_nonfinite<FP16, WIDE>(P, S, b, h, len, node, col, 4, out);
  }
}

template <int D, bool FP16, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2)
    tree_attention(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ Params P) {
  using Ge = Geo<D, WIDE>;
  extern __shared__ uint8_t raw[];
  __shared__ Ctl S;
  uint8_t* data = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  uint8_t* ring = data + Ge::kQ;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = (int)cluster_size(), rank = (int)cluster_rank();

  const int unit = blockIdx.x / C, head = unit / P.units;
  const int b = head / P.hkv, h = head - b * P.hkv;
  const int first = (unit - head * P.units) * P.nt;  // first node of the block's row tile
  const int row = tid & 127;  // of a softmax thread
  const int local = (int)(row * P.inv_g >> 16);

  // ---- start: whatever needs no input first ----
  if (warp == kTmaWarp) {
    if (lane == 0) {
      prefetch_tensormap(&map_k);
      prefetch_tensormap(&map_v);
#pragma unroll 1
      for (int i = 0; i < Ge::kStages; ++i) {
        mbar_init(&S.full[i], 1);
        mbar_init(&S.empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&S.s_full[i], 1);
        mbar_init(&S.p_full[i], kSoft);
      }
      mbar_init(&S.o_done, 1);
      mbar_init(&S.o_full, 1);
      mbar_init(&S.q_full, kSoft);
      mbar_init(&S.mma_done, 1);
      mbar_init(&S.anc_full, 1);
      S.abort = S.bad_v = S.bad_any = S.v_issued = S.v_clean[0] = S.v_clean[1] = 0;
      fence_mbar_init();
    }
  } else if (warp == kMmaWarp) {
    tc_alloc(&S.tmem, Ge::kCols);
    tc_relinquish();
  }
  griddep_wait();  // inputs and outputs belong to what ran before until here
  int len = P.lens[b], nn = P.n_nodes ? P.n_nodes[b] : P.n, parent = -1;
  if (warp == kHelper) {
    if (lane < P.n) parent = P.parents[(int64_t)b * P.n + lane];
  } else if (warp < kSoft) {
    // Q rows into the swizzled tile: 16-byte piece c of row r goes to piece c ^ (r % 8).  Rows of
    // the tile without a node keep what is there: they only reach their own, unused, results.
    const int c = row % (D / 8), used = min(P.nt, P.n - first) * P.G;
    const int64_t src = (int64_t)b * P.q_seq + (int64_t)first * P.q_node + (int64_t)h * P.G * P.q_head + c * 8;
    uint8_t* const dst = data + (c / 8) * kRows * 128;
#pragma unroll 1
    for (int r = row / (D / 8); r < used; r += kRows / (D / 8)) {
      const int lr = (int)(r * P.inv_g >> 16);
      const int64_t at = src + (int64_t)lr * P.q_node + (int64_t)(r - lr * P.G) * P.q_head;
      uint8_t* to = dst + r * 128 + ((c & 7) ^ (r & 7)) * 16;
      if constexpr (WIDE) {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(P.q) + at);
        const float4 x = f[0], y = f[1];
        uint4 hi, lo;
        split16<FP16>(x.x, x.y, hi.x, lo.x);
        split16<FP16>(x.z, x.w, hi.y, lo.y);
        split16<FP16>(y.x, y.y, hi.z, lo.z);
        split16<FP16>(y.z, y.w, hi.w, lo.w);
        *reinterpret_cast<uint4*>(to) = hi;
        *reinterpret_cast<uint4*>(to + Ge::kQTile) = lo;
      } else {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)),
                     "l"(static_cast<const uint16_t*>(P.q) + at)
                     : "memory");
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;

  len = min(max(len, 0), P.max_seq), nn = min(min(max(nn, 0), P.n), P.max_seq - len);
  const bool on = first < nn;                      // else there is no node here (the whole cluster alike)
  const int T_all = on ? (len + nn + kKeys - 1) / kKeys : 0;
  const int t0 = rank * T_all / C, T = (rank + 1) * T_all / C - t0;
  const int edge = max(0, len / kKeys - t0);  // first tile of this block that has rows behind len
  const int rows = min(nn - first, P.nt) * P.G, per = (rows + C - 1) / C;  // rows; of these to finish

  if (warp == kTmaWarp) {
    // ---- loads: K and V of a tile in turn ----
    if (lane == 0 && (int)blockIdx.x != P.drop_block) {
      int x = 0;
      auto load = [&](const CUtensorMap* map, int tile) {
        const int stage = x % Ge::kStages, use = x / Ge::kStages;
        if (use > 0 && !wait(&S.empty[stage], (use - 1) & 1, P, S)) return false;
        mbar_arrive_expect_tx(&S.full[stage], Ge::kTile);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_4d(ring + stage * Ge::kTile + c * kKeys * 128, map, c * 64, (t0 + tile) * kKeys, h, b, &S.full[stage]);
        ++x;
        return true;
      };
#pragma unroll 1
      for (int j = -2; j < T; ++j) {
        if (j + 2 < T && j < 0 && !load(&map_k, j + 2)) break;
        if (j >= 0) {
          if (!load(&map_v, j)) break;
          if (j >= edge) count_up(&S.v_issued);
          if (j + 2 < T && !load(&map_k, j + 2)) break;
        }
      }
      if (x < 2 * T)  // given up: leave no copy in flight
        for (int y = max(0, x - Ge::kStages); y < x; ++y)
          wait_slow(&S.full[y % Ge::kStages], (y / Ge::kStages) & 1, P.timeout_ns, S, true);
    }
  } else if (warp == kMmaWarp) {
    // ---- products ----
    if (T > 0) {
      constexpr uint32_t type = FP16 ? 0u : 1u;
      constexpr uint32_t idesc = (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)(kRows >> 4) << 24);
      const uint32_t idesc_s = idesc | P.negate | ((uint32_t)(kKeys >> 3) << 17);
      constexpr uint32_t idesc_o = idesc | (1u << 16) | ((uint32_t)(D >> 3) << 17);  // V is MN-major
      const uint32_t tm = __reduce_or_sync(0xffffffffu, tmem);
      const uint64_t q_desc = desc128(smem_u32(data), 16, 1024), k_desc = desc128(smem_u32(ring), 16, 1024),
                     v_desc = desc128(smem_u32(ring), kKeys * 128, 1024);
      bool ok = wait_warp(&S.q_full, 0, P, S);
      tc_fence_after();
      // step j = -2 .. T - 1: O += P V of tile j, then S = Q K^T of tile j + 2, over the S and P of
      // tile j: a tile's scores are there before its softmax can begin
#pragma unroll 1
      for (int j = -2; ok && j < T; ++j) {
        const int buf = j & 1;
        if (j >= 0) {
          const int x = v_index(j, T), stage = x % Ge::kStages;
          ok = wait_warp(&S.full[stage], (x / Ge::kStages) & 1, P, S) &&
               (j < edge || (wait_count_warp(&S.v_clean[0], j - edge + 1, P, S) &&
                             wait_count_warp(&S.v_clean[1], j - edge + 1, P, S))) &&
               wait_warp(&S.p_full[buf], (j >> 1) & 1, P, S);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = v_desc + (uint32_t)(stage * (Ge::kTile >> 4));
          if (elect()) {
#pragma unroll
            for (int s = 0; s < kKeys / 16; ++s)
              mma_ts(tm + 128, tm + buf * 64 + s * 8, vd + s * (2048 >> 4), idesc_o, j != 0 || s != 0);
            if constexpr (WIDE)
#pragma unroll
              for (int s = 0; s < kKeys / 16; ++s)
                mma_ts(tm + 128, tm + buf * 64 + 32 + s * 8, vd + s * (2048 >> 4), idesc_o, 1);
            tc_commit(&S.o_done);
            tc_commit(&S.empty[stage]);
          }
          __syncwarp();
        }
        if (j + 2 < T) {
          const int x = k_index(j + 2), stage = x % Ge::kStages;
          ok = wait_warp(&S.full[stage], (x / Ge::kStages) & 1, P, S);
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = k_desc + (uint32_t)(stage * (Ge::kTile >> 4));
          if (elect()) {
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              tc_mma_f16(tm + buf * 64, q_desc + (((s / 4) * kRows * 128 + (s % 4) * 32) >> 4),
                         kd + (((s / 4) * kKeys * 128 + (s % 4) * 32) >> 4), idesc_s, s != 0);
            if constexpr (WIDE)
#pragma unroll
              for (int s = 0; s < D / 16; ++s)
                tc_mma_f16(tm + buf * 64, q_desc + ((Ge::kQTile + (s / 4) * kRows * 128 + (s % 4) * 32) >> 4),
                           kd + (((s / 4) * kKeys * 128 + (s % 4) * 32) >> 4), idesc_s, 1);
            tc_commit(&S.s_full[buf]);
            tc_commit(&S.empty[stage]);
          }
          __syncwarp();
        }
      }
      if (elect()) {
        if (ok) tc_commit(&S.o_full);
        tc_commit(&S.mma_done);  // nothing in flight when TMEM is freed
      }
      __syncwarp();
      __all_sync(0xffffffffu, wait_slow(&S.mma_done, 0, P.timeout_ns, S, true));
    }
  } else if (warp >= kHelper) {
    // ---- helpers: the tree, and V tiles that end the sequence ----
    if (on && warp == kHelper) {
      ancestors(P.parents + (int64_t)b * P.n, parent, nn, S.anc, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.anc_full);
    }
    // 0 x inf and 0 x NaN must not reach rows that do not see the key: rows behind the last node
    // become zero, and so do infinite and NaN values of drafts (their own descendants get them
    // back at the end).
#pragma unroll 1
    for (int j = edge; j < T; ++j) {
      const int x = v_index(j, T), stage = x % Ge::kStages;
      if (!wait_count_warp(&S.v_issued, j - edge + 1, P, S)) break;
      if (!wait_warp(&S.full[stage], (x / Ge::kStages) & 1, P, S)) break;
      uint4* tile = reinterpret_cast<uint4*>(ring + stage * Ge::kTile);
      const int key0 = (t0 + j) * kKeys, from = max(0, len - key0);
      const int drafts = min(kKeys, len + nn - key0);  // keys from .. drafts - 1 are drafts
      // each helper takes every other group of four keys: 8 pieces of 16 bytes per key and half
#pragma unroll 1
      for (int key = (from & ~3) + (warp - kHelper) * 4 + lane / 8; key < kKeys; key += 8) {
        if (key < from) continue;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint4* at = tile + (c * kKeys + key) * 8 + lane % 8;
          uint4 val = make_uint4(0, 0, 0, 0);
          if (key < drafts) {
            val = *at;
            uint32_t* e = reinterpret_cast<uint32_t*>(&val);
            bool bad = false;
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              if (nonfinite16<FP16>(e[z])) e[z] &= 0xffff0000u, bad = true;
              if (nonfinite16<FP16>(e[z] >> 16)) e[z] &= 0xffffu, bad = true;
            }
            if (!bad) continue;
            S.bad_v = 1;
          }
          *at = val;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) count_up(&S.v_clean[warp - kHelper]);
    }
  } else {
    // ---- softmax: one thread per row ----
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.q_full);
    __syncwarp();  // here and below: the warp-wide tcgen05 forms want the lanes together
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_at = lane_base, o_at = lane_base + 128;
    const int node = first + local;
    const bool real = local < P.nt && node < nn;
    const bool any = __any_sync(0xffffffffu, real);  // else the warp's rows are left alone (their P is garbage)
    const uint32_t* anc = S.anc + (real ? node : 0) * kAncStride;
    constexpr float kBias = FP16 ? 7.f : 0.f;
    float m = -INFINITY, l = 0.f;  // maximum that P is taken against; sum of P
    bool ok = true;
#pragma unroll 1
    for (int j = 0; j < T; ++j) {
      if (j == edge) ok = ok && wait_warp(&S.anc_full, 0, P, S);
      ok = ok && wait_warp(&S.s_full[j & 1], (j >> 1) & 1, P, S);
      tc_fence_after();
      if (any) {
        uint32_t s[kKeys];
        tmem_ld32(s_at + (j & 1) * 64, s);
        tmem_ld32(s_at + (j & 1) * 64 + 32, s + 32);
        tmem_wait_ld();
        tmem_use32(s);
        tmem_use32(s + 32);
        if (j >= edge) {  // the tile has drafts, or rows behind the last one
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t see = visible32(anc, (t0 + j) * kKeys + k * 32 - len);
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!(see >> x & 1)) s[k * 32 + x] = 0xff800000u;
          }
        }
        float mx[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < kKeys; x += 2)
          mx[x / 2 & 3] = fmaxf(mx[x / 2 & 3], fmaxf(__uint_as_float(s[x]), __uint_as_float(s[x + 1])));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const bool move = real && (top - m) * P.c > 8.f;  // also from -inf; false for -inf - -inf
        if (__any_sync(0xffffffffu, move)) {
          const float f = top == -INFINITY ? 1.f : ex2((m - top) * P.c);
          m = top;
          l *= f;
          if (j > 0) {
            ok = ok && wait_warp(&S.o_done, (j - 1) & 1, P, S);  // (tile j - 2's is: S of tile j came after it)
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
              uint32_t o[32];
              tmem_ld32(o_at + k * 32, o);
              tmem_wait_ld();
              tmem_use32(o);
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
              tmem_st32(o_at + k * 32, o);
            }
          }
        }
        const float nm = m == -INFINITY ? 0.f : kBias - m * P.c;
        const uint64_t nm2 = pack2(nm, nm), c2 = pack2(P.c, P.c);
        uint64_t e[kKeys / 2];
#pragma unroll
        for (int x = 0; x < kKeys / 2; ++x) {
          const uint64_t y = pack2(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1]));
          asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e[x]) : "l"(y), "l"(c2), "l"(nm2));
        }
#pragma unroll
        for (int x = 0; x < kKeys / 2; ++x) {
          const float2 y = unpack2(e[x]);
          e[x] = pack2(ex2(y.x), ex2(y.y));
        }
        uint64_t sum[4] = {e[0], e[1], e[2], e[3]};
        uint32_t p[kKeys / 2], low[WIDE ? kKeys / 2 : 1];
#pragma unroll
        for (int x = 0; x < kKeys / 2; ++x) {
          const float2 y = unpack2(e[x]);
          if constexpr (WIDE)
            split16<FP16>(y.x, y.y, p[x], low[x]);
          else
            p[x] = pack16<FP16>(y.x, y.y);
          if (x >= 4) asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum[x & 3]) : "l"(e[x]));
        }
        tmem_st32(s_at + (j & 1) * 64, p);  // over scores that are read
        if constexpr (WIDE) tmem_st32(s_at + (j & 1) * 64 + 32, low);
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum[0]) : "l"(sum[1]));
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum[2]) : "l"(sum[3]));
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum[0]) : "l"(sum[2]));
        l += unpack2(sum[0]).x + unpack2(sum[0]).y;
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.p_full[j & 1]);
      __syncwarp();
    }
    // ---- the end: every product is done, Q and the ring are read out ----
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the next kernel may take the places that fall free
    if (T > 0) ok = ok && wait_warp(&S.o_full, 0, P, S);
    tc_fence_after();
    if (C > 1) cluster_sync();  // every block's Q and ring are read out
    if (any) {
      if (C == 1) {
        if (ok) ok = wait_warp(&S.anc_full, 0, P, S);
        const float inv = !real || !alive(S, node) ? 0.f : 1.f / l;  // (l = 0, scores of -infinity only: 0 x inf, NaN)
        Out<WIDE>* out = static_cast<Out<WIDE>*>(P.o) + (int64_t)b * P.o_seq + (int64_t)node * P.o_node +
                         (int64_t)(h * P.G + row - local * P.G) * P.o_head;
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          uint32_t o[32];
          tmem_ld32(o_at + k * 32, o);
          tmem_wait_ld();
          tmem_use32(o);
          if (real)
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
              float f[8];
#pragma unroll
              for (int y = 0; y < 8; ++y) f[y] = inv == 0.f ? 0.f : __uint_as_float(o[x + y]) * inv;
              if constexpr (WIDE) {
                *reinterpret_cast<float4*>(out + k * 32 + x) = make_float4(f[0], f[1], f[2], f[3]);
                *reinterpret_cast<float4*>(out + k * 32 + x + 4) = make_float4(f[4], f[5], f[6], f[7]);
              } else {
                *reinterpret_cast<uint4*>(out + k * 32 + x) = make_uint4(
                    pack16<FP16>(f[0], f[1]), pack16<FP16>(f[2], f[3]), pack16<FP16>(f[4], f[5]), pack16<FP16>(f[6], f[7]));
              }
            }
          __syncwarp();
        }
        if (real && found_bad_v(S)) add_nonfinite<FP16, WIDE>(P, S, b, h, len, node, 0, D, out);
      } else {
        // a row's statistics and O to the block that finishes it, over that block's Q and ring
        const int owner = real ? row / per : 0, x = row - owner * per;
        if (real) {
          st_peer_f2(mapa(smem_u32(&S.stat[x * C + rank]), owner), m, l);
          if (found_bad_v(S)) st_peer_u32(mapa(smem_u32(&S.bad_any), owner), 1);
        }
        __syncwarp();
        if (T > 0) {
          // 32 columns at a time through a corner of shared memory, so that a row's 128 bytes leave
          // together: eight lanes per row
          const uint32_t dst = mapa(smem_u32(data) + (uint32_t)((rank * per + x) * Ge::kOStride * 4), owner);
          float* corner = reinterpret_cast<float*>(data + Ge::kStageAt) + warp * 32 * Ge::kStageStride;
          const int rows_here = min(32, rows - warp * 32);
#pragma unroll 1
          for (int k = 0; k < D / 32; ++k) {
            uint32_t o[32];
            tmem_ld32(o_at + k * 32, o);
            tmem_wait_ld();
            tmem_use32(o);
#pragma unroll
            for (int y = 0; y < 32; y += 4)
              *reinterpret_cast<uint4*>(corner + lane * Ge::kStageStride + y) = make_uint4(o[y], o[y + 1], o[y + 2], o[y + 3]);
            __syncwarp();
#pragma unroll 2
            for (int y = 0; y < rows_here; y += 4) {
              const int from = y + lane / 8;
              const uint32_t to = __shfl_sync(0xffffffffu, dst, from & 31);
              const uint4 v = *reinterpret_cast<const uint4*>(corner + from * Ge::kStageStride + lane % 8 * 4);
              if (from < rows_here) st_peer_v4(to + (k * 32 + lane % 8 * 4) * 4, v);
            }
            __syncwarp();
          }
        }
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  if (C > 1) {
    if (warp >= kSoft) cluster_sync();
    cluster_sync();  // every partial result has arrived; no block touches another's memory after this
  } else {
    __syncthreads();
  }
  tc_fence_after();
  if (warp == kMmaWarp) tc_dealloc(tmem, Ge::kCols);
  if (C > 1 && on)
    merge<D, FP16, WIDE>(P, S, reinterpret_cast<const float*>(data), b, h, first, rows, per, rank, C, len, warp, lane);
}

// Clusters of 2, 4, 8 and 16 blocks that the device runs at once, asked once per device and kernel.
// (The query counts one block per SM for this kernel at any size of shared memory; two run where
// that has room for them, by their active warps, and its answer is doubled there.)
template <int D, bool FP16, bool WIDE>
static cudaError_t clusters_at_once(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int* fit) {
  static std::atomic<uint64_t> known[64];  // four counts of 16 bits, 1 + each
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  uint64_t v = dev < 64 ? known[dev].load() : 0;
  if (!v) {
    const auto kernel = tree_attention<D, FP16, WIDE>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)  // two blocks per SM need nearly all of its shared memory
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    for (int k = 0; k < 4; ++k) {
      attr[0].val.clusterDim.x = 2u << k;
      cfg.gridDim = dim3(2u << k);
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
      }
      v |= (uint64_t)(1 + (n < 60000 ? n : 60000)) << (16 * k);
    }
    if (dev < 64) known[dev].store(v);
  }
  const int per_sm = cfg.dynamicSmemBytes > 100 * 1024 ? 1 : 2;
  for (int k = 0; k < 4; ++k) fit[k] = per_sm * ((int)(v >> (16 * k) & 0xffff) - 1);
  return cudaSuccess;
}

template <int D, bool FP16, bool WIDE>
static cudaError_t launch(const CUtensorMap& mk_, const CUtensorMap& mv, Params& P, int B, int n_sms, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Geo<D, WIDE>::kData + 1024;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  int fit[4];
  const cudaError_t e = clusters_at_once<D, FP16, WIDE>(cfg, attr, fit);
  if (e != cudaSuccess) return e;
  P.units = (P.n + P.nt - 1) / P.nt;
  const int64_t units = (int64_t)B * P.hkv * P.units;
  if (units > (1 << 27)) return cudaErrorInvalidValue;
  // Blocks that share a unit's keys: the split with the least estimated time.  A block takes as long
  // as 7.3 tiles (0.7 us each) for its start and end, a cluster's exchange some more, and all that half
  // as long again where two share an SM; more clusters than run at once go in turns (a few more than
  // one turn's cost little).  Measured, us for 1, 2, 4, 8, 16 blocks: 8 units of 144 rows 6.5 7.2 7.2 7.5
  // 8.2; 8 of 1040 rows 16 12 9.2 8.2 9.9; 8 of 4122 rows 53 35 25 19 18; 16 of 2056 rows 31 23 17 14 23;
  // 32 of 1040 rows 16 13 10 12 25; 128 of 1040 rows 17.8 18.3 24 36 78; 64 of 16448 rows 192 107 82 110
  // 150; 512 of 4352 rows 136 147 180 270 577.
  constexpr double exchange[5] = {0.0, 2.1, 2.7, 3.5, 6.0};
  const double tiles = (double)P.max_seq / kKeys;
  int C = 1;
  double best = 0.0;
  for (int k = 0; k < 5 && (k == 0 || (int64_t)kKeys << (k - 1) < P.max_seq); ++k) {
    const int at_once = k == 0 ? (cfg.dynamicSmemBytes > 100 * 1024 ? 1 : 2) * n_sms : fit[k - 1];
    if (at_once < 1) continue;
    const double turns = (double)units / at_once;
    const double t = (7.3 + exchange[k] + tiles / (1 << k)) * (units << k > n_sms ? 1.5 : 1.0) *
                     (turns <= 1.0 ? 1.0 : turns <= 1.1 ? turns : ceil(turns));
    if (k == 0 || t < best) best = t, C = 1 << k;
  }
  attr[0].val.clusterDim.x = C;
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, tree_attention<D, FP16, WIDE>, mk_, mv, P);
}

static bool encode(CUtensorMap* map, const void* base, int fp16, int D, int max_seq, int hkv, int B, int64_t seq,
                   int64_t head, int64_t row) {
  auto fn = get_tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)max_seq, (cuuint64_t)hkv, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)row * 2, (cuuint64_t)head * 2, (cuuint64_t)seq * 2};
  cuuint32_t box[4] = {64, kKeys, 1, 1}, one[4] = {1, 1, 1, 1};
  return fn(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
            dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tree

int tree_attention(const mk_tree_shape& s, const void* q, const void* k, const void* v, void* o,
                   const int32_t* parents, const int32_t* n_nodes, const int32_t* lens, float scale, int n_sms,
                   cudaStream_t stream, std::string* err) {
  using namespace tree;
  Params P;
  P.q = q;
  P.v = static_cast<const uint16_t*>(v);
  P.o = o;
  P.parents = parents, P.n_nodes = n_nodes, P.lens = lens;
  P.q_seq = s.q_seq, P.q_node = s.q_node, P.q_head = s.q_head;
  P.o_seq = s.o_seq, P.o_node = s.o_node, P.o_head = s.o_head;
  P.v_seq = s.v_seq, P.v_head = s.v_head, P.v_row = s.v_row;
  P.n = s.n, P.hkv = s.n_kv_heads, P.G = s.n_q_heads / s.n_kv_heads, P.max_seq = s.max_seq;
  P.nt = kRows / P.G;
  P.inv_g = 65536u / P.G + 1;
  P.c = fabsf(scale) * 1.44269504088896340736f;
  P.negate = scale < 0.f ? 1u << 13 : 0u;
  P.timeout_ns = attention_wait_timeout_ns();
  P.drop_block = attention_drop_unit();
  const int fp16 = s.dtype == MK_FP16;
  CUtensorMap mk_, mv;
  if (!encode(&mk_, k, fp16, s.head_dim, s.max_seq, s.n_kv_heads, s.B, s.k_seq, s.k_head, s.k_row) ||
      !encode(&mv, v, fp16, s.head_dim, s.max_seq, s.n_kv_heads, s.B, s.v_seq, s.v_head, s.v_row)) {
    *err = "cuTensorMapEncodeTiled failed for the cache (strides of 2^40 bytes or more?)";
    return MK_ERR_INVALID_ARG;
  }
  cudaError_t e;
#define MK_LAUNCH(D, F) (s.wide ? launch<D, F, true>(mk_, mv, P, s.B, n_sms, stream) : launch<D, F, false>(mk_, mv, P, s.B, n_sms, stream))
  if (s.head_dim == 128)
    e = fp16 ? MK_LAUNCH(128, true) : MK_LAUNCH(128, false);
  else
    e = fp16 ? MK_LAUNCH(64, true) : MK_LAUNCH(64, false);
#undef MK_LAUNCH
  if (e != cudaSuccess) {
    *err = std::string("tree_attention launch: ") + cudaGetErrorString(e);
    return MK_ERR_CUDA;
  }
  return MK_OK;
}

int tree_attention_status(cudaStream_t stream, std::string* err) {
  cudaError_t e = cudaStreamSynchronize(stream);
  uint32_t word = 0;
  const uint32_t zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&word, tree::g_err, 4);
  if (e == cudaSuccess && word) e = cudaMemcpyToSymbol(tree::g_err, &zero, 4);
  if (e != cudaSuccess) {
    *err = std::string("reading the tree attention's error word: ") + cudaGetErrorString(e);
    return MK_ERR_CUDA;
  }
  if (word) {
    *err = "mk_tree_attention: a device wait timed out (its output is undefined)";
    return MK_ERR_DEVICE_TIMEOUT;
  }
  return MK_OK;
}

}  // namespace mk
