// mk_tree_attention.cu -- attention of a tree of drafted tokens over a KV cache.
//
// Formula.  Sequence b has len rows in the cache and nn drafted nodes behind them, node i at row
// len + i; A(i) is node i with its ancestors.  For query head h of node i (KV head h / G):
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j),  j in {0..len-1} + {len + a : a in A(i)}.
//
// Mapping.  The G query heads of a KV head and the nodes share their keys, so they are the rows
// of one matrix product: a row tile is 128 rows (floor(128 / G) nodes x G heads) and both
// products run on the tensor cores (M = 128, fp32 accumulators in TMEM): S = Q K^T over 128-key
// tiles, O += P V with P as the TMEM operand.  K tiles are K-major, V tiles MN-major, both as
// TMA writes them with the 128-byte swizzle.  128 rows cost the same as 1: a 128-key tile takes
// the tensor cores 2 x 0.13 us, while its 64 KB take an SM's share of HBM 1.4 us.
//
// A block holds one row tile (two blocks per SM, so that one block's start, end and softmax run
// beside the other's loads and products) or, for more than 128 rows, two row tiles that share
// every key tile (one block per SM: half the reads from L2).  Each row tile has four softmax
// warps; one warp issues the loads, one the products, and two helpers prepare the tree: the
// ancestor bits of every node, and V tiles that end the sequence.
//
// The keys of a (sequence, KV head, row tiles) unit are split over a thread-block cluster, whose
// blocks merge their partial results through distributed shared memory: no workspace, no
// atomics, a fixed order of summation.
//
// Precision.  S, the softmax statistics and O are fp32.  P is rounded to the inputs' 16-bit type
// for the second product (relative 2^-9 / 2^-12, the size of the output's own rounding).  The
// maximum that P is taken against is only moved when it grows by more than 2^8; fp16 takes P
// times 2^7, so that small weights stay clear of fp16's subnormals (largest 2^15).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <atomic>

#include "mk_internal.h"
#include "mk_ptx.cuh"

namespace mk {
namespace tree {

constexpr int kKeys = 128;        // keys per tile
constexpr int kRows = 128;        // rows per row tile
constexpr int kMaxNodes = MK_MAX_TREE_NODES;
constexpr int kAncStride = kMaxNodes / 32 + 1;  // odd: rows fall on different banks
constexpr int kMaxCluster = 16;
constexpr int kCh = 32;            // keys of a row of S in registers at a time

// NT: row tiles of a block (1 or 2).
template <int D, int NT>
struct Geo {
  static constexpr int kSoft = 8 * NT;             // softmax warps; then loads, products, two helpers
  static constexpr int kThreads = (kSoft + 4) * 32;
  static constexpr int kTile = kKeys * D * 2;      // bytes of a K, V or Q tile
  static constexpr int kStages = (NT == 1 ? 2 : 4) * (128 / D) + (NT == 1 && D == 64 ? 1 : 0);
  static constexpr int kOStride = D + 4;           // floats: 16-byte rows, no bank conflicts
  static constexpr int kData = (NT + kStages) * kTile;
  // Tensor memory: S_w at w * 128 (P over it: keys 0..63 at 0, 64..127 at 64), O_w at NT * 128 + w * D
  static constexpr uint32_t kCols = NT * 256;
  // Shared memory bounds the blocks per SM to 512 / kCols: one more would wait for tensor memory
  // while its cluster's other blocks hold theirs.
  static_assert(NT == 1 ? kData > 76 * 1024 : kData > 116 * 1024, "blocks per SM");
  static_assert(NT * kRows * kOStride * 4 <= kData, "partial O fits over Q and the ring");
};

struct Params {
  const uint16_t* q;
  const uint16_t* v;
  uint16_t* o;
  const int32_t *parents, *n_nodes, *lens;
  int64_t q_seq, q_node, q_head, o_seq, o_node, o_head, v_seq, v_head, v_row;
  int n, hq, hkv, G, max_seq;
  int nt;        // nodes per row tile
  int units;     // blocks' worth of row tiles per (sequence, KV head)
  uint32_t inv_g;  // r / G = r * inv_g >> 16 for r < 256
  float c;       // |scale| * log2(e)
  uint32_t negate; // scale < 0: the product takes -Q (a bit of the instruction descriptor)
  uint64_t timeout_ns;
  int drop_block;  // test hook: the block that issues no loads (-1: none)
};

struct Ctl {
  uint64_t full[8], empty[8], s_full[2], p_full[2], o_full, q_full, mma_done, anc_full;
  uint32_t tmem, abort;
  uint32_t bad_v;  // infinite or NaN values among the drafts that this block saw
  // Counters that only grow, for roles that may be more than one step apart (an mbarrier's parity
  // cannot tell two steps from none): V tiles to clean that were issued; helpers' shares done.
  uint32_t v_issued, v_clean;
  uint32_t bad_any;  // some block of the cluster has bad_v set
  float pair[2][2][2 * kRows];  // what the two threads of a row tell each other, by turns
  // (maximum, sum) of every row that this block finishes from every block of the cluster
  float2 stat[2 * kRows + kMaxCluster];
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
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15};" ::MK_I8(r, 0), MK_I8(r, 8), "r"(taddr)
      : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_st_n(uint32_t taddr, const uint32_t* r) {
  if constexpr (N == 16)
    tmem_st16(taddr, r);
  else
    tmem_st32(taddr, r);
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

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

// Whether a 16-bit value is infinite or NaN; its value.
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

// Address of a peer CTA's shared memory, and loads from there.
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_peer_u32(uint32_t addr, uint32_t x) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ void st_peer_f2(uint32_t addr, float x, float y) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ float4 ld_peer_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
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

// Infinite and NaN values of drafts that the node sees, added to n output values at `out`.
template <bool FP16>
__device__ __noinline__ void add_nonfinite(const Params& P, const Ctl& S, int b, int h, int len, int node, int col,
                                           int n, uint16_t* out) {
  if (!alive(S, node)) return;
  for (int a = 0; a <= node; ++a) {
    if (!(S.anc[node * kAncStride + (a >> 5)] >> (a & 31) & 1)) continue;
    const uint16_t* val = P.v + (int64_t)b * P.v_seq + (int64_t)h * P.v_head + (int64_t)(len + a) * P.v_row + col;
    for (int x = 0; x < n; ++x)
      if (nonfinite16<FP16>(val[x]))
        out[x] = (uint16_t)pack16<FP16>(value16<FP16>(out[x]) + value16<FP16>(val[x]), 0.f);
  }
}

// Output rows that this block finishes: row r's partial results, weighted, from the C blocks.
// The loops are kept rolled: this runs once, and its instructions come from memory.
template <int D, bool FP16, int NT>
__device__ __forceinline__ void merge(const Params& P, const Ctl& S, const uint8_t* data, int b, int h, int first,
                                      int rows, int per, int rank, int C, int len, int warp, int lane) {
  using Ge = Geo<D, NT>;
  constexpr int kLanes = D / 4, kPer = 32 / kLanes;  // lanes per row, rows per warp side by side
  const int sub = lane / kLanes, in = lane % kLanes, col = in * 4;
  const int r0 = rank * per, r1 = min(rows, r0 + per), tile_rows = P.nt * P.G;
  if (r0 >= r1) return;
#pragma unroll 1
  for (int base = r0 + warp * kPer; base < r1; base += Ge::kThreads / 32 * kPer) {
    const int r = min(base + sub, r1 - 1);
    // lane p of the row's group holds part p's weight (C <= 16 <= kLanes)
    const float2 st = S.stat[(r - r0) * C + (in & (C - 1))];
    float mx = st.x;
    for (int off = C / 2; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    // a part that saw no key has no O to read
    float f = st.x == -INFINITY && st.y == 0.f ? 0.f : mx == -INFINITY ? 1.f : ex2((st.x - mx) * P.c);
    float sum = st.y * f;
    for (int off = C / 2; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const int t = NT == 2 && r >= tile_rows, lr = r - t * tile_rows;
    const int local = (int)(lr * P.inv_g >> 16), g = lr - local * P.G, node = first + t * P.nt + local;
    f = sum == 0.f || !alive(S, node) ? 0.f : __fdividef(f, sum);
    const uint32_t src = smem_u32(data) + (uint32_t)(((t * kRows + lr) * Ge::kOStride + col) * 4);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int p0 = 0; p0 < C; p0 += 8) {
      float fp[8];
      float4 v[8];
#pragma unroll
      for (int p = 0; p < 8; ++p) {  // eight loads in flight
        fp[p] = __shfl_sync(0xffffffffu, f, p0 + p, kLanes);
        v[p] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p0 + p >= C) fp[p] = 0.f;
        if (fp[p] != 0.f) v[p] = ld_peer_f4(mapa(src, p0 + p));
      }
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        acc[0] = fmaf(fp[p], v[p].x, acc[0]);
        acc[1] = fmaf(fp[p], v[p].y, acc[1]);
        acc[2] = fmaf(fp[p], v[p].z, acc[2]);
        acc[3] = fmaf(fp[p], v[p].w, acc[3]);
      }
    }
    if (base + sub >= r1) continue;
    uint16_t* out = P.o + (int64_t)b * P.o_seq + (int64_t)node * P.o_node + (int64_t)(h * P.G + g) * P.o_head + col;
    *reinterpret_cast<uint2*>(out) = make_uint2(pack16<FP16>(acc[0], acc[1]), pack16<FP16>(acc[2], acc[3]));
    if (S.bad_any) add_nonfinite<FP16>(P, S, b, h, len, node, col, 4, out);
  }
}

template <int D, bool FP16, int NT>
__global__ void __launch_bounds__(Geo<D, NT>::kThreads, 3 - NT)
    tree_attention(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ Params P) {
  using Ge = Geo<D, NT>;
  extern __shared__ uint8_t raw[];
  __shared__ Ctl S;
  constexpr int kTmaWarp = Ge::kSoft, kMmaWarp = Ge::kSoft + 1, kHelper = Ge::kSoft + 2;
  uint8_t* data = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  uint8_t* ring = data + NT * Ge::kTile;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = (int)cluster_size(), rank = (int)cluster_rank();

  const int unit = blockIdx.x / C, head = unit / P.units;
  const int b = head / P.hkv, h = head - b * P.hkv;
  const int first = (unit - head * P.units) * NT * P.nt;  // first node of the block's row tiles
  int len = P.lens[b], nn = P.n_nodes ? P.n_nodes[b] : P.n;
  // softmax warps: row tile, row, and which half of a tile's keys (and of O's columns) of that row
  const int w = warp >> 3, row = tid & 127, half = (warp >> 2) & 1;
  const int local = (int)(row * P.inv_g >> 16);

  // ---- start: whatever does not need the lengths first ----
  int parent = -1;
  if (warp == kTmaWarp) {
    if (lane == 0) {
#pragma unroll 1
      for (int i = 0; i < Ge::kStages; ++i) {
        mbar_init(&S.full[i], 1);
        mbar_init(&S.empty[i], 1);
      }
#pragma unroll 1
      for (int i = 0; i < NT; ++i) {
        mbar_init(&S.s_full[i], 1);
        mbar_init(&S.p_full[i], 8);
      }
      mbar_init(&S.o_full, 1);
      mbar_init(&S.q_full, Ge::kSoft);
      mbar_init(&S.mma_done, 1);
      mbar_init(&S.anc_full, 1);
      S.abort = S.bad_v = S.bad_any = S.v_issued = S.v_clean = 0;
      fence_mbar_init();
    }
  } else if (warp == kMmaWarp) {
    tc_alloc(&S.tmem, Ge::kCols);
    tc_relinquish();
  } else if (warp == kHelper) {
    if (lane < P.n) parent = P.parents[(int64_t)b * P.n + lane];
  } else if (warp < Ge::kSoft) {
    // Q rows into the swizzled tile: 16-byte piece c of row r goes to piece c ^ (r % 8).  Rows of
    // the tile without a node keep what is there: they only reach their own, unused, results.
    const int x0 = tid & 255, c = x0 % (D / 8), used = min(P.nt, P.n - first - w * P.nt) * P.G;
    const uint16_t* src = P.q + (int64_t)b * P.q_seq + (int64_t)(first + w * P.nt) * P.q_node +
                          (int64_t)h * P.G * P.q_head + c * 8;
    const uint32_t dst = smem_u32(data) + w * Ge::kTile + (c / 8) * kRows * 128;
#pragma unroll 1
    for (int r = x0 / (D / 8); r < used; r += 2 * kRows / (D / 8)) {
      const int lr = (int)(r * P.inv_g >> 16);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + r * 128 + ((c & 7) ^ (r & 7)) * 16),
                   "l"(src + (int64_t)lr * P.q_node + (int64_t)(r - lr * P.G) * P.q_head)
                   : "memory");
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (C > 1) cluster_arrive();  // every block of the cluster has started: waited for before the first access
  const uint32_t tmem = S.tmem;

  len = min(max(len, 0), P.max_seq), nn = min(min(max(nn, 0), P.n), P.max_seq - len);
  const bool on = first < nn;                      // else there is no node here (the whole cluster alike)
  const bool two = NT == 2 && first + P.nt < nn;   // the second row tile has nodes
  const int T_all = on ? (len + nn + kKeys - 1) / kKeys : 0;
  const int t0 = rank * T_all / C, T = (rank + 1) * T_all / C - t0;
  const int edge = max(0, len / kKeys - t0);  // first tile of this block that has rows behind len
  const int rows = min(nn - first, NT * P.nt) * P.G, per = (rows + C - 1) / C;  // rows; of these to finish

  if (warp == kTmaWarp) {
    // ---- loads: K and V of a tile in turn ----
    if (lane == 0 && (int)blockIdx.x != P.drop_block) {
      int x = 0;
#pragma unroll 1
      for (; x < 2 * T; ++x) {
        const int stage = x % Ge::kStages, use = x / Ge::kStages;
        if (use > 0 && !wait(&S.empty[stage], (use - 1) & 1, P, S)) break;
        mbar_arrive_expect_tx(&S.full[stage], Ge::kTile);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_4d(ring + stage * Ge::kTile + c * kKeys * 128, x & 1 ? &map_v : &map_k, c * 64, (t0 + (x >> 1)) * kKeys,
                 h, b, &S.full[stage]);
        if ((x & 1) && (x >> 1) >= edge) count_up(&S.v_issued);
      }
      if (x < 2 * T)  // given up: leave no copy in flight
        for (int y = max(0, x - Ge::kStages); y < x; ++y)
          wait_slow(&S.full[y % Ge::kStages], (y / Ge::kStages) & 1, P.timeout_ns, S, true);
    }
  } else if (warp == kMmaWarp) {
    // ---- products: one row tile's beside the other's (or the other block's) softmax ----
    if (lane == 0 && T > 0) {
      constexpr uint32_t type = FP16 ? 0u : 1u;
      constexpr uint32_t idesc = (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)(kRows >> 4) << 24);
      const uint32_t idesc_s = idesc | P.negate | ((uint32_t)(kKeys >> 3) << 17);
      constexpr uint32_t idesc_o = idesc | (1u << 16) | ((uint32_t)(D >> 3) << 17);  // V is MN-major
      const uint32_t q_base = smem_u32(data), ring_base = smem_u32(ring);
      const int last = two ? 1 : 0;
      bool ok = wait(&S.q_full, 0, P, S);
      tc_fence_after();
      // step y = -1 .. T - 1, for each row tile t: O_t += P_t V of tile y, then S_t = Q_t K^T of tile y + 1
#pragma unroll 1
      for (int y = -last - 1; ok && y < (last + 1) * T; ++y) {
        const int t = (y + last + 1) & last, j = last ? y >> 1 : y;
        if (j >= 0) {
          const int x = 2 * j + 1, stage = x % Ge::kStages;
          ok = wait(&S.full[stage], (x / Ge::kStages) & 1, P, S) &&
               (j < edge || wait_count(&S.v_clean, 2 * (j - edge + 1), P, S)) && wait(&S.p_full[t], j & 1, P, S);
          if (!ok) break;
          tc_fence_after();
          const uint32_t bb = ring_base + stage * Ge::kTile;
#pragma unroll
          for (int s = 0; s < kKeys / 16; ++s)
            mma_ts(tmem + NT * kKeys + t * D, tmem + t * kKeys + (s & 4) * 16 + (s & 3) * 8, desc128(bb + s * 2048, kKeys * 128, 1024),
                   idesc_o, j != 0 || s != 0);
          if (t == last) tc_commit(&S.empty[stage]);
        }
        if (j + 1 < T) {
          const int x = 2 * j + 2, stage = x % Ge::kStages;
          ok = wait(&S.full[stage], (x / Ge::kStages) & 1, P, S);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = q_base + t * Ge::kTile, bb = ring_base + stage * Ge::kTile;
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t off = (s / 4) * kKeys * 128 + (s % 4) * 32;
            tc_mma_f16(tmem + t * kKeys, desc128(a + off, 16, 1024), desc128(bb + off, 16, 1024), idesc_s, s != 0);
          }
          tc_commit(&S.s_full[t]);
          if (t == last) tc_commit(&S.empty[stage]);
        }
      }
      if (ok) tc_commit(&S.o_full);
      tc_commit(&S.mma_done);  // nothing in flight when TMEM is freed
      wait_slow(&S.mma_done, 0, P.timeout_ns, S, true);
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
      const int x = 2 * j + 1, stage = x % Ge::kStages;
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
      if (lane == 0) count_up(&S.v_clean);
    }
  } else {
    // ---- softmax: two threads per row, one for each half of a tile's keys ----
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.q_full);
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_at = lane_base + w * kKeys + half * 64, o_at = lane_base + NT * kKeys + w * D + half * (D / 2);
    const int node = first + w * P.nt + local;
    const bool real = local < P.nt && node < nn;
    const bool any = __any_sync(0xffffffffu, real);  // else the warp's rows are left alone (their P is garbage)
    const uint32_t* anc = S.anc + (real ? node : 0) * kAncStride;
    const int count = w == 0 || two ? T : 0;
    // the row's other thread: tell it x, get its x (turn: a slot is written again two turns later)
    auto tell = [&](float x, int turn) {
      S.pair[turn & 1][half][w * kRows + row] = x;
      named_bar_sync(1 + w * 4 + (warp & 3), 64);
      return S.pair[turn & 1][half ^ 1][w * kRows + row];
    };
    constexpr float kBias = FP16 ? 7.f : 0.f;
    float m = -INFINITY, l = 0.f;  // maximum that P is taken against; sum of P over this thread's keys
    bool ok = count == 0 || edge >= T || wait_warp(&S.anc_full, 0, P, S);
#pragma unroll 1
    for (int j = 0; j < count; ++j) {
      ok = ok && wait_warp(&S.s_full[w], j & 1, P, S);
      tc_fence_after();
      if (any) {
        // a row of S is read twice, kCh keys at a time: for the maximum, and for the weights
        const int rel = (t0 + j) * kKeys + half * 64 - len;  // > -64: drafts, or rows behind the last one
        auto scores = [&](int k, uint32_t* s) {
          tmem_ld32(s_at + k * kCh, s);
          tmem_wait_ld();
          tmem_use32(s);
          if (rel + k * kCh > -kCh) {
            const uint32_t see = visible32(anc, rel + k * kCh);
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!(see >> x & 1)) s[x] = 0xff800000u;
          }
        };
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
        for (int k = 0; k < 64 / kCh; ++k) {
          uint32_t s[kCh];
          scores(k, s);
#pragma unroll
          for (int x = 0; x < kCh; x += 4) {
            mx[0] = fmaxf(mx[0], fmaxf(__uint_as_float(s[x]), __uint_as_float(s[x + 1])));
            mx[1] = fmaxf(mx[1], fmaxf(__uint_as_float(s[x + 2]), __uint_as_float(s[x + 3])));
          }
        }
        const float mine = fmaxf(mx[0], mx[1]);
        const float top = fmaxf(fmaxf(mine, tell(mine, j)), m);
        const bool move = real && (top - m) * P.c > 8.f;  // also from -inf; false for -inf - -inf
        if (__any_sync(0xffffffffu, move)) {
          const float f = top == -INFINITY ? 1.f : ex2((m - top) * P.c);
          m = top;
          l *= f;
          if (j > 0) {
#pragma unroll 1
            for (int k = 0; k < D / 64; ++k) {
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
        float sum[2] = {0.f, 0.f};
#pragma unroll 1
        for (int k = 0; k < 64 / kCh; ++k) {
          uint32_t s[kCh], p[kCh / 2];
          scores(k, s);
#pragma unroll
          for (int x = 0; x < kCh / 2; ++x) {
            float a0 = nm, a1 = nm;
            fma2(a0, a1, __uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1]), P.c, P.c);
            a0 = ex2(a0), a1 = ex2(a1);
            sum[0] += a0;
            sum[1] += a1;
            p[x] = pack16<FP16>(a0, a1);
          }
          tmem_st16(s_at + k * (kCh / 2), p);  // over scores that this thread has read
        }
        l += sum[0] + sum[1];
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.p_full[w]);
    }
    // ---- the end: every product is done, Q and the ring are read out ----
    if (T > 0) ok = ok && wait_warp(&S.o_full, 0, P, S);
    tc_fence_after();
    if (C > 1) cluster_wait();
    if (any) {
      l += tell(l, count);
      if (C == 1) {
        if (ok) ok = wait_warp(&S.anc_full, 0, P, S);
        const float inv = l == 0.f || !real || !alive(S, node) ? 0.f : 1.f / l;
        uint16_t* out = P.o + (int64_t)b * P.o_seq + (int64_t)node * P.o_node +
                        (int64_t)(h * P.G + row - local * P.G) * P.o_head + half * (D / 2);
#pragma unroll 1
        for (int k = 0; k < D / 64; ++k) {
          uint32_t o[32];
          tmem_ld32(o_at + k * 32, o);
          tmem_wait_ld();
          tmem_use32(o);
          if (real)
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
              uint32_t p[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float f0 = __uint_as_float(o[x + 2 * y]), f1 = __uint_as_float(o[x + 2 * y + 1]);
                p[y] = inv == 0.f ? 0u : pack16<FP16>(f0 * inv, f1 * inv);
              }
              *reinterpret_cast<uint4*>(out + k * 32 + x) = make_uint4(p[0], p[1], p[2], p[3]);
            }
        }
        if (S.bad_v && real) add_nonfinite<FP16>(P, S, b, h, len, node, half * (D / 2), D / 2, out);
      } else {
        // this block's partial result: O over Q's and the ring's room, and each row's statistics to
        // the block that finishes the row
        if (real && half == 0) {
          const int r = w * P.nt * P.G + row, owner = r / per;
          st_peer_f2(mapa(smem_u32(&S.stat[(r - owner * per) * C + rank]), owner), m, l);
          if (S.bad_v) st_peer_u32(mapa(smem_u32(&S.bad_any), owner), 1);
        }
        if (count > 0) {
          float* dst = reinterpret_cast<float*>(data) + (size_t)(w * kRows + row) * Ge::kOStride + half * (D / 2);
#pragma unroll 1
          for (int k = 0; k < D / 64; ++k) {
            uint32_t o[32];
            tmem_ld32(o_at + k * 32, o);
            tmem_wait_ld();
            tmem_use32(o);
            if (real)
#pragma unroll
              for (int x = 0; x < 32; x += 4)
                *reinterpret_cast<uint4*>(dst + k * 32 + x) = make_uint4(o[x], o[x + 1], o[x + 2], o[x + 3]);
          }
        }
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  if (C > 1) {
    if (warp >= Ge::kSoft) cluster_wait();
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  tc_fence_after();
  if (warp == kMmaWarp) tc_dealloc(tmem, Ge::kCols);
  if (C > 1) {
    if (on) merge<D, FP16, NT>(P, S, data, b, h, first, rows, per, rank, C, len, warp, lane);
    __syncwarp();
    cluster_arrive();  // peers read this block's shared memory until here
    cluster_wait();
  }
}

template <int D, bool FP16, int NT>
static cudaError_t launch(const CUtensorMap& mk_, const CUtensorMap& mv, const Params& P, int64_t units, int n_sms,
                          cudaStream_t stream) {
  constexpr int kSmem = Geo<D, NT>::kData + 1024;
  const auto kernel = tree_attention<D, FP16, NT>;
  // the largest cluster that fits the device, found once per device: 16, or the portable 8
  static std::atomic<int> largest[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(Geo<D, NT>::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int most = dev < 64 ? largest[dev].load() : 0;
  if (!most) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr[0].val.clusterDim.x = kMaxCluster;
    cfg.gridDim = dim3(kMaxCluster);
    int fit = 0;
    if (cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      fit = 0;
    }
    most = fit >= 1 ? kMaxCluster : 8;
    if (dev < 64) largest[dev].store(most);
  }
  // Keys are split while that gives idle SMs work, down to one tile per block.
  int C = 1;
  while (2 * C <= most && units * 2 * C <= n_sms && (int64_t)C * kKeys < P.max_seq) C *= 2;
  attr[0].val.clusterDim.x = C;
  cfg.gridDim = dim3((unsigned)(units * C));
  return cudaLaunchKernelEx(&cfg, kernel, mk_, mv, P);
}

template <int D, bool FP16>
static cudaError_t launch(const CUtensorMap& mk_, const CUtensorMap& mv, Params& P, int B, int n_sms,
                          cudaStream_t stream) {
  const int tiles = (P.n + P.nt - 1) / P.nt, NT = tiles > 1 ? 2 : 1;
  P.units = (tiles + NT - 1) / NT;
  const int64_t units = (int64_t)B * P.hkv * P.units;
  if (units > 0x7fffffff) return cudaErrorInvalidValue;
  return NT == 2 ? launch<D, FP16, 2>(mk_, mv, P, units, n_sms, stream)
                 : launch<D, FP16, 1>(mk_, mv, P, units, n_sms, stream);
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
  P.q = static_cast<const uint16_t*>(q);
  P.v = static_cast<const uint16_t*>(v);
  P.o = static_cast<uint16_t*>(o);
  P.parents = parents, P.n_nodes = n_nodes, P.lens = lens;
  P.q_seq = s.q_seq, P.q_node = s.q_node, P.q_head = s.q_head;
  P.o_seq = s.o_seq, P.o_node = s.o_node, P.o_head = s.o_head;
  P.v_seq = s.v_seq, P.v_head = s.v_head, P.v_row = s.v_row;
  P.n = s.n, P.hq = s.n_q_heads, P.hkv = s.n_kv_heads, P.G = s.n_q_heads / s.n_kv_heads, P.max_seq = s.max_seq;
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
  if (s.head_dim == 128)
    e = fp16 ? launch<128, true>(mk_, mv, P, s.B, n_sms, stream) : launch<128, false>(mk_, mv, P, s.B, n_sms, stream);
  else
    e = fp16 ? launch<64, true>(mk_, mv, P, s.B, n_sms, stream) : launch<64, false>(mk_, mv, P, s.B, n_sms, stream);
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
