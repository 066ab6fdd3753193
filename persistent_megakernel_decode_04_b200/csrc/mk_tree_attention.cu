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
// Two streams of four softmax warps each keep the tensor cores and the loads fed: with one row
// tile the streams take alternate key tiles, each with its own running maximum, sum and O; with
// two row tiles (more than 128 rows) stream w is row tile w and every key tile serves both.
// The keys of a (sequence, KV head, row tiles) unit are split over a thread-block cluster, whose
// CTAs merge their partial results through distributed shared memory: no workspace, no atomics,
// a fixed order of summation.
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
#include <mutex>

#include "mk_internal.h"
#include "mk_ptx.cuh"

namespace mk {
namespace tree {

constexpr int kKeys = 128;        // keys per tile
constexpr int kRows = 128;        // rows per row tile
constexpr int kSoftWarps = 8;     // two streams of four
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 320;
constexpr int kMaxNodes = MK_MAX_TREE_NODES;
constexpr int kAncStride = kMaxNodes / 32 + 1;  // odd: rows fall on different banks
constexpr int kMaxCluster = 16;
constexpr uint32_t kTmemCols = 512;  // S0 S1 at 0, 128 (P over their first 64), O0 O1 at 256, 256 + D

template <int D>
struct Geo {
  static constexpr int kTile = kKeys * D * 2;      // bytes of a K, V or Q tile
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kOStride = D + 4;           // floats: 16-byte rows, no bank conflicts
  static constexpr int kData = 2 * kTile + kStages * kTile;
  // more than half of an SM's shared memory, so that one CTA runs per SM: a second one would
  // wait for TMEM columns while its cluster's other CTAs hold theirs
  static_assert(kData > 116 * 1024, "one CTA per SM");
  static_assert(2 * kRows * kOStride * 4 <= kData, "partial O fits over Q and the ring");
};

struct Params {
  const uint16_t* q;
  const uint16_t* v;
  uint16_t* o;
  const int32_t *parents, *n_nodes, *lens;
  int64_t q_seq, q_node, q_head, o_seq, o_node, o_head, v_seq, v_head, v_row;
  int n, hq, hkv, G, max_seq;
  int nt;        // nodes per row tile
  int mt, mp;    // row tiles, units of up to two row tiles
  float c;       // |scale| * log2(e)
  uint32_t flip; // sign bits flipped in q: scale < 0
  uint64_t timeout_ns;
  int drop_block;  // test hook: the block that issues no loads (-1: none)
};

struct Ctl {
  uint64_t full[8], empty[8], s_full[2], p_full[2], o_full[2], q_full, mma_done;
  uint32_t tmem, abort, bad_v, pad;
  float m[2][kRows], l[2][kRows];
  uint32_t anc[kMaxNodes * kAncStride];
  int16_t up[2][kMaxNodes];
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
__device__ __forceinline__ float ld_peer_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_peer_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_peer_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
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

// The position in load order of key tile j's K and V: K runs `ahead` tiles before V.
__device__ __forceinline__ int k_index(int j, int ahead) { return j < ahead ? j : 2 * j - ahead + 1; }
__device__ __forceinline__ int v_index(int j, int ahead, int T) { return j + min(T, j + ahead); }

template <int D, bool FP16>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attention(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ Params P) {
  using Ge = Geo<D>;
  extern __shared__ uint8_t raw[];
  __shared__ Ctl S;
  uint8_t* data = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  uint8_t* ring = data + 2 * Ge::kTile;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = (int)cluster_size(), rank = (int)cluster_rank();

  const int unit = blockIdx.x / C;
  const int pair = unit % P.mp, h = (unit / P.mp) % P.hkv, b = unit / P.mp / P.hkv;
  const int len = min(max(P.lens[b], 0), P.max_seq);
  const int nn = min(min(P.n_nodes ? max(P.n_nodes[b], 0) : P.n, P.n), P.max_seq - len);
  if (pair * 2 * P.nt >= nn) return;  // no node here (the whole cluster alike)
  const int tiles = min(2, P.mt - pair * 2) == 2 && (pair * 2 + 1) * P.nt < nn ? 2 : 1;
  const int total = len + nn, T_all = (total + kKeys - 1) / kKeys;
  const int t0 = (int)((int64_t)rank * T_all / C), T = (int)((int64_t)(rank + 1) * T_all / C) - t0;
  const int ahead = tiles == 2 ? 1 : 2;  // K tiles loaded before the first V tile

  if (tid == 0) {
    for (int i = 0; i < Ge::kStages; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], 4);
      mbar_init(&S.o_full[i], 1);
    }
    mbar_init(&S.q_full, kSoftWarps);
    mbar_init(&S.mma_done, 1);
    S.abort = 0;
    S.bad_v = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc_alloc(&S.tmem, kTmemCols);
    tc_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;

  if (warp == kTmaWarp) {
    // ---- loads: K and V tiles in the order in which the products consume them ----
    if (lane == 0) {
      int x = 0;  // loads issued
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
      bool ok = (int)blockIdx.x != P.drop_block;
      int k = 0;
      for (; ok && k < min(T, ahead); ++k) ok = load(&map_k, k);
      for (int v = 0; ok && v < T; ++v) {
        ok = load(&map_v, v);
        if (ok && k < T) ok = load(&map_k, k++);
      }
      if (*reinterpret_cast<volatile uint32_t*>(&S.abort))  // leave no copy in flight
        for (int y = max(0, x - Ge::kStages); y < x; ++y)
          wait_slow(&S.full[y % Ge::kStages], (y / Ge::kStages) & 1, P.timeout_ns, S, true);
    }
  } else if (warp == kMmaWarp) {
    // ---- products, in an order that keeps one stream's product beside the other's softmax ----
    if (lane == 0) {
      constexpr uint32_t type = FP16 ? 0u : 1u;
      constexpr uint32_t idesc = (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)(kRows >> 4) << 24);
      constexpr uint32_t idesc_s = idesc | ((uint32_t)(kKeys >> 3) << 17);
      constexpr uint32_t idesc_o = idesc | (1u << 16) | ((uint32_t)(D >> 3) << 17);  // V is MN-major
      const uint32_t q_base = smem_u32(data), ring_base = smem_u32(ring);
      const int n0 = tiles == 2 ? T : (T + 1) / 2, n1 = tiles == 2 ? T : T / 2;
      bool ok = T > 0 && wait(&S.q_full, 0, P, S);
      tc_fence_after();
      auto scores = [&](int w, int it) {  // S_w = Q K^T of the stream's it-th tile
        const int j = tiles == 2 ? it : 2 * it + w, x = k_index(j, ahead), stage = x % Ge::kStages;
        if (!wait(&S.full[stage], (x / Ge::kStages) & 1, P, S)) return false;
        tc_fence_after();
        const uint32_t a = q_base + (tiles == 2 ? w : 0) * Ge::kTile, bb = ring_base + stage * Ge::kTile;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t off = (s / 4) * kKeys * 128 + (s % 4) * 32;
          tc_mma_f16(tmem + w * kKeys, desc128(a + off, 16, 1024), desc128(bb + off, 16, 1024), idesc_s, s != 0);
        }
        tc_commit(&S.s_full[w]);
        if (tiles == 1 || w == 1) tc_commit(&S.empty[stage]);
        return true;
      };
      auto output = [&](int w, int it) {  // O_w += P_w V
        const int j = tiles == 2 ? it : 2 * it + w, x = v_index(j, ahead, T), stage = x % Ge::kStages;
        if (!wait(&S.full[stage], (x / Ge::kStages) & 1, P, S)) return false;
        if (!wait(&S.p_full[w], it & 1, P, S)) return false;
        // both streams have cleaned their halves of a tile that ends the sequence
        if (tiles == 2 && w == 0 && (t0 + j + 1) * kKeys > len && !wait(&S.p_full[1], it & 1, P, S)) return false;
        tc_fence_after();
        const uint32_t bb = ring_base + stage * Ge::kTile;
#pragma unroll
        for (int s = 0; s < kKeys / 16; ++s)
          mma_ts(tmem + 256 + w * D, tmem + w * kKeys + s * 8, desc128(bb + s * 2048, kKeys * 128, 1024), idesc_o,
                 it != 0 || s != 0);
        if (tiles == 1 || w == 1) tc_commit(&S.empty[stage]);
        return true;
      };
      if (ok) ok = scores(0, 0);
      if (ok && n1 > 0) ok = scores(1, 0);
      for (int it = 0; ok && it < n0; ++it) {
        ok = output(0, it);
        if (ok && it + 1 < n0) ok = scores(0, it + 1);
        if (ok && it + 1 == n0) tc_commit(&S.o_full[0]);
        if (ok && it < n1) {
          ok = output(1, it);
          if (ok && it + 1 < n1) ok = scores(1, it + 1);
          if (ok && it + 1 == n1) tc_commit(&S.o_full[1]);
        }
      }
      tc_commit(&S.mma_done);  // nothing in flight when TMEM is freed
      wait_slow(&S.mma_done, 0, P.timeout_ns, S, true);
    }
  } else {
    // ---- softmax: one thread per row ----
    const int w = warp >> 2, row = tid & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    // Q rows into the swizzled tiles: 16-byte piece c of row r goes to piece c ^ (r % 8)
    {
      const int pieces = D / 8;
      for (int x = tid; x < tiles * kRows * pieces; x += kSoftWarps * 32) {
        const int t = x / (kRows * pieces), r = (x / pieces) % kRows, c = x % pieces;
        const int node = (pair * 2 + t) * P.nt + r / P.G;
        uint4 val = make_uint4(0, 0, 0, 0);
        if (r < P.nt * P.G && node < nn) {
          val = *reinterpret_cast<const uint4*>(P.q + (int64_t)b * P.q_seq + (int64_t)node * P.q_node +
                                                (int64_t)(h * P.G + r % P.G) * P.q_head + c * 8);
          val.x ^= P.flip, val.y ^= P.flip, val.z ^= P.flip, val.w ^= P.flip;
        }
        *reinterpret_cast<uint4*>(data + t * Ge::kTile + (c / 8) * kRows * 128 + r * 128 +
                                  ((c & 7) ^ (r & 7)) * 16) = val;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.q_full);
    }
    // Ancestor bits of every node by doubling: in each round a node takes over the bits of the
    // node it points at and then points where that one points.
    {
      const int i = tid;  // 256 threads, kMaxNodes nodes
      int up = -1;
      bool live = i < nn;
      if (live) {
        up = P.parents[(int64_t)b * P.n + i];
        if (up < -1 || up >= i) live = false, up = -1;  // not a tree's: the node sees nothing
      }
#pragma unroll
      for (int k = 0; k < kMaxNodes / 32; ++k) S.anc[i * kAncStride + k] = live && (i >> 5) == k ? 1u << (i & 31) : 0u;
      S.up[0][i] = (int16_t)(live ? up : -2);
      named_bar_sync(1, kSoftWarps * 32);
      for (int rnd = 0;; ++rnd) {
        const int cur = S.up[rnd & 1][i];
        uint32_t add[kMaxNodes / 32];
        int nxt = cur;
        if (cur >= 0) {
          nxt = S.up[rnd & 1][cur];
#pragma unroll
          for (int k = 0; k < kMaxNodes / 32; ++k) add[k] = S.anc[cur * kAncStride + k];
        }
        // the barrier with a vote: also the end, once no node points at another
        int more;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
            "barrier.cta.red.or.pred q, 1, 256, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
            : "=r"(more)
            : "r"((int)(cur >= 0))
            : "memory");
        if (!more) break;
        if (cur >= 0) {
#pragma unroll
          for (int k = 0; k < kMaxNodes / 32; ++k)
            S.anc[i * kAncStride + k] = nxt == -2 ? 0u : S.anc[i * kAncStride + k] | add[k];
        }
        S.up[(rnd + 1) & 1][i] = (int16_t)nxt;
        named_bar_sync(1, kSoftWarps * 32);
      }
    }
    const int node = (pair * 2 + (tiles == 2 ? w : 0)) * P.nt + row / P.G;
    const bool real = row < P.nt * P.G && node < nn;
    const uint32_t* anc = S.anc + (real ? node : 0) * kAncStride;
    const bool dead = real && !(anc[node >> 5] >> (node & 31) & 1);  // its parents are not a tree's
    const int count = tiles == 2 ? T : w == 0 ? (T + 1) / 2 : T / 2;
    constexpr float kBias = FP16 ? 7.f : 0.f;
    float m = -INFINITY, l = 0.f;  // maximum that P is taken against; this row's sum of P
    for (int it = 0; it < count; ++it) {
      const int j = tiles == 2 ? it : 2 * it + w, key0 = (t0 + j) * kKeys;
      if (!wait_warp(&S.s_full[w], it & 1, P, S)) break;
      tc_fence_after();
      uint32_t s[kKeys];
#pragma unroll
      for (int k = 0; k < 4; ++k) tmem_ld32(lane_base + w * kKeys + k * 32, s + k * 32);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 4; ++k) tmem_use32(s + k * 32);
      const bool edge = key0 + kKeys > len;  // the tile has drafts, or rows behind the last one
      if (edge || dead) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t see = dead ? 0u : visible32(anc, key0 + k * 32 - len);
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (!(see >> x & 1)) s[k * 32 + x] = 0xff800000u;
        }
      }
      float mx[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) mx[k] = __uint_as_float(s[k]);
#pragma unroll
      for (int x = 4; x < kKeys; ++x) mx[x & 3] = fmaxf(mx[x & 3], __uint_as_float(s[x]));
      const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), m);
      const bool move = (top - m) * P.c > 8.f;  // also from -inf; false for -inf - -inf
      if (__any_sync(0xffffffffu, move)) {
        const float f = top == -INFINITY ? 1.f : ex2((m - top) * P.c);
        m = top;
        l *= f;
        if (it > 0) {
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            uint32_t o[32];
            tmem_ld32(lane_base + 256 + w * D + k * 32, o);
            tmem_wait_ld();
            tmem_use32(o);
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
            tmem_st32(lane_base + 256 + w * D + k * 32, o);
          }
        }
      }
      const float nm = m == -INFINITY ? 0.f : kBias - m * P.c;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t p[kKeys / 2];
#pragma unroll
      for (int x = 0; x < kKeys / 2; ++x) {
        const float a = ex2(fmaf(__uint_as_float(s[2 * x]), P.c, nm));
        const float e = ex2(fmaf(__uint_as_float(s[2 * x + 1]), P.c, nm));
        sum[(2 * x) & 3] += a;
        sum[(2 * x + 1) & 3] += e;
        p[x] = pack16<FP16>(a, e);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tmem_st32(lane_base + w * kKeys, p);
      tmem_st32(lane_base + w * kKeys + 32, p + 32);
      tmem_wait_st();
      if (edge) {
        // 0 x inf and 0 x NaN must not reach rows that do not see the key: rows behind the last
        // node become zero, and so do infinite and NaN values of drafts (their own descendants
        // get them back at the end).  The streams that use the tile share the work.
        const int x = v_index(j, ahead, T), stage = x % Ge::kStages;
        if (!wait_warp(&S.full[stage], (x / Ge::kStages) & 1, P, S)) break;
        uint4* tile = reinterpret_cast<uint4*>(ring + stage * Ge::kTile);
        const int part = tiles == 2 ? tid : row, step = tiles == 2 ? 256 : 128;
        for (int y = part; y < Ge::kTile / 16; y += step) {
          const int rel = key0 + (y / 8) % kKeys - len;  // 8 pieces of 16 bytes per key and half
          if (rel < 0) continue;
          uint4 val = make_uint4(0, 0, 0, 0);
          if (rel < nn) {
            val = tile[y];
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
          tile[y] = val;
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.p_full[w]);
    }
    // ---- this CTA's partial result: statistics, and O over Q's and the ring's room ----
    bool good = true;
    if (tiles == 2 || T > 0) good = count == 0 || wait_warp(&S.o_full[w], 0, P, S);
    if (T > 0 && (tiles == 2 || T > 1)) good = wait_warp(&S.o_full[w ^ 1], 0, P, S) && good;  // the ring is read out
    tc_fence_after();
    S.m[w][row] = m;
    S.l[w][row] = l;
    if (good && count > 0) {
      float* dst = reinterpret_cast<float*>(data) + (size_t)(w * kRows + row) * Ge::kOStride;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        uint32_t o[32];
        tmem_ld32(lane_base + 256 + w * D + k * 32, o);
        tmem_wait_ld();
        tmem_use32(o);
#pragma unroll
        for (int x = 0; x < 32; x += 4)
          *reinterpret_cast<uint4*>(dst + k * 32 + x) = make_uint4(o[x], o[x + 1], o[x + 2], o[x + 3]);
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  if (warp == kMmaWarp) tc_dealloc(tmem, kTmemCols);

  // ---- merge: this CTA finishes a share of the rows, D / 4 lanes per row ----
  if (warp < kSoftWarps) {
    constexpr int kLanes = D / 4, kPer = 32 / kLanes;  // rows per warp at a time
    const int first = pair * 2 * P.nt;
    const int rows = (min(nn, first + tiles * P.nt) - first) * P.G;
    const int per = (rows + C - 1) / C, r1 = min(rows, (rank + 1) * per);
    const int parts = tiles == 2 ? C : 2 * C;
    const int sub = lane / kLanes, col = (lane % kLanes) * 4;
    uint32_t bad = 0;
    for (int x = 0; x < C; ++x) bad |= ld_peer_u32(mapa(smem_u32(&S.bad_v), x));
    for (int base = rank * per + warp * kPer; base < r1; base += kSoftWarps * kPer) {
      const int r = base + sub;
      const bool on = r < r1;
      const int node = first + (on ? r : base) / P.G, g = (on ? r : base) % P.G;
      const int t = (node - first) / P.nt, lr = (node - first - t * P.nt) * P.G + g;  // row tile, row in it
      // lane x of the row's group looks after parts x, x + kLanes
      float mx = -INFINITY, pm[2], pl[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int part = lane % kLanes + y * kLanes;
        pm[y] = -INFINITY, pl[y] = 0.f;
        if (part < parts) {
          const int w = tiles == 2 ? t : part & 1, who = tiles == 2 ? part : part >> 1;
          pm[y] = ld_peer_f32(mapa(smem_u32(&S.m[w][lr]), who));
          pl[y] = ld_peer_f32(mapa(smem_u32(&S.l[w][lr]), who));
        }
        mx = fmaxf(mx, pm[y]);
      }
#pragma unroll
      for (int off = kLanes / 2; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      float f[2], sum = 0.f;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        // a part that saw no key has no O to read
        f[y] = pm[y] == -INFINITY && pl[y] == 0.f ? 0.f : mx == -INFINITY ? 1.f : ex2((pm[y] - mx) * P.c);
        sum += pl[y] * f[y];
      }
#pragma unroll
      for (int off = kLanes / 2; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      for (int p0 = 0; p0 < parts; p0 += 4) {
        float fp[4];
        float4 v[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {  // parts beyond the last have weight 0
          const int part = p0 + y;
          fp[y] = __shfl_sync(0xffffffffu, part < kLanes ? f[0] : f[1], part % kLanes, kLanes);
          const int w = tiles == 2 ? t : part & 1, who = tiles == 2 ? part : part >> 1;
          v[y] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (fp[y] != 0.f)
            v[y] = ld_peer_f4(
                mapa(smem_u32(reinterpret_cast<float*>(data) + (size_t)(w * kRows + lr) * Ge::kOStride + col), who));
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          acc[0] = fmaf(fp[y], v[y].x, acc[0]);
          acc[1] = fmaf(fp[y], v[y].y, acc[1]);
          acc[2] = fmaf(fp[y], v[y].z, acc[2]);
          acc[3] = fmaf(fp[y], v[y].w, acc[3]);
        }
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[x] *= inv;
      if (bad && on) {  // infinite and NaN values of drafts that the node sees
        for (int a = 0; a <= node; ++a) {
          if (!(S.anc[node * kAncStride + (a >> 5)] >> (a & 31) & 1)) continue;
          const uint16_t* src = P.v + (int64_t)b * P.v_seq + (int64_t)h * P.v_head + (int64_t)(len + a) * P.v_row + col;
          for (int x = 0; x < 4; ++x)
            if (nonfinite16<FP16>(src[x])) acc[x] += value16<FP16>(src[x]);
        }
      }
      if (on)
        *reinterpret_cast<uint2*>(P.o + (int64_t)b * P.o_seq + (int64_t)node * P.o_node +
                                  (int64_t)(h * P.G + g) * P.o_head + col) =
            make_uint2(pack16<FP16>(acc[0], acc[1]), pack16<FP16>(acc[2], acc[3]));
    }
  }
  __syncwarp();
  cluster_sync();  // peers read this CTA's shared memory until here
}

template <int D, bool FP16>
static cudaError_t launch(const CUtensorMap& mk_, const CUtensorMap& mv, const Params& P, int64_t units, int n_sms,
                          cudaStream_t stream) {
  constexpr int kSmem = Geo<D>::kData + 1024;
  // the largest cluster that fits the device, found once per device: 16, or the portable 8
  static std::atomic<int> largest[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int most = dev < 64 ? largest[dev].load() : 0;
  if (!most) {
    e = cudaFuncSetAttribute(tree_attention<D, FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(tree_attention<D, FP16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr[0].val.clusterDim.x = kMaxCluster;
    cfg.gridDim = dim3(kMaxCluster);
    int fit = 0;
    if (cudaOccupancyMaxActiveClusters(&fit, tree_attention<D, FP16>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      fit = 0;
    }
    most = fit >= 1 ? kMaxCluster : 8;
    if (dev < 64) largest[dev].store(most);
  }
  // Keys are split while that gives idle SMs work, down to one tile per block.
  int C = 1;
  while (2 * C <= most && units * 2 * C <= n_sms && (int64_t)C * kKeys < P.max_seq) C *= 2;
  if (units * C > 0x7fffffff) return cudaErrorInvalidValue;
  attr[0].val.clusterDim.x = C;
  cfg.gridDim = dim3((unsigned)(units * C));
  return cudaLaunchKernelEx(&cfg, tree_attention<D, FP16>, mk_, mv, P);
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
  P.mt = (s.n + P.nt - 1) / P.nt;
  P.mp = (P.mt + 1) / 2;
  P.c = fabsf(scale) * 1.44269504088896340736f;
  P.flip = scale < 0.f ? 0x80008000u : 0u;
  P.timeout_ns = attention_wait_timeout_ns();
  P.drop_block = attention_drop_unit();
  const int fp16 = s.dtype == MK_FP16;
  CUtensorMap mk_, mv;
  if (!encode(&mk_, k, fp16, s.head_dim, s.max_seq, s.n_kv_heads, s.B, s.k_seq, s.k_head, s.k_row) ||
      !encode(&mv, v, fp16, s.head_dim, s.max_seq, s.n_kv_heads, s.B, s.v_seq, s.v_head, s.v_row)) {
    *err = "cuTensorMapEncodeTiled failed for the cache (strides of 2^40 bytes or more?)";
    return MK_ERR_INVALID_ARG;
  }
  const int64_t units = (int64_t)s.B * s.n_kv_heads * P.mp;
  cudaError_t e;
  if (s.head_dim == 128)
    e = fp16 ? launch<128, true>(mk_, mv, P, units, n_sms, stream) : launch<128, false>(mk_, mv, P, units, n_sms, stream);
  else
    e = fp16 ? launch<64, true>(mk_, mv, P, units, n_sms, stream) : launch<64, false>(mk_, mv, P, units, n_sms, stream);
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
