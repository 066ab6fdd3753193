// mk_tree_verify.cu -- which drafted tokens the target's probabilities accept, and the next token.
//
// Rule (rejection sampling, node by node).  p_i, q_i: softmax of the target's / the draft's logits
// after node i over its temperature.  From node 0 with P = p_0: the children c of the current node
// are asked in index order; c is accepted if u_c q(x_c) < P(x_c), then it is the current node with
// P = p_c; else P becomes max(P - q, 0), scaled to sum 1.  Without draft logits a child was drafted
// for certain: q is 1 at its token.  When no child is accepted the next token is the first one
// whose cumulative P exceeds r.  Its law is p's whatever q is.  Temperature 0: P is 1 at the
// largest logit's lowest index.
//
// Two kernels.  row_stats reads every logit once and leaves, per row and chunk, the maximum, its
// index (at temperature 0) and the sum of exponentials (the other kernel's reads come from L2).
// walk, a thread-block cluster per sequence, goes down the tree with scalars only; where a whole
// row is needed (the rest after a rejected sampled draft, the final draw) the cluster's blocks
// take a slice each and exchange one partial sum through distributed shared memory.
//
// Bound: the walk's latency.  A pass over a row of 128255 words by 8 blocks takes 6 to 9 us, a third
// of it exchange and control, the rest fp64 arithmetic at half its rate (16 blocks: 4 to 5).  16
// sequences x 9 nodes of that size (bf16, sampled drafts) take 52 to 65 us by their drafts, of which
// row_stats 15 and the longest walk nearly all the rest; one chain of 5 (fp32, 128256 words) 17 us; 4 x 26
// nodes of 65536 words without a draft 20 us.  At temperature 0 no pass is left: 25, 7.5 and 14.5 us.
//
// Precision.  A draw from 1e5 words by cumulative sums meets a border within 1e-7 in about every
// hundredth draw, so sums that decide a draw are formed in fp64 from exponentials good to 1e-13.
// Acceptance compares two numbers, each with one row's fp32 sum in it: those decide unless the two
// are within kClose; then the rows' sums are formed in fp64 first.  A sum is off by less than 9e-6
// relative: 2^-22 for each of at most 13 exponentials in a row (a value's own and what takes it to
// higher maxima) and 2^-24 for the product with each, 2^-24 for each of at most 40 additions in a row,
// and 2.5e-6 from the exponents: the difference, the product and log2(e) / temperature are rounded
// four times, which moves a value by 4 x 2^-24 ln 2 of its exponent, whose mean over the sum's weights is
// at most 15.2 (2^20 words).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "mk_internal.h"
#include "mk_ptx.cuh"

namespace mk {
namespace verify {

constexpr int kMaxNodes = MK_MAX_TREE_NODES;
constexpr int kStatThreads = 256;
constexpr int kChunk = 8192;        // elements of a row per block of row_stats
constexpr int kThreads = 512;       // walk
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr float kClose = 2e-5f;     // two sums' errors
// elements per thread and step of a pass: eight keep more exponentials in flight; without a draft
// four need few enough registers for row_stats's blocks beside the walk's
template <bool DRAFT>
constexpr int kPerOf = DRAFT ? 8 : 4;
constexpr int kMaxDyn = 204 * 1024;  // walk: dynamic shared memory, beside 21 KB of Ctl

struct Stat {  // of one row's chunk
  float m, s;
  int idx, pad;
};

struct Params {
  const void *target, *draft;
  int64_t t_seq, t_node, d_seq, d_node;
  const int32_t *tokens, *parents, *n_nodes;
  const float *u, *r, *temperature, *draft_temperature;
  int32_t *path, *n_path, *next_token;
  Stat* stats;  // [target | draft][B][n][chunks]
  int B, n, V, chunks;
  // walk: whether a pass keeps what it has of P in shared memory, and of how many of its steps the
  // draft's exponentials
  int keep, q_steps;
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

// -infinity; the largest of a 16-byte piece (NaN left out); its values.
template <typename T>
__device__ __forceinline__ T lowest();
template <>
__device__ __forceinline__ float lowest<float>() { return -INFINITY; }
template <>
__device__ __forceinline__ __nv_bfloat16 lowest<__nv_bfloat16>() { return __ushort_as_bfloat16(0xff80); }
template <>
__device__ __forceinline__ __half lowest<__half>() { return __ushort_as_half(0xfc00); }

template <typename T>
__device__ __forceinline__ void floats_of(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 4) {
      x[k] = __uint_as_float(w[k]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      x[2 * k] = bf16lo(w[k]), x[2 * k + 1] = bf16hi(w[k]);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
      x[2 * k] = f.x, x[2 * k + 1] = f.y;
    }
  }
}
template <typename T>
__device__ __forceinline__ float max_of(const uint4& v) {
  if constexpr (sizeof(T) == 4) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  } else {
    const __half2* h = reinterpret_cast<const __half2*>(&v);
    const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
}

__device__ __forceinline__ int in_use(const Params& P, int b) {
  return P.n_nodes ? min(max(P.n_nodes[b], 0), P.n) : P.n;
}

// ---- row_stats: one block per (chunk, row) ----
// Bound by memory latency: 27 MB (4 x 26 rows of 65536 fp32) in 8.3 us, 3.3 TB/s.  Chunks of 4096 to
// 16384 elements and blocks of 128 to 512 threads are all within 3 % of this one.
// Chunks are cut at 16-byte borders, counted from the last border before the row.
template <typename T>
__global__ void __launch_bounds__(kStatThreads) row_stats(const Params P) {
  griddep_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (all that ran before is complete)
  constexpr int kVec = 16 / sizeof(T), kSteps = kChunk / kVec / kStatThreads, kStatWarps = kStatThreads / 32;
  const int b = blockIdx.y / P.n, i = blockIdx.y - b * P.n, draft = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nn = in_use(P, b);
  const float temp = P.temperature ? P.temperature[b] : 1.f;
  float scale = temp;
  bool wanted = i < nn;
  if (draft) {
    // the draft's probabilities are asked for where a child was drawn from this row
    scale = P.draft_temperature ? P.draft_temperature[b] : 1.f;
    bool parent = false;
    for (int c = i + 1 + lane; c < nn; c += 32) parent |= P.parents[(int64_t)b * P.n + c] == i;
    wanted = wanted && temp != 0.f && __any_sync(0xffffffffu, parent);
  }
  if (!wanted) return;
  const float c = 1.44269504088896340736f / (temp == 0.f ? 1.f : scale);  // (at 0 the sum shows NaN and infinities)
  const T* row = draft ? static_cast<const T*>(P.draft) + b * P.d_seq + i * P.d_node
                       : static_cast<const T*>(P.target) + b * P.t_seq + i * P.t_node;
  const int lead = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));  // elements since the last border
  const int j0 = blockIdx.x * kChunk - lead;
  uint4 raw[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int j = j0 + (s * kStatThreads + (int)threadIdx.x) * kVec;
    if (j >= 0 && j + kVec <= P.V) {
      raw[s] = *reinterpret_cast<const uint4*>(row + j);
    } else {
      T* e = reinterpret_cast<T*>(&raw[s]);
#pragma unroll
      for (int k = 0; k < kVec; ++k) e[k] = j + k >= 0 && j + k < P.V ? row[j + k] : lowest<T>();
    }
  }
  // Every thread sums by its own maximum, so that the block waits for its warps only once.  NaN
  // takes no part in the maximum; it comes out of the sum.
  float own = -INFINITY;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) own = fmaxf(own, max_of<T>(raw[s]));
  const float base = own == -INFINITY ? 0.f : own;
  const uint64_t nb = pack2(-base, -base), cc = pack2(c, c);
  uint64_t acc = 0;  // two sums
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    float x[kVec];
    floats_of<T>(raw[s], x);
#pragma unroll
    for (int k = 0; k < kVec; k += 2) {  // exp2((x - base) c)
      uint64_t y = pack2(x[k], x[k + 1]);
      asm("add.rn.f32x2 %0, %0, %1;" : "+l"(y) : "l"(nb));
      asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(y) : "l"(cc));
      const float2 e = unpack2(y);
      y = pack2(ex2(e.x), ex2(e.y));
      asm("add.rn.f32x2 %0, %0, %1;" : "+l"(acc) : "l"(y));
    }
  }
  __shared__ float sm[kStatWarps], ss[kStatWarps];
  __shared__ int si[kStatWarps];
  float m = own;
#pragma unroll
  for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  float sum = (unpack2(acc).x + unpack2(acc).y) * ex2((own - (m == -INFINITY ? 0.f : m)) * c);
#pragma unroll
  for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  int idx = 0x7fffffff;
  if (temp == 0.f) {  // the lowest place of the maximum
    if (own == m) {
#pragma unroll 1
      for (int s = 0; s < kSteps; ++s) {
        const int j = j0 + (s * kStatThreads + (int)threadIdx.x) * kVec;
        for (int k = 0; k < kVec; ++k)
          if (j + k >= 0 && j + k < P.V && to_f(row[j + k]) == m) idx = min(idx, j + k);
      }
    }
    idx = __reduce_min_sync(0xffffffffu, idx);
  }
  if (lane == 0) sm[warp] = m, ss[warp] = sum, si[warp] = idx;
  __syncthreads();
  if (threadIdx.x < kStatWarps) {
    constexpr uint32_t all = (1u << kStatWarps) - 1;
    m = sm[lane], sum = ss[lane], idx = si[lane];
    float top = m;
#pragma unroll
    for (int off = kStatWarps / 2; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(all, top, off));
    sum *= ex2((m - (top == -INFINITY ? 0.f : top)) * c);
#pragma unroll
    for (int off = kStatWarps / 2; off; off >>= 1) sum += __shfl_xor_sync(all, sum, off);
    idx = __reduce_min_sync(all, m == top ? idx : 0x7fffffff);
    if (lane == 0) P.stats[((int64_t)(draft * P.B + b) * P.n + i) * P.chunks + blockIdx.x] = Stat{top, sum, idx, 0};
  }
}

// ---- walk ----
__device__ __forceinline__ void st_peer_f64(uint32_t addr, double x) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(x) : "memory");
}

// 2^y, y = d c, for -1000 <= y <= 0 by a table of 2^(k / 16) and the series of 2^r in the remainder (|r| <=
// 1/32; the term behind the fifth is below 1.5e-13).  The method is P. T. P. Tang's, "Table-driven
// implementation of the exponential function in IEEE floating-point arithmetic", 1989.  The table
// is kept 16 times, a copy for every other lane, so that lookups meet no bank conflicts (with 256
// entries once they took half of a pass).  `low`: y is below -1000, the value 0 (told apart in fp32,
// without a branch: several run side by side).  d is a logit minus the row's largest: the largest one's
// exponential is 1 to the bit, and y as good as d, however small the temperature.
constexpr int kTable = 16, kCopies = 16;
__device__ __forceinline__ double exp2_table(double d, double c, bool low, const double* table) {
  constexpr double kMagic = 6755399441055744.0 / kTable;  // 1.5 * 2^52 / 16: the sum's low bits are round(16 y)
  const double t = fma(d, c, kMagic);
  const int k = __double2loint(t);
  const double r = fma(d, c, kMagic - t);
  constexpr double c1 = 0.69314718055994530942, c2 = c1 * c1 / 2, c3 = c2 * c1 / 3, c4 = c3 * c1 / 4, c5 = c4 * c1 / 5;
  double e = table[(k & (kTable - 1)) * kCopies + (threadIdx.x & (kCopies - 1))];
  e = __hiloint2double(__double2hiint(e) + ((k >> 4) << 20), __double2loint(e));
  e = fma(e, r * fma(r, fma(r, fma(r, fma(r, c5, c4), c3), c2), c1), e);
  return low ? 0.0 : e;
}

template <int N>
__device__ __forceinline__ double sum_of(const double (&v)[N]) {
  double w = (v[0] + v[1]) + (v[2] + v[3]);
  if constexpr (N == 8) w += (v[4] + v[5]) + (v[6] + v[7]);
  return w;
}

// max(v f - q, 0) of a value and the draft's probability.  The product is rounded as q's was, and
// the sums behind f and q's factor are formed in one order: where target and draft are the same
// row the rest is exactly 0.  (A NaN stays.)
__device__ __forceinline__ double rest(double v, double f, double q) {
  const double x = __dsub_rn(__dmul_rn(v, f), q);
  return x < 0.0 ? 0.0 : x;
}

enum Op { OP_DONE, OP_SUMS, OP_LAST, OP_REST, OP_AGAIN, OP_APART };

struct Ctl {
  double table[kTable * kCopies];
  double sums[2][2][kMaxCluster];  // a pass's partial sums (P, q) of every block, by turns
  double warp_sum[2][kWarps];
  double total;                    // of the last pass
  double iP, iQ, iZ[kMaxNodes];    // 1 / sum of a node's exponentials; 1 / sum of its rests so far
  double p[kMaxNodes], q[kMaxNodes];  // exponentials of a child's token in its parent's rows
  float m[2][kMaxNodes], z[2][kMaxNodes], u[kMaxNodes], logit[2][kMaxNodes], pf[kMaxNodes];  // pf: a child's probability
  int idx[kMaxNodes];
  int32_t token[kMaxNodes], gone[kMaxNodes];  // of a child; of the current node's rejected children
  int16_t parent[kMaxNodes];
  uint8_t first[kMaxNodes];        // a child's answer when it is the first one asked: 0, 1, 2 (too close)
  uint8_t again[kMaxNodes];        // a child whose token an earlier sibling had, or outside the vocabulary
  int op, cur, rounds, n_gone;
  // What each block is about to do, by turns.  They decide alike from the same numbers; where those
  // changed under the call (inputs or a workspace that something else writes meanwhile) the blocks part
  // at the next barrier instead of waiting for one another there for ever.
  uint32_t step, steps[2][kMaxCluster];
  int kept;  // rejections that the kept values stand for (0: the exponentials), -1: none are kept
};

template <typename T, bool DRAFT>
__global__ void __launch_bounds__(kThreads) walk(const Params P) {
  constexpr int kPer = kPerOf<DRAFT>, kPass = kThreads * kPer;
  __shared__ Ctl S;
  // this block's slice of a row: the last pass's values of it (element k of thread t in step s at
  // (s kPer + k) kThreads + t), the draft's exponentials alike, and sums of 32 kPer elements each
  extern __shared__ double dyn[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t C = cluster_size(), rank = cluster_rank();
  const int b = blockIdx.x / C, n = P.n, V = P.V, nn = in_use(P, b);
  const float temp = P.temperature ? P.temperature[b] : 1.f;
  const bool greedy = temp == 0.f, sampled = DRAFT && !greedy;
  const double kLog2e = 1.44269504088896340736;
  const double tc = kLog2e / (greedy ? 1.0 : (double)temp);
  const double dc = sampled ? kLog2e / (double)(P.draft_temperature ? P.draft_temperature[b] : 1.f) : 0.0;
  const float tcf = (float)tc, dcf = (float)dc;
  const T* target = static_cast<const T*>(P.target) + b * P.t_seq;
  const T* draft = static_cast<const T*>(P.draft) + (sampled ? b * P.d_seq : 0);

  // the tree, and the logits of its tokens (a thread per node: n <= kThreads)
  if (tid < nn) {
    const int par = max(-1, min(P.parents[(int64_t)b * n + tid], n)), x = P.tokens[(int64_t)b * n + tid];
    const bool asked = par >= 0 && par < tid && x >= 0 && x < V && !greedy;
    S.parent[tid] = (int16_t)par;
    S.token[tid] = x;
    S.u[tid] = greedy ? 0.f : P.u[(int64_t)b * n + tid];
    S.logit[0][tid] = asked ? to_f(target[par * P.t_node + x]) : -INFINITY;
    S.logit[1][tid] = asked && sampled ? to_f(draft[par * P.d_node + x]) : -INFINITY;
  }
  if (tid < kTable * kCopies && !greedy) S.table[tid] = exp2(tid / kCopies / (double)kTable);
  cluster_sync();  // also: every block of the cluster has started
  griddep_wait();  // row_stats is done
  // a row's statistics from its chunks, half a warp per row (its lanes side by side take 16 chunks);
  // for the draft's rows of nodes without children, which row_stats leaves out, they mean nothing and are not used
  const int n_rows = nn * (sampled ? 2 : 1), in = lane & 15;
#pragma unroll 1
  for (int x = warp * 2 + (lane >> 4); __any_sync(0xffffffffu, x < n_rows); x += kWarps * 2) {
    const bool there = x < n_rows;
    const int d = x >= nn, i = d ? x - nn : x;
    const Stat* st = P.stats + ((int64_t)(d * P.B + b) * n + i) * P.chunks;
    float m = -INFINITY, z = 0.f;
    int idx = 0x7fffffff;
    const float c = d ? dcf : tcf;
#pragma unroll 1
    for (int k = there ? in : P.chunks; k < P.chunks; k += 16) {
      const Stat s = st[k];
      if (s.m > m) idx = s.idx;  // chunks in order: an equal maximum keeps the lower index
      const float top = fmaxf(m, s.m), base = top == -INFINITY ? 0.f : top;
      z = z * ex2((m - base) * c) + s.s * ex2((s.m - base) * c);
      m = top;
    }
    __syncwarp();
    float top = m;
#pragma unroll
    for (int off = 8; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    z *= ex2((m - (top == -INFINITY ? 0.f : top)) * c);
    idx = m == top ? idx : 0x7fffffff;
#pragma unroll
    for (int off = 8; off; off >>= 1) {
      z += __shfl_xor_sync(0xffffffffu, z, off);
      idx = min(idx, __shfl_xor_sync(0xffffffffu, idx, off));
    }
    if (there && in == 0) {
      S.m[d][i] = top, S.z[d][i] = z;
      if (!d) S.idx[i] = z > 0.f && z < INFINITY ? idx : -1;  // (else no distribution)
    }
  }
  __syncthreads();
  if (tid < nn && !greedy) {
    const int par = S.parent[tid];
    const float lt = S.logit[0][tid], ld = S.logit[1][tid];
    double p = 0.0, q = 0.0;
    if (lt != -INFINITY) {  // (a NaN stays)
      const float mt = S.m[0][par];
      p = exp2_table((double)lt - (double)mt, tc, (lt - mt) * tcf <= -1000.f, S.table);
    }
    if (sampled && ld != -INFINITY) {
      const float md = S.m[1][par];
      q = exp2_table((double)ld - (double)md, dc, (ld - md) * dcf <= -1000.f, S.table);
    }
    S.p[tid] = p, S.q[tid] = q;
    if (!DRAFT) S.pf[tid] = par >= 0 && par < tid ? (float)p / S.z[0][par] : 0.f;
    if (par >= 0 && par < tid) {
      // u q / ZQ < p / ZP without divisions
      const double a = (double)S.u[tid] * (sampled ? q : 1.0) * (double)S.z[0][par];
      const double e = p * (sampled ? (double)S.z[1][par] : 1.0), top = fmax(a, e);
      // (sums that are NaN, as fp32's are at temperatures below 2^-127, settle nothing either)
      S.first[tid] = !(fabs(a - e) > (double)kClose * top) && top != 0.0 ? 2 : a < e;
    }
    const int x = S.token[tid];
    bool again = x < 0 || x >= V;
    if (!sampled)
      for (int k = par + 1; k < tid; ++k) again |= S.parent[k] == par && S.token[k] == x;
    S.again[tid] = again;
  }
  __syncthreads();

  // Warp 0 of every block walks, its lanes alike; what it decides follows from the same numbers in
  // each block.
  int32_t* path = P.path + (int64_t)b * n;
  int cur = 0, depth = nn > 0 ? 1 : 0, c = 1;  // warp 0's
  bool exact = false;                          // iP, iQ are the current node's
  bool summed = false;                         // `piece` holds the current P
  bool apart = false;                          // the blocks' decisions differ
  float left = 1.f;                            // without draft: what of P is not gone,
  double left_exact = 1.0;                     // and the same from exact sums
  if (tid == 0) S.rounds = S.n_gone = 0, S.kept = -1;
  int turn = 0;
  const int slice = (((V + 3 + (int)C - 1) / (int)C) + 3) & ~3;  // elements per block
  const int room = (slice + kPass - 1) / kPass * kPass;
  double* const kept_v = dyn + tid;
  double* const kept_q = kept_v + room;
  double* const piece = dyn + P.keep * room + P.q_steps * kPass;
  __syncwarp();
  for (;;) {
    if (warp == 0) {
      int op = OP_DONE;
      int rounds = S.rounds, n_gone = S.n_gone;
      while (!apart) {
        // the current node's next child from c on
        uint32_t kids = 0;
        int base = c;
        for (; base < nn; base += 32) {
          kids = __ballot_sync(0xffffffffu, base + lane < nn && S.parent[base + lane] == cur);
          if (kids) break;
        }
        c = kids ? base + __ffs(kids) - 1 : nn;
        if (c >= nn) break;
        bool take;
        if (greedy) {
          const int x = S.token[c];
          take = x >= 0 && x == S.idx[cur];
        } else if (!exact) {
          int first = S.first[c];
          if (!DRAFT && n_gone > 0) {
            // (fp32 statistics and this sum know what is left to kClose + 6e-8 per term)
            const float p = S.again[c] ? 0.f : S.pf[c], a = S.u[c] * left, top = fmaxf(a, p);
            first = !(left >= 0.125f) || (!(fabsf(a - p) * left > (kClose + 6e-8f * n_gone) * top) && top != 0.f) ? 2 : a < p;
          }
          if (first == 2) {
            op = OP_SUMS;  // too close for fp32 statistics: come back with exact ones
            break;
          }
          take = first;
        } else {
          double p = S.p[c] * S.iP, a = (double)S.u[c];
          if (sampled) {
            const double q = S.q[c] * S.iQ;
            for (int k = 0; k < rounds; ++k) p = fmax(p - q, 0.0) * S.iZ[k];
            a *= q;
          } else {
            if (S.again[c]) p = 0.0;
            a *= left_exact;
          }
          take = a < p;
        }
        if (take) {
          if (rank == 0 && lane == 0) path[depth] = c;
          ++depth;
          cur = c;
          exact = summed = false;
          rounds = n_gone = 0;
          left = 1.f;
        } else if (greedy) {
        } else if (sampled) {
          op = exact ? OP_REST : OP_SUMS;  // rejected: what is left of P
          break;
        } else if (!S.again[c]) {
          if (lane == 0) S.gone[n_gone] = c;
          ++n_gone;
          left -= S.pf[c];
          if (exact) left_exact -= S.p[c] * S.iP;
          summed = false;
        }
        ++c;
      }
      if (op == OP_DONE && !greedy && nn > 0 && !summed) op = rounds > 0 ? OP_AGAIN : OP_LAST;
      if (apart) op = OP_APART;
      __syncwarp();
      if (lane == 0) {
        S.rounds = rounds, S.n_gone = n_gone;
        S.op = op;
        S.cur = cur;
        S.step = 1u << 31 | (uint32_t)op << 28 | rounds << 18 | cur << 9 | c;
      }
    }
    __syncthreads();
    const int op = S.op;
    if (op == OP_DONE || op == OP_APART) break;
    // ---- a pass over the current node's rows: this block's slice, kPer elements per thread and step.
    // OP_SUMS: sums of the exponentials (without the tokens that are gone: also what is drawn
    // from when nothing was rejected).  OP_LAST: the same for the draw alone, with no child left to
    // ask; it reads no draft row (a node without children need not have one).  OP_REST: the sum of the
    // rest after one more rejection; OP_AGAIN: after the rejections so far (the last OP_REST left
    // nothing, and P stayed).
    const int node = S.cur;
    const T* tp = target + node * P.t_node;
    const bool with_q = sampled && op != OP_LAST;
    const T* dp = draft + (with_q ? node * P.d_node : 0);
    // slices and steps are counted from the last 4-element border before the target's row
    const int lead = (int)((reinterpret_cast<uintptr_t>(tp) / sizeof(T)) & 3);
    const bool d_vec = ((reinterpret_cast<uintptr_t>(dp) / sizeof(T)) & 3) == (uintptr_t)lead;
    const int lo = (int)rank * slice - lead, hi = min(V, lo + slice);
    const float mtf = S.m[0][node], mdf = S.m[1][node];
    const double mp = mtf, mq = mdf;
    const int rounds = op == OP_SUMS || op == OP_LAST ? 0 : S.rounds + (op == OP_REST), n_gone = S.n_gone;
    const double iP = S.iP, iQ = S.iQ;
    auto load4 = [&](const T* row, bool vec, int j, float* x) {
      if (vec && j >= 0 && j + 4 <= hi) {
        if constexpr (sizeof(T) == 4) {
          const float4 v = *reinterpret_cast<const float4*>(row + j);
          x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(row + j);
          const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = to_f(e[k]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = j + k >= 0 && j + k < hi ? to_f(row[j + k]) : -INFINITY;
      }
    };
    // Rejections one after another start from what the pass before kept, not from the logits.
    const bool store = sampled && P.keep > 0;
    const bool from_kept = store && op == OP_REST && S.kept == rounds - 1;
    const double scale = rounds > 1 ? S.iZ[rounds > 1 ? rounds - 2 : 0] : iP;
    double sv = 0.0, sq = 0.0;
    float tl[kPer], dl[kPer] = {};
#pragma unroll 1
    for (int s = 0, j = lo + tid * kPer; lo + s * kPass < hi; ++s, j += kPass) {
      double v[kPer], q[kPer];
      double* const at_v = kept_v + s * kPass;
      double* const at_q = kept_q + s * kPass;
      const bool keep_q = store && s < P.q_steps, q_from_kept = from_kept && keep_q;
      if (!from_kept)
#pragma unroll
        for (int k = 0; k < kPer; k += 4) load4(tp, true, j + k, tl + k);
      if (with_q && !q_from_kept)
#pragma unroll
        for (int k = 0; k < kPer; k += 4) load4(dp, d_vec, j + k, dl + k);
      if (from_kept) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] = at_v[k * kThreads];
      } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] = exp2_table((double)tl[k] - mp, tc, (tl[k] - mtf) * tcf <= -1000.f, S.table);
      }
      if (with_q) {
        if (q_from_kept) {
#pragma unroll
          for (int k = 0; k < kPer; ++k) q[k] = at_q[k * kThreads];
        } else {
#pragma unroll
          for (int k = 0; k < kPer; ++k) q[k] = exp2_table((double)dl[k] - mq, dc, (dl[k] - mdf) * dcf <= -1000.f, S.table);
          if (keep_q)
#pragma unroll
            for (int k = 0; k < kPer; ++k) at_q[k * kThreads] = q[k];
        }
        if (rounds == 0) {
          sq += sum_of<kPer>(q);
        } else {
#pragma unroll
          for (int k = 0; k < kPer; ++k) q[k] *= iQ;
          // all rejections so far, or only the last one
#pragma unroll 1
          for (int y = from_kept ? rounds - 1 : 0; y < rounds; ++y) {
            const double f = from_kept ? scale : y == 0 ? iP : S.iZ[y - 1];
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
              v[k] = rest(v[k], f, q[k]);
            }
          }
        }
      }
      if (sampled) {
        if (store)
#pragma unroll
          for (int k = 0; k < kPer; ++k) at_v[k * kThreads] = v[k];
      } else {
        for (int y = 0; y < n_gone; ++y) {
          const int at = S.token[S.gone[y]] - j;
#pragma unroll
          for (int k = 0; k < kPer; ++k)
            if (at == k) v[k] = 0.0;
        }
      }
      double w = sum_of<kPer>(v);
      sv += w;
#pragma unroll
      for (int off = 16; off; off >>= 1) w += __shfl_xor_sync(0xffffffffu, w, off);
      if (lane == 0) piece[s * kWarps + warp] = w;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      sv += __shfl_xor_sync(0xffffffffu, sv, off);
      sq += __shfl_xor_sync(0xffffffffu, sq, off);
    }
    if (lane == 0) S.warp_sum[0][warp] = sv, S.warp_sum[1][warp] = sq;
    const int slot = turn++ & 1;
    __syncthreads();
    if (warp < 2) {
      double x = lane < kWarps ? S.warp_sum[warp][lane] : 0.0;
#pragma unroll
      for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      if (lane < (int)C) st_peer_f64(mapa(smem_u32(&S.sums[slot][warp][rank]), lane), x);
    } else if (warp == 2 && lane < (int)C) {
      st_peer_u32(mapa(smem_u32(&S.steps[slot][rank]), lane), S.step);
    }
    cluster_sync();
    if (warp == 0) {
      apart = __any_sync(0xffffffffu, lane < (int)C && S.steps[slot][lane] != S.step);
      double t = lane < (int)C ? S.sums[slot][0][lane] : 0.0, z = lane < (int)C ? S.sums[slot][1][lane] : 0.0;
#pragma unroll
      for (int off = kMaxCluster / 2; off; off >>= 1) {
        t += __shfl_xor_sync(0xffffffffu, t, off);
        z += __shfl_xor_sync(0xffffffffu, z, off);
      }
      if (lane == 0) S.total = t;
      if (op == OP_SUMS || op == OP_LAST) {
        // what was taken out of P belongs to the sum of its exponentials (and a NaN makes it none)
        for (int k = 0; k < S.n_gone; ++k) t += S.p[S.gone[k]];
        if (!DRAFT && lane == 0 && isnan(t)) S.total = t;
        const double iP = 1.0 / (lane == 1 ? z : t);
        if (lane == 0) S.iP = iP, S.kept = 0;
        if (lane == 1) S.iQ = iP;
        exact = summed = true;
        if (!DRAFT) {
          __syncwarp();
          left_exact = 1.0;
          for (int k = 0; k < S.n_gone; ++k) left_exact -= S.p[S.gone[k]] * S.iP;
        }
      } else if (op == OP_AGAIN) {
        summed = true;
        if (lane == 0) S.kept = S.rounds;
      } else {
        // (a sum that is NaN counts as something: the draw then finds no distribution)
        summed = !(t <= 0.0);  // else nothing would be left: P stays
        if (lane == 0) {
          if (summed) S.iZ[S.rounds++] = 1.0 / t;
          S.kept = summed ? S.rounds : -1;
        }
        ++c;  // this child is dealt with
      }
      __syncwarp();
    }
  }

  if (S.op == OP_APART) {  // (nobody waits for this block, nor stores into it, any more)
    if (rank == 0) {
      for (int k = tid; k < n; k += kThreads) path[k] = -1;
      if (tid == 0) P.n_path[b] = 0, P.next_token[b] = -1;
    }
    return;
  }
  if (warp == 2 && lane < (int)C) st_peer_u32(mapa(smem_u32(&S.steps[turn & 1][rank]), lane), S.step);

  // ---- the draw: `piece` and S.sums hold the final P, unscaled, in order ----
  if (tid == 0 && rank == 0) {
    for (int k = depth; k < n; ++k) path[k] = -1;
    if (depth > 0) path[0] = 0;
    P.n_path[b] = depth;
  }
  if (greedy || nn == 0) {
    if (tid == 0 && rank == 0) P.next_token[b] = nn > 0 ? S.idx[S.cur] : -1;
  } else if (warp == 0) {
    const int slot = (turn - 1) & 1;
    const double total = S.total, want = P.r[b] > 0.f ? (double)P.r[b] * total : 0.0;
    double before = 0.0;  // of the blocks before this one
    int last = -1;        // the last block with any P: takes what rounding leaves over
    for (int k = 0; k < (int)C; ++k) {
      if (k < (int)rank) before += S.sums[slot][0][k];
      if (S.sums[slot][0][k] > 0.0) last = k;
    }
    const double mine = S.sums[slot][0][rank];
    if (!(total > 0.0 && total < INFINITY)) {
      if (tid == 0 && rank == 0) P.next_token[b] = -1;  // no distribution
    } else if (before <= want && (before + mine > want || (int)rank == last) && mine > 0.0) {
      // pieces of 32 kPer elements, then the elements of one piece
      const T* tp = target + S.cur * P.t_node;
      const T* dp = draft + (sampled ? S.cur * P.d_node : 0);
      const int lead = (int)((reinterpret_cast<uintptr_t>(tp) / sizeof(T)) & 3);
      const int lo = (int)rank * slice - lead, hi = min(V, lo + slice);
      const int n_piece = (hi - lo + kPass - 1) / kPass * kWarps;
      int at = -1, keep = -1;
      double base = before, sure = before;
      for (int k0 = 0; k0 < n_piece && at < 0; k0 += 32) {
        const double x = k0 + lane < n_piece ? piece[k0 + lane] : 0.0;
        double cum = x;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const double o = __shfl_up_sync(0xffffffffu, cum, off);
          if (lane >= off) cum += o;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, x > 0.0 && base + cum > want);
        const uint32_t some = __ballot_sync(0xffffffffu, x > 0.0);
        if (hit) {
          const int l = __ffs(hit) - 1;
          at = k0 + l;
          base += __shfl_sync(0xffffffffu, cum - x, l);
        } else {
          if (some) {
            const int l = 31 - __clz(some);
            keep = k0 + l;
            sure = base + __shfl_sync(0xffffffffu, cum - x, l);
          }
          base += __shfl_sync(0xffffffffu, cum, 31);
        }
      }
      if (at < 0) at = keep, base = sure;
      // the rows once more, as the last pass saw them
      const int rounds = S.rounds;
      const float mtf = S.m[0][S.cur], mdf = S.m[1][S.cur];
      const double mp = mtf, mq = mdf;
      double v[kPer], sum = 0.0;
      const int j = lo + at / kWarps * kPass + (at % kWarps * 32 + lane) * kPer;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        v[k] = 0.0;
        if (j + k >= 0 && j + k < hi) {
          if (sampled && P.keep > 0 && S.kept == rounds) {
            v[k] = dyn[(at / kWarps * kPer + k) * kThreads + at % kWarps * 32 + lane];
          } else {
            const float tl = to_f(tp[j + k]);
            v[k] = exp2_table((double)tl - mp, tc, (tl - mtf) * tcf <= -1000.f, S.table);
            if (rounds > 0) {
              const float dl = to_f(dp[j + k]);
              const double q = exp2_table((double)dl - mq, dc, (dl - mdf) * dcf <= -1000.f, S.table) * S.iQ;
              for (int y = 0; y < rounds; ++y) {
                v[k] = rest(v[k], y == 0 ? S.iP : S.iZ[y - 1], q);
              }
            } else {
              for (int y = 0; y < S.n_gone; ++y)
                if (S.token[S.gone[y]] == j + k) v[k] = 0.0;
            }
          }
        }
        sum += v[k];
      }
      double cum = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, cum, off);
        if (lane >= off) cum += o;
      }
      double run = base + (cum - sum);
      int hit = 0x7fffffff, any = -1;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        run += v[k];
        if (v[k] > 0.0) {
          any = j + k;
          if (run > want && hit == 0x7fffffff) hit = j + k;
        }
      }
      hit = __reduce_min_sync(0xffffffffu, hit);
      any = __reduce_max_sync(0xffffffffu, any);
      if (lane == 0) P.next_token[b] = hit != 0x7fffffff ? hit : any;
    }
  }
  cluster_sync();  // no block leaves while a peer may still store into it
}

}  // namespace verify

size_t tree_verify_workspace_bytes(int B, int n, int V) {
  const int chunks = (V + 8 + verify::kChunk - 1) / verify::kChunk;
  return (size_t)2 * B * n * chunks * sizeof(verify::Stat);
}

template <typename T, bool DRAFT>
static cudaError_t verify_launch(verify::Params P, cudaStream_t stream) {
  using namespace verify;
  constexpr int kPass = kThreads * kPerOf<DRAFT>;
  static std::atomic<int> largest[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = launch_early(row_stats<T>, dim3(P.chunks, P.B * P.n, P.draft ? 2 : 1), kStatThreads, stream, P);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  int most = dev < 64 ? largest[dev].load() : 0;
  if (!most) {
    e = cudaFuncSetAttribute(walk<T, DRAFT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(walk<T, DRAFT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDyn);
    if (e != cudaSuccess) return e;
    cfg.dynamicSmemBytes = kMaxDyn;
    cfg.numAttrs = 1;
    attr[0].val.clusterDim.x = kMaxCluster;
    cfg.gridDim = dim3(kMaxCluster);
    int fit = 0;
    if (cudaOccupancyMaxActiveClusters(&fit, walk<T, DRAFT>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      fit = 0;
    }
    most = fit >= 1 ? kMaxCluster : 8;
    if (dev < 64) largest[dev].store(most);
  }
  // A sequence's walk waits for its own passes: as many blocks as the batch leaves room for.
  int C = P.B * 16 <= 128 ? most : 8;
  while (C > 1 && (int64_t)(C - 1) * kPass >= P.V) C /= 2;
  // shared memory as the kernel lays it out
  const int slice = ((P.V + 3 + C - 1) / C + 3) & ~3, steps = (slice + kPass - 1) / kPass;
  const size_t row = (size_t)steps * kPass * sizeof(double), pieces = (size_t)steps * kWarps * sizeof(double);
  const size_t step = kPass * sizeof(double);
  P.keep = P.draft && row + pieces <= kMaxDyn;
  P.q_steps = P.keep ? (int)std::min<size_t>(steps, (kMaxDyn - row - pieces) / step) : 0;
  cfg.dynamicSmemBytes = P.keep * row + P.q_steps * step + pieces;
  if (cfg.dynamicSmemBytes > kMaxDyn) return cudaErrorInvalidValue;
  attr[0].val.clusterDim.x = C;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3(C * P.B);
  return cudaLaunchKernelEx(&cfg, walk<T, DRAFT>, P);
}

int tree_verify(const TreeVerify& a, void* workspace, cudaStream_t stream, std::string* err) {
  verify::Params P;
  P.target = a.target, P.draft = a.draft;
  P.t_seq = a.t_seq, P.t_node = a.t_node, P.d_seq = a.d_seq, P.d_node = a.d_node;
  P.tokens = a.tokens, P.parents = a.parents, P.n_nodes = a.n_nodes;
  P.u = a.u, P.r = a.r, P.temperature = a.temperature, P.draft_temperature = a.draft_temperature;
  P.path = a.path, P.n_path = a.n_path, P.next_token = a.next_token;
  P.stats = static_cast<verify::Stat*>(workspace);
  P.B = a.B, P.n = a.n, P.V = a.vocab;
  P.chunks = (a.vocab + 8 + verify::kChunk - 1) / verify::kChunk;
  const cudaError_t e = a.dtype == MK_FP32   ? (P.draft ? verify_launch<float, true>(P, stream) : verify_launch<float, false>(P, stream))
                        : a.dtype == MK_BF16 ? (P.draft ? verify_launch<__nv_bfloat16, true>(P, stream) : verify_launch<__nv_bfloat16, false>(P, stream))
                                             : (P.draft ? verify_launch<__half, true>(P, stream) : verify_launch<__half, false>(P, stream));
  if (e != cudaSuccess) {
    *err = std::string("tree_verify launch: ") + cudaGetErrorString(e);
    return MK_ERR_CUDA;
  }
  return MK_OK;
}

}  // namespace mk
