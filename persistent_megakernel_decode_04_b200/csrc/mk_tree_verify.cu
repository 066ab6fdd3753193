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
// index and the sum of exponentials (bound by memory: the other kernel's reads come from L2).
// walk, a thread-block cluster per sequence, goes down the tree with scalars only; where a whole
// row is needed (the rest after a rejected sampled draft, the final draw) the cluster's blocks
// take a slice each and exchange one partial sum through distributed shared memory.
//
// Precision.  A draw from 1e5 words by cumulative sums meets a border within 1e-7 in about every
// hundredth draw, so sums that decide a draw are formed in fp64 from exponentials good to 1e-13.
// Acceptance compares two numbers: fp32 statistics (relative error below 4e-6: 2^-22 for each
// exponential and at most 2^-24 x 64 for the sums) decide unless the two are that close; then the
// row's sums are formed in fp64 first.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <atomic>

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
constexpr int kPass = kThreads * 4;  // elements of a block's pass step: 4 per thread
constexpr float kClose = 1e-5f;

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
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ int in_use(const Params& P, int b) {
  return P.n_nodes ? min(max(P.n_nodes[b], 0), P.n) : P.n;
}

// ---- row_stats: one block per (chunk, row) ----
// Chunks are cut at 16-byte borders, counted from the last border before the row.
template <typename T>
__global__ void __launch_bounds__(kStatThreads) row_stats(const Params P) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kVec = 16 / sizeof(T), kSteps = kChunk / kVec / kStatThreads;
  const int b = blockIdx.y / P.n, i = blockIdx.y - b * P.n, draft = blockIdx.z;
  const int nn = in_use(P, b);
  if (i >= nn) return;
  const float temp = P.temperature ? P.temperature[b] : 1.f;
  float scale = temp;
  if (draft) {
    if (temp == 0.f) return;  // the draft's probabilities are not asked for
    scale = P.draft_temperature ? P.draft_temperature[b] : 1.f;
    bool parent = false;
    for (int c = i + 1 + threadIdx.x; c < nn; c += kStatThreads) parent |= P.parents[(int64_t)b * P.n + c] == i;
    if (!__syncthreads_or(parent)) return;  // no child was drawn from this row
  }
  const float c = 1.44269504088896340736f / scale;
  const T* row = draft ? static_cast<const T*>(P.draft) + b * P.d_seq + i * P.d_node
                       : static_cast<const T*>(P.target) + b * P.t_seq + i * P.t_node;
  const int lead = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));  // elements since the last border
  const int j0 = blockIdx.x * kChunk - lead;
  float x[kSteps][kVec];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int j = j0 + (s * kStatThreads + (int)threadIdx.x) * kVec;
    if (j >= 0 && j + kVec <= P.V) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + j);
      const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (int k = 0; k < kVec; ++k) x[s][k] = to_f(e[k]);
    } else {
#pragma unroll
      for (int k = 0; k < kVec; ++k) x[s][k] = j + k >= 0 && j + k < P.V ? to_f(row[j + k]) : -INFINITY;
    }
  }
  float m = -INFINITY;
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
#pragma unroll
    for (int k = 0; k < kVec; ++k) m = fmaxf(m, x[s][k]);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float sm[kStatThreads / 32], ss[kStatThreads / 32];
  __shared__ int si[kStatThreads / 32];
#pragma unroll
  for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (lane == 0) sm[warp] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kStatThreads / 32; ++k) m = fmaxf(m, sm[k]);
  const float base = m == -INFINITY ? 0.f : m;
  float sum = 0.f;
  int idx = 0x7fffffff;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int j = j0 + (s * kStatThreads + (int)threadIdx.x) * kVec;
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      sum += ex2((x[s][k] - base) * c);  // at temperature 0 c is infinite: the sum is not used
      if (x[s][k] == m && j + k >= 0 && j + k < P.V) idx = min(idx, j + k);
    }
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, off);
    idx = min(idx, __shfl_xor_sync(0xffffffffu, idx, off));
  }
  if (lane == 0) ss[warp] = sum, si[warp] = idx;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kStatThreads / 32; ++k) sum += ss[k], idx = min(idx, si[k]);
    P.stats[((int64_t)(draft * P.B + b) * P.n + i) * P.chunks + blockIdx.x] = Stat{m, sum, idx, 0};
  }
}

// ---- walk ----
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_peer_f64(uint32_t addr, double x) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(x) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 2^y for y <= 0 by a table of 2^(k / 256) and a cubic in the remainder (|r| <= 2^-9: the next
// term of the series is below 1.4e-13).  The method is P. T. P. Tang's, "Table-driven
// implementation of the exponential function in IEEE floating-point arithmetic", 1989.
__device__ __forceinline__ double exp2_table(double y, const double* table) {
  constexpr double kMagic = 6755399441055744.0 / 256;  // 1.5 * 2^52 / 256: the sum's low bits are round(256 y)
  if (!(y > -1000.0)) return y != y ? y : 0.0;
  const double t = y + kMagic;
  const int k = __double2loint(t);
  const double r = y - (t - kMagic);
  constexpr double c1 = 0.69314718055994530942, c2 = c1 * c1 / 2, c3 = c1 * c1 * c1 / 6;
  double e = table[k & 255];
  e = __hiloint2double(__double2hiint(e) + ((k >> 8) << 20), __double2loint(e));
  return fma(e, r * fma(r, fma(r, c3, c2), c1), e);
}

enum Op { OP_DONE, OP_SUMS, OP_REST, OP_AGAIN };

struct Ctl {
  double table[256];
  double sums[2][3][kMaxCluster];  // a pass's partial sums of every block, by turns
  double warp_sum[kWarps];
  double total[3];
  double ZP, ZQ, Z[kMaxNodes];    // sums of a node's exponentials; of its rests so far
  float m[2][kMaxNodes], z[2][kMaxNodes];
  int idx[kMaxNodes];
  int16_t parent[kMaxNodes], gone[kMaxNodes];
  int32_t token[kMaxNodes];
  float u[kMaxNodes];
  double p[kMaxNodes], q[kMaxNodes];  // exponentials of a child's token in its parent's rows
  int op, cur, rounds, n_gone, found;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) walk(const Params P) {
  __shared__ Ctl S;
  extern __shared__ double piece[];  // sums of 128 elements each, in order: this block's slice of a row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t C, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(C));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int b = blockIdx.x / C, n = P.n, V = P.V, nn = in_use(P, b);
  const float temp = P.temperature ? P.temperature[b] : 1.f;
  const bool greedy = temp == 0.f, sampled = P.draft != nullptr && !greedy;
  const double kLog2e = 1.44269504088896340736;
  const double tc = kLog2e / (double)temp;
  const double dc = sampled ? kLog2e / (double)(P.draft_temperature ? P.draft_temperature[b] : 1.f) : 0.0;
  const T* target = static_cast<const T*>(P.target) + b * P.t_seq;
  const T* draft = static_cast<const T*>(P.draft) + (sampled ? b * P.d_seq : 0);

  for (int i = tid; i < nn; i += kThreads) {
    S.parent[i] = (int16_t)max(-1, min(P.parents[(int64_t)b * n + i], n));
    S.token[i] = P.tokens[(int64_t)b * n + i];
    S.u[i] = greedy ? 0.f : P.u[(int64_t)b * n + i];
  }
  if (tid < 256 && !greedy) S.table[tid] = exp2(tid / 256.0);
  cluster_sync();  // also: every block of the cluster has started
  asm volatile("griddepcontrol.wait;" ::: "memory");  // row_stats is done
  // a row's statistics from its chunks, a warp per row
  for (int x = warp; x < nn * (sampled ? 2 : 1); x += kWarps) {
    const int d = x >= nn, i = d ? x - nn : x;
    const Stat* st = P.stats + ((int64_t)(d * P.B + b) * n + i) * P.chunks;
    float m = -INFINITY, z = 0.f;
    int idx = 0x7fffffff;
    const float c = (float)(d ? dc : tc);
    for (int k = lane; k < P.chunks; k += 32) {
      const Stat s = st[k];
      if (s.m > m) idx = s.idx;  // chunks in order: an equal maximum keeps the lower index
      const float top = fmaxf(m, s.m), base = top == -INFINITY ? 0.f : top;
      z = z * ex2((m - base) * c) + s.s * ex2((s.m - base) * c);
      m = top;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, off), z2 = __shfl_xor_sync(0xffffffffu, z, off);
      const int i2 = __shfl_xor_sync(0xffffffffu, idx, off);
      const float top = fmaxf(m, m2), base = top == -INFINITY ? 0.f : top;
      idx = m == m2 ? min(idx, i2) : m > m2 ? idx : i2;
      z = z * ex2((m - base) * c) + z2 * ex2((m2 - base) * c);
      m = top;
    }
    if (lane == 0) {
      S.m[d][i] = m, S.z[d][i] = z;
      if (!d) S.idx[i] = idx;
    }
  }
  __syncthreads();
  if (!greedy)
    for (int c = tid; c < nn; c += kThreads) {
      const int par = S.parent[c], x = S.token[c];
      double p = 0.0, q = 0.0;
      if (par >= 0 && par < c && x >= 0 && x < V) {
        p = exp2_table(((double)to_f(target[par * P.t_node + x]) - (double)S.m[0][par]) * tc, S.table);
        if (sampled) q = exp2_table(((double)to_f(draft[par * P.d_node + x]) - (double)S.m[1][par]) * dc, S.table);
      }
      S.p[c] = p, S.q[c] = q;
    }
  __syncthreads();

  // Thread 0 of every block walks; what it decides follows from the same numbers in each.
  int32_t* path = P.path + (int64_t)b * n;
  int cur = 0, depth = nn > 0 ? 1 : 0, c = 1;  // thread 0's
  bool exact = false;                          // ZP, ZQ are the current node's
  bool summed = false;                         // `piece` holds the current P
  if (tid == 0) {
    S.rounds = S.n_gone = 0;
    S.found = -1;
  }
  int turn = 0;
  const int slice = (((V + (int)C - 1) / (int)C) + 3) & ~3;  // elements per block
  const int lo = min(V, (int)rank * slice), hi = min(V, lo + slice);
  for (;;) {
    if (tid == 0) {
      int op = OP_DONE;
      for (; c < nn; ++c) {
        if (S.parent[c] != cur) continue;
        const int x = S.token[c];
        if (greedy) {
          if (x < 0 || x != S.idx[cur]) continue;
        } else {
          const double ZP = exact ? S.ZP : (double)S.z[0][cur], ZQ = sampled ? (exact ? S.ZQ : (double)S.z[1][cur]) : 1.0;
          double p = S.p[c] / ZP, q = sampled ? S.q[c] / ZQ : 1.0, left = 1.0;
          if (sampled) {
            for (int k = 0; k < S.rounds; ++k) p = fmax(p - q, 0.0) / S.Z[k];
          } else {
            for (int k = 0; k < S.n_gone; ++k) {
              left -= S.p[S.gone[k]] / ZP;
              if (S.token[S.gone[k]] == x) p = 0.0;
            }
            p /= left;
          }
          const double a = (double)S.u[c] * q;
          // (what is left of P is known to kClose / left)
          if (!exact && (left < 0.125 || (fabs(a - p) <= kClose / left * fmax(a, p) && fmax(a, p) > 0.0))) {
            op = OP_SUMS;  // too close for fp32 statistics: come back with exact ones
            break;
          }
          if (!(a < p)) {
            // rejected: what is left of P
            if (sampled) {
              op = exact ? OP_REST : OP_SUMS;
              break;
            }
            bool known = x < 0 || x >= V;
            for (int k = 0; k < S.n_gone; ++k) known |= S.token[S.gone[k]] == x;
            if (!known) S.gone[S.n_gone++] = (int16_t)c, summed = false;
            continue;
          }
        }
        if (rank == 0) path[depth] = c;
        ++depth;
        cur = c;
        exact = summed = false;
        S.rounds = S.n_gone = 0;
      }
      if (op == OP_DONE && !greedy && nn > 0 && !summed) op = S.rounds > 0 ? OP_AGAIN : OP_SUMS;
      S.op = op;
      S.cur = cur;
    }
    __syncthreads();
    const int op = S.op;
    if (op == OP_DONE) break;
    // ---- a pass over the current node's rows: this block's slice, 4 elements per thread and step.
    // OP_SUMS: sums of the exponentials (without the tokens that are gone: also what is drawn
    // from when nothing was rejected).  OP_REST: the sum of the rest after one more rejection;
    // OP_AGAIN: after the rejections so far (the last OP_REST left nothing, and P stayed).
    const int node = S.cur;
    const T* tp = target + node * P.t_node;
    const T* dp = draft + (sampled ? node * P.d_node : 0);
    const double mp = (double)S.m[0][node] * tc, mq = sampled ? (double)S.m[1][node] * dc : 0.0;
    const int rounds = op == OP_SUMS ? 0 : S.rounds + (op == OP_REST), n_gone = S.n_gone;
    const bool wants_q = sampled && (rounds > 0 || op == OP_SUMS);
    const double iP = 1.0 / S.ZP, iQ = 1.0 / S.ZQ;
    // the current P (op: SUMS unscaled, else after `rounds` rejections; the last one not yet scaled)
    auto value = [&](int j, float tl, float dl, double& q) {
      double v = exp2_table(fma((double)tl, tc, -mp), S.table);
      if (wants_q) q = exp2_table(fma((double)dl, dc, -mq), S.table);
      if (op != OP_SUMS) {
        v *= iP;
        const double qq = q * iQ;
        for (int k = 0; k < rounds - 1; ++k) v = fmax(v - qq, 0.0) / S.Z[k];
        v = fmax(v - qq, 0.0);
      } else {
        for (int k = 0; k < n_gone; ++k)
          if (S.token[S.gone[k]] == j) v = 0.0;
      }
      return v;
    };
    const bool t_vec = (reinterpret_cast<uintptr_t>(tp + lo) & (4 * sizeof(T) - 1)) == 0;
    const bool d_vec = (reinterpret_cast<uintptr_t>(dp + lo) & (4 * sizeof(T) - 1)) == 0;
    auto load4 = [&](const T* row, bool vec, int j, float* x) {
      if (vec && j + 4 <= hi) {
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
        for (int k = 0; k < 4; ++k) x[k] = j + k < hi ? to_f(row[j + k]) : -INFINITY;
      }
    };
    double sv = 0.0, sq = 0.0, full = 0.0;
    for (int s = 0, j = lo + tid * 4; lo + s * kPass < hi; ++s, j += kPass) {
      float tl[4], dl[4] = {0.f, 0.f, 0.f, 0.f};
      load4(tp, t_vec, j, tl);
      if (wants_q) load4(dp, d_vec, j, dl);
      double v = 0.0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        double q = 0.0;
        v += value(j + k, tl[k], dl[k], q);
        sq += q;
      }
      sv += v;
#pragma unroll
      for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
      if (lane == 0) piece[s * kWarps + warp] = v;
    }
    // what was taken out of P belongs to the sum of its exponentials
    if (op == OP_SUMS && rank == 0 && tid == 0)
      for (int k = 0; k < n_gone; ++k) full += S.p[S.gone[k]];
    const int slot = turn++ & 1;
    for (int y = 0; y < 2; ++y) {
      double x = y ? sq : sv;
#pragma unroll
      for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      if (lane == 0) S.warp_sum[warp] = x;
      __syncthreads();
      if (tid < (int)C) {
        double t = 0.0;
        for (int k = 0; k < kWarps; ++k) t += S.warp_sum[k];
        st_peer_f64(mapa(smem_u32(&S.sums[slot][y][rank]), tid), t);
      }
      __syncthreads();
    }
    if (tid < (int)C) st_peer_f64(mapa(smem_u32(&S.sums[slot][2][rank]), tid), __shfl_sync((1u << C) - 1u, full, 0));
    cluster_sync();
    if (tid == 0) {
      double t[3] = {0.0, 0.0, 0.0};
      for (int y = 0; y < 3; ++y)
        for (int k = 0; k < (int)C; ++k) t[y] += S.sums[slot][y][k];
      S.total[0] = t[0];
      if (op == OP_SUMS) {
        S.ZP = t[0] + t[2], S.ZQ = t[1];
        exact = true;
        summed = true;
      } else if (op == OP_AGAIN) {
        summed = true;
      } else {
        // (a sum that is NaN counts as something: the draw then finds no distribution)
        summed = !(t[0] <= 0.0);
        if (summed) S.Z[S.rounds++] = t[0];  // else nothing would be left: P stays
        ++c;  // this child is dealt with
      }
    }
    __syncthreads();
  }

  // ---- the draw: `piece` and S.sums hold the final P, unscaled, in order ----
  if (tid == 0 && rank == 0) {
    for (int k = depth; k < n; ++k) path[k] = -1;
    if (depth > 0) path[0] = 0;
    P.n_path[b] = depth;
  }
  if (greedy || nn == 0) {
    if (tid == 0 && rank == 0) P.next_token[b] = nn > 0 && S.idx[S.cur] < V ? S.idx[S.cur] : -1;
  } else {
    const int slot = (turn - 1) & 1;
    const double total = S.total[0], want = P.r[b] > 0.f ? (double)P.r[b] * total : 0.0;
    double before = 0.0;  // of the blocks before this one
    for (int k = 0; k < (int)rank; ++k) before += S.sums[slot][0][k];
    const double mine = S.sums[slot][0][rank];
    int last = -1;  // the last block with any P: takes what rounding leaves over
    for (int k = 0; k < (int)C; ++k)
      if (S.sums[slot][0][k] > 0.0) last = k;
    const bool fits = total > 0.0 && total < INFINITY;
    if (!fits) {
      if (tid == 0 && rank == 0) P.next_token[b] = -1;  // no distribution
    } else if (warp == 0 && before <= want && (before + mine > want || (int)rank == last) && mine > 0.0) {
      // pieces of 128 elements, then the elements of one piece
      const int n_piece = (hi - lo + kPass - 1) / kPass * kWarps;
      int at = -1;
      double base = before, sure = before;
      int keep = -1;
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
      const T* tp = target + S.cur * P.t_node;
      const T* dp = draft + (sampled ? S.cur * P.d_node : 0);
      const double mp = (double)S.m[0][S.cur] * tc, mq = sampled ? (double)S.m[1][S.cur] * dc : 0.0;
      double v[4], sum = 0.0;
      const int j = lo + at / kWarps * kPass + at % kWarps * 128 + lane * 4;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = 0.0;
        if (j + k < hi) {
          v[k] = exp2_table(fma((double)to_f(tp[j + k]), tc, -mp), S.table);
          if (rounds > 0) {
            const double qq = exp2_table(fma((double)to_f(dp[j + k]), dc, -mq), S.table) * (1.0 / S.ZQ);
            v[k] *= 1.0 / S.ZP;
            for (int y = 0; y < rounds - 1; ++y) v[k] = fmax(v[k] - qq, 0.0) / S.Z[y];
            v[k] = fmax(v[k] - qq, 0.0);
          } else {
            for (int y = 0; y < S.n_gone; ++y)
              if (S.token[S.gone[y]] == j + k) v[k] = 0.0;
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
      int mineat = 0x7fffffff, lastat = -1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        run += v[k];
        if (v[k] > 0.0) {
          lastat = j + k;
          if (run > want && mineat == 0x7fffffff) mineat = j + k;
        }
      }
#pragma unroll
      for (int off = 16; off; off >>= 1) {
        mineat = min(mineat, __shfl_xor_sync(0xffffffffu, mineat, off));
        lastat = max(lastat, __shfl_xor_sync(0xffffffffu, lastat, off));
      }
      if (lane == 0) P.next_token[b] = mineat != 0x7fffffff ? mineat : lastat;
    }
  }
  cluster_sync();  // no block leaves while a peer may still store into it
}

}  // namespace verify

size_t tree_verify_workspace_bytes(int B, int n, int V) {
  const int chunks = (V + 8 + verify::kChunk - 1) / verify::kChunk;
  return (size_t)2 * B * n * chunks * sizeof(verify::Stat);
}

template <typename T>
static cudaError_t verify_launch(const verify::Params& P, cudaStream_t stream) {
  using namespace verify;
  static std::atomic<int> largest[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  row_stats<T><<<dim3(P.chunks, P.B * P.n, P.draft ? 2 : 1), kStatThreads, 0, stream>>>(P);
  e = cudaGetLastError();
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
    e = cudaFuncSetAttribute(walk<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(walk<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
    if (e != cudaSuccess) return e;
    cfg.numAttrs = 1;
    attr[0].val.clusterDim.x = kMaxCluster;
    cfg.gridDim = dim3(kMaxCluster);
    int fit = 0;
    if (cudaOccupancyMaxActiveClusters(&fit, walk<T>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      fit = 0;
    }
    most = fit >= 1 ? kMaxCluster : 8;
    if (dev < 64) largest[dev].store(most);
  }
  // A sequence's walk waits for its own passes: as many blocks as the batch leaves room for.
  int C = P.B * 16 <= 128 ? most : 8;
  while (C > 1 && (int64_t)(C - 1) * kPass >= P.V) C /= 2;
  const int slice = ((P.V + C - 1) / C + 3) & ~3;
  cfg.dynamicSmemBytes = (size_t)(slice + kPass - 1) / kPass * kWarps * sizeof(double);
  if (cfg.dynamicSmemBytes > 128 * 1024) return cudaErrorInvalidValue;
  attr[0].val.clusterDim.x = C;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3(C * P.B);
  return cudaLaunchKernelEx(&cfg, walk<T>, P);
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
  const cudaError_t e = a.dtype == MK_FP32   ? verify_launch<float>(P, stream)
                        : a.dtype == MK_BF16 ? verify_launch<__nv_bfloat16>(P, stream)
                                             : verify_launch<__half>(P, stream);
  if (e != cudaSuccess) {
    *err = std::string("tree_verify launch: ") + cudaGetErrorString(e);
    return MK_ERR_CUDA;
  }
  return MK_OK;
}

}  // namespace mk
