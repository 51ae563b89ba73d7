// Verification of drafted tokens against the target's probabilities, and the draw of the next token.
//
// At a node with target P and draft Q a child x is accepted with probability min(1, R(x) / Q(x)); a
// rejection leaves the residual R' = max(0, R - Q) / sum. With R = w / Z, w = max(0, P - a Q):
//   max(0, R - Q) = max(0, w - Z Q) / Z = max(0, P - (a + Z) Q) / Z     (Q >= 0),
// so a node's state is the two numbers a and Z, and only a rejection costs a pass over the vocabulary,
// for Z. Point masses: w is P without the rejected tokens and Z needs no pass at all. The draw is the
// lowest v with w(0) + .. + w(v) > u sum w; its sums are those of the last pass where the path ended in
// a rejection.
//
// Borders between neighbouring tokens lie as close as their probabilities are small, so sums are kept in
// two floats (error-free additions, 2^-46 and better; fp64 adds run at 1/64 of the rate here) and joined
// in fp64: the result does not depend on the split. w is P - a Q in two floats likewise.
//
// A cluster of blocks takes a request, a block a contiguous slice of the vocabulary, a warp chunks of it;
// each chunk's sum stays in shared memory, so that the draw reads only one chunk again. Every block walks
// the tree by itself (a few dependent steps over numbers gathered once); block totals cross by distributed
// shared memory. Without sampling the passes are arg-max passes, one for each node of the path.
// Bound: latency with few requests, HBM (P and Q rows once) with many.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_common.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxNodes = 64;
constexpr int kMaxChunks = 1024;   // of a block
constexpr int kMaxCluster = 8;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

// a sum in two floats: hi + lo, lo what hi's roundings left
struct Sum2 {
  float hi, lo;
  __device__ __forceinline__ void add(float x, float y) {  // x + y, |y| small beside x
    const float h = __fadd_rn(hi, x), b = __fsub_rn(h, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(__fsub_rn(hi, __fsub_rn(h, b)), __fsub_rn(x, b)), y));
    hi = h;
  }
  __device__ __forceinline__ void shuffle_add(int off) {
    const float x = __shfl_xor_sync(0xFFFFFFFFu, hi, off), y = __shfl_xor_sync(0xFFFFFFFFu, lo, off);
    add(x, y);
  }
  __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

// a, in two floats
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two split(double x) {
  Two t;
  t.hi = (float)x;
  t.lo = (float)(x - (double)t.hi);
  return t;
}
// w = max(0, p - a q) in two floats
__device__ __forceinline__ Two weight(float p, float q, Two a) {
  const float h = __fmul_rn(a.hi, q), l = __fmaf_rn(a.lo, q, __fmaf_rn(a.hi, q, -h));  // a q = h + l
  const float d = __fsub_rn(p, h), b = __fsub_rn(d, p);
  const float e = __fsub_rn(__fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(h, b)), l);  // what d's rounding left, and l
  const float s = __fadd_rn(d, e);
  if (!(s > 0.f)) return {0.f, 0.f};
  return {s, __fsub_rn(e, __fsub_rn(s, d))};
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void store_remote(void* p, uint32_t rank, uint64_t v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.b64 [a], %2;\n\t}" ::"r"(smem_u32(p)),
      "r"(rank), "l"(v)
      : "memory");
}

// Entries v .. v + 3 of a row, 0 from `end` on. wide: the row's address and v allow one load.
template <typename T>
__device__ __forceinline__ void load4(const T* row, int v, int end, bool wide, float (&x)[4]) {
  if (wide && v + 4 <= end) {
    if constexpr (sizeof(T) == 4) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(row + v));
      x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
    } else {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(row + v));
      T t[4];
      *reinterpret_cast<uint2*>(t) = u;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = to_f(t[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = v + i < end ? to_f(row[v + i]) : 0.f;
  }
}

struct Shared {
  double chunk[kMaxChunks];
  uint64_t total[2][kMaxCluster];  // of the cluster's blocks, by turns
  double part[kWarps];
  float pz[kMaxNodes], qz[kMaxNodes], u[kMaxNodes];
  int token[kMaxNodes], parent[kMaxNodes], path[kMaxNodes], gone[kMaxNodes];
  int bad, node, count, n_gone, at, pass, found;
  double a, z, target;
  uint64_t best[kWarps];
};

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a) {
  __shared__ Shared s;
  const int C = gridDim.x / a.B;
  const int b = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = C > 1 ? cluster_rank() : 0;
  const int nd = a.n_draft ? min(max(a.n_draft[b], 0), a.N) : a.N;
  if (nd == 0) {  // the whole cluster
    if (rank == 0 && tid == 0) a.n_accept[b] = 0;
    return;
  }
  const T* P = static_cast<const T*>(a.p) + b * a.p_sb;
  const T* Q = a.q ? static_cast<const T*>(a.q) + b * a.q_sb : nullptr;
  if (tid == 0) s.bad = 0;
  __syncthreads();
  if (tid < nd) {
    const int i = tid, x = a.token[(size_t)b * a.N + i], par = i ? a.parent[(size_t)b * a.N + i] : 0;
    const bool ok = x >= 0 && x < a.V && par >= 0 && (i == 0 || par < i);
    if (!ok) s.bad = 1;
    s.token[i] = x;
    s.parent[i] = i ? par : -1;
    s.u[i] = a.u ? a.u[(size_t)b * a.N + i] : 0.f;
    if (ok && i && a.u) {
      s.pz[i] = to_f(P[par * a.p_st + x]);
      s.qz[i] = Q ? to_f(Q[par * a.q_st + x]) : 1.f;
    }
  }
  __syncthreads();
  if (s.bad) {
    if (rank == 0 && tid == 0) {
      a.n_accept[b] = 0;
      set_error(a.err, KVQ_ERR_INVALID_ARG);
    }
    return;
  }
  if (C > 1) cluster_sync();  // every block's shared memory is there
  const int v0 = min(a.V, (int)rank * a.slice), v1 = min(a.V, v0 + a.slice);
  const int n_chunks = (v1 - v0 + a.chunk - 1) / a.chunk;
  int turn = 0;
  auto share = [&](uint64_t mine) {  // this block's value to every block; all values in s.total[turn]
    if (C > 1) {
      if (tid < C) store_remote(&s.total[turn][rank], tid, mine);
      cluster_sync();
    } else {
      if (tid == 0) s.total[turn][0] = mine;
      __syncthreads();
    }
  };

  if (!a.u) {
    // ---- no sampling: the arg max of each node of the path ----
    int node = 0, count = 1, best = 0;
    if (tid == 0) s.path[0] = 0;
    for (;;) {
      const T* row = P + node * a.p_st;
      const bool wide = (reinterpret_cast<uintptr_t>(row) & (4 * sizeof(T) - 1)) == 0;  // v0 is a multiple of 4
      float top = -INFINITY;
      int at = 0x7FFFFFFF;
      constexpr int kAhead = 4;
      for (int v = v0 + 4 * tid; v < v1; v += 4 * kThreads * kAhead) {
        float x[kAhead][4];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) load4(row, v + 4 * kThreads * k, v1, wide, x[k]);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = v + 4 * kThreads * k + e;
            if (i < v1 && x[k][e] > top) {
              top = x[k][e];
              at = i;
            }
          }
      }
      // one number that is larger for larger values and, of equal ones, lower indices
      const uint32_t f = __float_as_uint(top + 0.f);  // -0 counts as 0
      uint64_t key = ((uint64_t)((f & 0x80000000u) ? ~f : f | 0x80000000u) << 32) | (0x7FFFFFFFu - (uint32_t)at);
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, off));
      if (lane == 0) s.best[warp] = key;
      __syncthreads();
      for (int w = 0; w < kWarps; ++w) key = max(key, s.best[w]);
      share(key);
      key = s.total[turn][0];
      for (int r = 1; r < C; ++r) key = max(key, s.total[turn][r]);
      turn ^= 1;
      best = (int)(0x7FFFFFFFu - (uint32_t)key);
      if (best == 0x7FFFFFFF) best = 0;  // nothing above the lowest value
      int next = 0;
      for (int i = node + 1; i < nd && !next; ++i)
        if (s.parent[i] == node && s.token[i] == best) next = i;
      if (!next) break;
      node = next;
      if (tid == 0) s.path[count] = next;
      ++count;
    }
    if (rank == 0) {
      __syncthreads();
      if (tid < count) a.path[(size_t)b * a.N + tid] = s.path[tid];
      if (tid == 0) {
        a.n_accept[b] = count;
        a.next[b] = best;
      }
    }
    if (C > 1) cluster_sync();  // nobody leaves while its shared memory is written
    return;
  }

  // ---- sampling ----
  if (tid == 0) {
    s.path[0] = 0;
    s.node = 0;
    s.count = 1;
    s.n_gone = 0;
    s.at = 1;
    s.a = 0.0;
    s.z = 1.0;
  }
  int fallback = 0;
  for (;;) {
    __syncthreads();
    if (tid == 0) {  // on until a pass is needed: after a rejection against Q, or at the end
      s.pass = 0;
      for (; s.at < nd; ++s.at) {
        const int i = s.at;
        if (s.parent[i] != s.node) continue;
        const float q = s.qz[i];
        bool gone = false;
        for (int k = 0; k < s.n_gone; ++k) gone = gone || s.gone[k] == s.token[i];
        double w = (double)s.pz[i];
        if (Q) w = fmax(w - s.a * (double)q, 0.0);
        else if (gone) w = 0.0;
        if ((double)s.u[i] * s.z * (double)q < w) {
          s.path[s.count++] = i;
          s.node = i;
          s.a = 0.0;
          s.z = 1.0;
          s.n_gone = 0;
        } else if (Q) {
          s.a += s.z;
          s.pass = 1;
          ++s.at;
          break;
        } else {
          s.z -= w;
          s.gone[s.n_gone++] = s.token[i];
        }
      }
      if (fallback) {
        s.a = 0.0;
        s.n_gone = 0;
      }
    }
    __syncthreads();
    const bool rejected = s.pass;  // else this pass is the draw's
    const T* row = P + s.node * a.p_st;
    const T* qrow = Q && s.a > 0.0 ? Q + s.node * a.q_st : nullptr;
    const bool wide = (reinterpret_cast<uintptr_t>(row) & (4 * sizeof(T) - 1)) == 0 &&
                      (!qrow || (reinterpret_cast<uintptr_t>(qrow) & (4 * sizeof(T) - 1)) == 0);
    const Two f = split(s.a);
    const int n_gone = s.n_gone;
    auto is_gone = [&](int v) {
      for (int k = 0; k < n_gone; ++k)
        if (s.gone[k] == v) return true;
      return false;
    };
    // ---- sums of w over the block's chunks ----
    for (int c = warp; c < n_chunks; c += kWarps) {
      const int c0 = v0 + c * a.chunk, c1 = min(v1, c0 + a.chunk);
      bool some_gone = false;
      for (int k = lane; k < n_gone; k += 32) some_gone = some_gone || (s.gone[k] >= c0 && s.gone[k] < c1);
      some_gone = __any_sync(0xFFFFFFFFu, some_gone);
      Sum2 sum = {0.f, 0.f};
      for (int v = c0 + 4 * lane; v < c1; v += 512) {
        float p[4][4], q[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) load4(row, v + 128 * k, c1, wide, p[k]);
        if (qrow) {
#pragma unroll
          for (int k = 0; k < 4; ++k) load4(qrow, v + 128 * k, c1, wide, q[k]);
        }
        if (some_gone) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (is_gone(v + 128 * k + e)) p[k][e] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (qrow) {
              const Two w = weight(p[k][e], q[k][e], f);
              sum.add(w.hi, w.lo);
            } else {
              sum.add(p[k][e], 0.f);
            }
          }
      }
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) sum.shuffle_add(off);
      if (lane == 0) s.chunk[c] = sum.value();
    }
    __syncthreads();
    double mine = 0.0;
    for (int c = tid; c < n_chunks; c += kThreads) mine += s.chunk[c];
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, off);
    if (lane == 0) s.part[warp] = mine;
    __syncthreads();
    mine = 0.0;
    for (int w = 0; w < kWarps; ++w) mine += s.part[w];
    share(__double_as_longlong(mine));
    double total = 0.0, before = 0.0;
    for (int r = 0; r < C; ++r) {
      if (r == (int)rank) before = total;
      total += __longlong_as_double(s.total[turn][r]);
    }
    turn ^= 1;
    if (rejected) {
      // the walk goes on if a later child of this node is left to test; else these are the draw's sums
      bool more = false;
      for (int i = s.at; i < nd; ++i) more = more || s.parent[i] == s.node;
      if (more) {
        __syncthreads();
        if (tid == 0) s.z = total;
        continue;
      }
    }
    if (!(total > 0.0) && !fallback) {
      fallback = 1;
      continue;
    }
    // ---- the draw: the block, the chunk, the entry in which the sums pass u total ----
    const double target = (double)s.u[0] * total;
    // each block's end is the next one's beginning, so exactly one holds the target
    if (rank == 0 && tid < s.count) a.path[(size_t)b * a.N + tid] = s.path[tid];
    if (rank == 0 && tid == 0) a.n_accept[b] = s.count;
    const bool none = !(total > 0.0);  // of a row without mass any token does
    if (none && rank == 0 && tid == 0) a.next[b] = 0;
    double end = 0.0;
    bool earlier = false;
    for (int r = 0; r <= (int)rank; ++r) {
      end += __longlong_as_double(s.total[turn ^ 1][r]);
      if (r < (int)rank) earlier = earlier || end > target;
    }
    if (!none && !earlier && end > target && warp == 0) {
      int c = 0;
      double base = before;
      for (; c + 1 < n_chunks; ++c) {
        const double e = base + s.chunk[c];
        if (e > target) break;
        base = e;
      }
      const int c0 = v0 + c * a.chunk, c1 = min(v1, c0 + a.chunk);
      int last = c0;  // the last entry with a weight, should roundings leave none past the target
      int found = -1;
      for (int v = c0 + 4 * lane; v - 4 * lane < c1 && found < 0; v += 128) {
        float p[4], q[4];
        load4(row, v, c1, wide, p);
        if (qrow) load4(qrow, v, c1, wide, q);
        double w[4], run = 0.0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (n_gone && is_gone(v + e)) p[e] = 0.f;
          Two t = {p[e], 0.f};
          if (qrow) t = weight(p[e], q[e], f);
          w[e] = (double)t.hi + (double)t.lo;
          run += w[e];
          if (w[e] > 0.0) last = max(last, v + e);
        }
        double upto = run;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const double y = __shfl_up_sync(0xFFFFFFFFu, upto, off);
          if (lane >= off) upto += y;
        }
        const unsigned past = __ballot_sync(0xFFFFFFFFu, base + upto > target);
        if (past) {
          const int src = __ffs(past) - 1;
          double at = base + (upto - run);
          int hit = v;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (w[e] > 0.0) hit = v + e;
#pragma unroll
          for (int e = 3; e >= 0; --e) {
            double x = at;
            for (int k = 0; k <= e; ++k) x += w[k];
            if (x > target) hit = v + e;
          }
          found = __shfl_sync(0xFFFFFFFFu, hit, src);
        }
        base += __shfl_sync(0xFFFFFFFFu, upto, 31);
      }
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) last = max(last, __shfl_xor_sync(0xFFFFFFFFu, last, off));
      if (lane == 0) a.next[b] = found >= 0 ? found : last;
    }
    break;
  }
  if (C > 1) cluster_sync();  // nobody leaves while its shared memory is written
}

template <typename T>
cudaError_t launch_typed(const VerifyArgs& args, cudaStream_t st) {
  VerifyArgs a = args;
  int C = 1;
  while (C < kMaxCluster && a.B * C * 2 <= 2 * device_sms() && a.V / (2 * C) >= 2048) C *= 2;
  a.slice = ((a.V + C - 1) / C + 511) / 512 * 512;
  a.chunk = 512;
  while ((a.slice + a.chunk - 1) / a.chunk > kMaxChunks) a.chunk *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = (unsigned)(a.B * C);
  cfg.blockDim = kThreads;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int dtype, cudaStream_t st) {
  if (dtype == KVQ_DT_FP32) return launch_typed<float>(a, st);
  if (dtype == KVQ_DT_BF16) return launch_typed<__nv_bfloat16>(a, st);
  return launch_typed<__half>(a, st);
}

}  // namespace kvq
