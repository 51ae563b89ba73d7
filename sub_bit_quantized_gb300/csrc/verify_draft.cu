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
// Bound: latency. With few requests dependent steps of 1 - 2 us (nodes, their numbers, a row, the cluster's barrier, the draw; one
// chain of 32768 entries 8 us, trees of 50021 14 - 20). With many: 64 chains of 131072 fp32 entries take 25 us, 65 MB at 38 % of
// the copy rate; 9.2 M instructions are 39 % of the issue slots while SMs are active, FMA 29 %, ALU 24 %. 256 blocks of at most two
// an SM leave 22 % of the warps and SMs active 74 % of the launch, too few loads on their way for HBM.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kvq_common.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kMaxNodes = 64;
constexpr int kMaxChunks = 1024;   // of a block
constexpr int kMaxCluster = 8;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

// A number in two floats, lo what hi's rounding left: sums and products are off by 2^-45 of themselves at most. (fp64
// operations run at 1/64 of the rate here and take a warp some hundred cycles each in a row.)
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two norm(float h, float l) {  // |l| <= |h|
  const float s = __fadd_rn(h, l);
  return {s, __fsub_rn(l, __fsub_rn(s, h))};
}
__device__ __forceinline__ Two plus(Two x, Two y) {
  const float h = __fadd_rn(x.hi, y.hi), b = __fsub_rn(h, x.hi);
  const float e = __fadd_rn(__fsub_rn(x.hi, __fsub_rn(h, b)), __fsub_rn(y.hi, b));
  return norm(h, __fadd_rn(e, __fadd_rn(x.lo, y.lo)));
}
__device__ __forceinline__ Two minus(Two x, Two y) { return plus(x, {-y.hi, -y.lo}); }
__device__ __forceinline__ Two times(Two x, Two y) {
  const float h = __fmul_rn(x.hi, y.hi);
  return norm(h, __fadd_rn(__fmaf_rn(x.hi, y.hi, -h), __fmaf_rn(x.hi, y.lo, __fmul_rn(x.lo, y.hi))));
}
__device__ __forceinline__ bool less(Two x, Two y) { return x.hi < y.hi || (x.hi == y.hi && x.lo < y.lo); }
__device__ __forceinline__ Two shfl(Two x, int lane) {
  return {__shfl_sync(0xFFFFFFFFu, x.hi, lane), __shfl_sync(0xFFFFFFFFu, x.lo, lane)};
}
// the sums of lanes 0 .. lane, of `lanes` lanes
__device__ __forceinline__ Two scan(Two x, int lane, int lanes) {
  for (int off = 1; off < lanes; off <<= 1) {
    const Two y = {__shfl_up_sync(0xFFFFFFFFu, x.hi, off), __shfl_up_sync(0xFFFFFFFFu, x.lo, off)};
    if (lane >= off) x = plus(y, x);
  }
  return x;
}
__device__ __forceinline__ uint64_t bits(Two x) { return (uint64_t)__float_as_uint(x.hi) << 32 | __float_as_uint(x.lo); }
__device__ __forceinline__ Two two(uint64_t b) { return {__uint_as_float((uint32_t)(b >> 32)), __uint_as_float((uint32_t)b)}; }

__device__ __forceinline__ float2 f2(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 neg2(float2 x) { return make_float2(-x.x, -x.y); }
__device__ __forceinline__ float2 sub2(float2 x, float2 y) { return __fadd2_rn(x, neg2(y)); }

// Two sums, each in two floats: hi + lo, lo what hi's roundings left
struct Sum2 {
  float2 hi, lo;
  __device__ __forceinline__ void add(float2 x) {
    const float2 h = __fadd2_rn(hi, x), b = sub2(h, hi);
    lo = __fadd2_rn(lo, __fadd2_rn(sub2(hi, sub2(h, b)), sub2(x, b)));
    hi = h;
  }
  __device__ __forceinline__ Two total() const { return plus(norm(hi.x, lo.x), norm(hi.y, lo.y)); }
};
__device__ __forceinline__ Two warp_sum(Two x) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) x = plus(x, {__shfl_xor_sync(0xFFFFFFFFu, x.hi, off), __shfl_xor_sync(0xFFFFFFFFu, x.lo, off)});
  return x;
}

// w = max(0, p - a q) of two entries, not normalised: hi + lo. a q = h + l; where p - h is not negative, or small beside
// them, what its rounding left is (p - d) - h.
struct Weight2 {
  float2 hi, lo;
};
__device__ __forceinline__ Weight2 weight(float2 p, float2 q, float a_hi, float a_lo) {
  const float2 h = __fmul2_rn(f2(a_hi), q), l = __ffma2_rn(f2(a_lo), q, __ffma2_rn(f2(a_hi), q, neg2(h)));
  const float2 d = sub2(p, h), e = sub2(sub2(sub2(p, d), h), l), s = __fadd2_rn(d, e);
  Weight2 w;
  w.hi = make_float2(s.x > 0.f ? d.x : 0.f, s.y > 0.f ? d.y : 0.f);
  w.lo = make_float2(s.x > 0.f ? e.x : 0.f, s.y > 0.f ? e.y : 0.f);
  return w;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// the same in two steps: every block's shared memory is there behind the second
__device__ __forceinline__ void cluster_begin() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_began() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void store_remote(void* p, uint32_t rank, uint64_t v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.b64 [a], %2;\n\t}" ::"r"(smem_u32(p)),
      "r"(rank), "l"(v)
      : "memory");
}

// Eight entries of a row for a lane, 0 from `end` on, as they lie in memory: converted where they are used, or the conversion
// would wait for the loads that are to be on their way meanwhile (64 chains of 131072 bf16 entries 51 us). wide (the row's
// address allows it): entries 4 k + e are at v + 128 k + 4 lane + e, in loads of four, 16-bit ones two a word; else entry j is
// at v + 32 j + lane, one by one, so that a warp's loads stay contiguous at any alignment.
constexpr int kStep = 256;  // entries of a warp's step
template <typename T>
__device__ __forceinline__ uint32_t raw(T x) {
  if constexpr (sizeof(T) == 4) return __float_as_uint(x);
  else return *reinterpret_cast<const uint16_t*>(&x);
}
template <typename T>
__device__ __forceinline__ void load8(const T* row, int v, int end, int lane, bool wide, uint32_t (&w)[8]) {
  if (wide) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int at = v + 128 * k + 4 * lane;
      if (at + 4 <= end) {
        if constexpr (sizeof(T) == 4) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + at));
          w[4 * k] = u.x; w[4 * k + 1] = u.y; w[4 * k + 2] = u.z; w[4 * k + 3] = u.w;
        } else {
          const uint2 u = __ldg(reinterpret_cast<const uint2*>(row + at));
          w[2 * k] = u.x; w[2 * k + 1] = u.y;
        }
      } else {
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = at + e < end ? raw(row[at + e]) : 0u;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[4 * k + e] = y[e];
        } else {
          w[2 * k] = y[0] | y[1] << 16;
          w[2 * k + 1] = y[2] | y[3] << 16;
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = v + 32 * j + lane;
      w[j] = at < end ? raw(row[at]) : 0u;
    }
  }
}
// entries 2 i, 2 i + 1 of them
template <typename T>
__device__ __forceinline__ float2 pair_of(const uint32_t (&w)[8], int i, bool wide) {
  if constexpr (sizeof(T) == 4) {
    return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  } else {
    const uint32_t u = wide ? w[i] : __byte_perm(w[2 * i], w[2 * i + 1], 0x5410);
    if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&u));
    else return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  }
}
// which entry that is
__device__ __forceinline__ int entry8(int v, int j, int lane, bool wide) {
  return wide ? v + 128 * (j >> 2) + 4 * lane + (j & 3) : v + 32 * j + lane;
}

// Of the cluster's blocks, by turns: what each found
struct Exchange {
  uint64_t total[2][kMaxCluster];
};
// The nodes of a request: lane l of every warp holds nodes l and l + 32
struct Nodes {
  int token[2], parent[2];
  // Of nd nodes; those that count have a parent before them and a token of the vocabulary. false: some has not (every
  // warp of every block sees the same).
  __device__ __forceinline__ bool load(const VerifyArgs& a, int b, int nd, int lane) {
    bool ok = true;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = lane + 32 * h;
      token[h] = parent[h] = -1;
      if (i < a.N) {
        token[h] = a.token[(size_t)b * a.N + i];
        parent[h] = a.parent[(size_t)b * a.N + i];
      }
      if (i >= nd) token[h] = parent[h] = -1;
      else ok = ok && token[h] >= 0 && token[h] < a.V && (i == 0 || (parent[h] >= 0 && parent[h] < i));
      if (i == 0) parent[h] = -1;
    }
    return __all_sync(0xFFFFFFFFu, ok) != 0;
  }
  // bit i: node i >= from is a child of `node` (and its token is x)
  __device__ __forceinline__ uint64_t children(int node, int from) const {
    const uint64_t m = (uint64_t)__ballot_sync(0xFFFFFFFFu, parent[0] == node) |
                       (uint64_t)__ballot_sync(0xFFFFFFFFu, parent[1] == node) << 32;
    return from >= 64 ? 0ull : m >> from << from;
  }
  __device__ __forceinline__ uint64_t say(int x) const {
    return (uint64_t)__ballot_sync(0xFFFFFFFFu, token[0] == x) | (uint64_t)__ballot_sync(0xFFFFFFFFu, token[1] == x) << 32;
  }
};
template <typename V>
__device__ __forceinline__ V of_node(const V (&x)[2], int i) {
  const V lo = __shfl_sync(0xFFFFFFFFu, x[0], i & 31), hi = __shfl_sync(0xFFFFFFFFu, x[1], i & 31);
  return i < 32 ? lo : hi;
}

// A request of a kernel's cluster and the block's slice of the vocabulary
template <typename T>
struct Part {
  int C, b, v0, v1, turn;
  uint32_t rank;
  bool began;
  const T* P;
  __device__ __forceinline__ explicit Part(const VerifyArgs& a) {
    C = a.blocks;
    b = blockIdx.x / C;
    rank = C > 1 ? cluster_rank() : 0;
    if (C > 1) cluster_begin();
    began = C == 1;
    P = static_cast<const T*>(a.p) + b * a.p_sb;
    v0 = min(a.V, (int)rank * a.slice);
    v1 = min(a.V, v0 + a.slice);
    turn = 0;
  }
  __device__ __forceinline__ void begin() {  // before this block's first access to the others' memory
    if (!began) cluster_began();
    began = true;
  }
  __device__ __forceinline__ void wait() {
    if (C > 1) cluster_sync();
    else __syncthreads();
  }
  // a request without nodes, or with bad ones: the whole cluster leaves
  __device__ __forceinline__ void leave(const VerifyArgs& a, int nd) {
    begin();
    if (rank == 0 && threadIdx.x == 0) {
      a.n_accept[b] = 0;
      if (nd > 0) set_error(a.err, KVQ_ERR_INVALID_ARG);
    }
  }
};

// ---- no sampling: the arg max of each node of the path ----
// The larger of the entries of a 16-byte piece, NaN left out
__device__ __forceinline__ float piece_max(const float4& x) { return fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)); }
template <typename T2>
__device__ __forceinline__ T2 pairs_max(const uint4& u) {
  const T2* t = reinterpret_cast<const T2*>(&u);
  return __hmax2(__hmax2(t[0], t[1]), __hmax2(t[2], t[3]));
}
template <typename T>
__device__ __forceinline__ float piece_max(const uint4& u) {
  if constexpr (sizeof(T) == 4) {
    return piece_max(*reinterpret_cast<const float4*>(&u));
  } else if constexpr (std::is_same<T, __half>::value) {
    const float2 m = __half22float2(pairs_max<__half2>(u));
    return fmaxf(m.x, m.y);
  } else {
    const float2 m = __bfloat1622float2(pairs_max<__nv_bfloat162>(u));
    return fmaxf(m.x, m.y);
  }
}

// A pass reads two rows, the node's and its first child's, each by half of the block: most likely the path goes on there,
// and then the pass has decided two nodes. Threads keep the largest 16-byte piece that they met and look into it at the end.
// 32 trees of 131072 bf16 entries: 27.6 us with a row a pass, 22.5 with two; 16 chains of 50021 fp16 33 and 20.5 (most rows
// there begin off 16 bytes). Two and eight pieces in flight a thread: 26.6 and 28.7; the next pass's row to L2 meanwhile: no
// gain, and 51 us for 31 where few drafts are accepted.
constexpr int kGreedyThreads = 512;
template <typename T>
__global__ void __launch_bounds__(kGreedyThreads, 2) verify_greedy_kernel(const VerifyArgs a) {
  constexpr int kThreads = kGreedyThreads / 2, kWarps = kThreads / 32;  // of a row
  __shared__ uint64_t all[2][2][kMaxCluster];  // by turns: of each row, what each block found
  __shared__ uint64_t best_of[2][kWarps];
  __shared__ int path[kMaxNodes];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = warp / kWarps, t = tid & (kThreads - 1);
  Part<T> part(a);
  const int b = part.b, C = part.C, v0 = part.v0, v1 = part.v1;
  const T* P = part.P;
  const int nd = a.n_draft ? min(max(a.n_draft[b], 0), a.N) : a.N;
  Nodes nodes;
  const bool ok = nodes.load(a, b, nd, lane);
  if (nd == 0 || !ok) return part.leave(a, nd);
  int node = 0, count = 1, best = 0;
  if (tid == 0) path[0] = 0;
  for (;;) {
    const uint64_t kids = nodes.children(node, node + 1);
    const int child = kids ? __ffsll(kids) - 1 : node;  // a leaf's row is halved instead
    const int mid = kids ? v1 : min(v1, v0 + (v1 - v0 + 1023) / 1024 * 512);
    const T* row = P + (r ? child : node) * a.p_st;
    const int from = !kids && r ? mid : v0, to = r ? v1 : mid;
    // whole 16-byte pieces from s on; single entries before and behind them
    constexpr int kLoad = 16 / (int)sizeof(T), kNone = 0x7FFFFFFF, kAhead = 4;
    const int off = (int)(reinterpret_cast<uintptr_t>(row + from) & 15) / (int)sizeof(T);
    const int s = min(to, from + (off ? kLoad - off : 0)), pieces = (to - s) / kLoad, e = s + pieces * kLoad + t;
    const float first = from + t < s ? to_f(row[from + t]) : -INFINITY, last = e < to ? to_f(row[e]) : -INFINITY;
    const uint4* wide = reinterpret_cast<const uint4*>(row + s);
    float top = -INFINITY;
    int at = kNone;
    uint4 piece = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
    for (int k0 = t; k0 < pieces; k0 += kAhead * kThreads) {
      uint4 u[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k0 + k * kThreads < pieces) u[k] = __ldg(wide + k0 + k * kThreads);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float m = k0 + k * kThreads < pieces ? piece_max<T>(u[k]) : -INFINITY;
        if (m > top) {
          top = m;
          at = k0 + k * kThreads;
          piece = u[k];
        }
      }
    }
    if (at != kNone) {
      const T* x = reinterpret_cast<const T*>(&piece);
      int in = 0;
#pragma unroll
      for (int i = kLoad - 1; i >= 0; --i)
        if (to_f(x[i]) == top) in = i;
      at = s + at * kLoad + in;
    }
    if (last > top) {
      top = last;
      at = e;
    }
    if (first > top || (first == top && at != kNone)) {  // before all others
      top = first;
      at = from + t;
    }
    // one number that is larger for larger values and, of equal ones, lower indices
    const uint32_t f = __float_as_uint(top + 0.f);  // -0 counts as 0
    uint64_t key = ((uint64_t)((f & 0x80000000u) ? ~f : f | 0x80000000u) << 32) | (0x7FFFFFFFu - (uint32_t)at);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, off));
    if (lane == 0) best_of[r][warp % kWarps] = key;
    part.begin();
    __syncthreads();
    // lanes 0 - 7 the first row (or half), 8 - 15 the second
    static_assert(kWarps == 8 && kMaxCluster == 8, "lanes of the two rows");
    auto join = [&](uint64_t x) {
#pragma unroll
      for (int off = 4; off >= 1; off >>= 1) x = max(x, __shfl_xor_sync(0xFFFFFFFFu, x, off));
      return x;
    };
    if (warp == 0) {
      key = join(best_of[lane >> 3 & 1][lane & 7]);
      if (lane < 16 && (lane & 7) < C) store_remote(&all[part.turn][lane >> 3][part.rank], lane & 7, key);
    }
    part.wait();
    key = lane < 16 && (lane & 7) < C ? all[part.turn][lane >> 3][lane & 7] : 0;
    key = join(key);
    part.turn ^= 1;
    uint64_t found[2] = {__shfl_sync(0xFFFFFFFFu, key, 0), __shfl_sync(0xFFFFFFFFu, key, 8)};
    if (!kids) found[0] = max(found[0], found[1]);
    auto index = [](uint64_t x) {
      const int i = (int)(0x7FFFFFFFu - (uint32_t)x);
      return i == kNone ? 0 : i;  // nothing above the lowest value
    };
    auto go_on = [&]() {  // to the child that is the arg max
      const uint64_t next = nodes.children(node, node + 1) & nodes.say(best);
      if (!next) return false;
      node = __ffsll(next) - 1;
      if (tid == 0) path[count] = node;
      ++count;
      return true;
    };
    best = index(found[0]);
    if (!go_on()) break;
    if (node == child) {
      best = index(found[1]);
      if (!go_on()) break;
    }
  }
  if (part.rank == 0 && warp == 0) {
    __syncwarp();
    for (int i = lane; i < count; i += 32) a.path[(size_t)b * a.N + i] = path[i];
    if (lane == 0) {
      a.n_accept[b] = count;
      a.next[b] = best;
    }
  }
  // the last writes into this block's memory were those that the last barrier waited for
}

// ---- sampling: warp 0 walks, all warps add ----
// THREADS a block: 512 where every block has an SM of its own, else 256 with twice the registers (128 of a thread either
// way: with 64 the pass's loads spill). Before a step's loads ran one ahead, 64 chains of 131072 entries took 33 us with 256,
// 39 with 512; 16 trees of 50021: 29 and 27; trees of points: 18 and 17.
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) verify_kernel(const VerifyArgs a) {
  constexpr int kWarps = THREADS / 32;
  __shared__ struct {
    Two chunk[kMaxChunks];
    Exchange x;
    float w[2][512 + 32];            // the drawn entries' weights in order, in two floats each (16 a lane, padded)
    int path[kMaxNodes], gone[kMaxNodes];
    int node, n_gone, done, c0, found;  // done: 1 the request is, 2 but for the draw from the chunk at c0
    float a_hi, a_lo;
  } s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Part<T> part(a);
  const int b = part.b, C = part.C, v0 = part.v0, v1 = part.v1;
  const uint32_t rank = part.rank;
  const T* P = part.P;
  const T* Q = a.q ? static_cast<const T*>(a.q) + b * a.q_sb : nullptr;
  const int nd = a.n_draft ? min(max(a.n_draft[b], 0), a.N) : a.N;
  Nodes nodes;
  const bool ok = nodes.load(a, b, nd, lane);
  if (nd == 0 || !ok) return part.leave(a, nd);
  float pz[2] = {0.f, 0.f}, qz[2] = {1.f, 1.f}, u[2] = {0.f, 0.f};
  if (warp == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = lane + 32 * h;
      if (i < nd) u[h] = a.u[(size_t)b * a.N + i];
      if (i < nd && i > 0) {
        pz[h] = to_f(P[nodes.parent[h] * a.p_st + nodes.token[h]]);
        if (Q) qz[h] = to_f(Q[nodes.parent[h] * a.q_st + nodes.token[h]]);
      }
    }
  }
  // the test of a child that is its node's first: u Q(x) < P(x)
  uint64_t at_once = 0;
  if (warp == 0) {
    bool yes[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) yes[h] = less(times({u[h], 0.f}, {qz[h], 0.f}), {pz[h], 0.f});
    at_once = (uint64_t)__ballot_sync(0xFFFFFFFFu, yes[0]) | (uint64_t)__ballot_sync(0xFFFFFFFFu, yes[1]) << 32;
  }
  const int n_chunks = (v1 - v0 + a.chunk - 1) / a.chunk;
  int node = 0, at = 1, count = 1;   // warp 0's
  uint64_t gone = 0;                 // children of the node that were rejected (point masses)
  Two wa = {0.f, 0.f}, wz = {1.f, 0.f};
  bool fallback = false;
  if (tid == 0) s.path[0] = 0;
  for (;;) {
    bool rejected = false;
    if (warp == 0) {  // on until a pass is needed: after a rejection against Q, or at the end
      for (;;) {
        const uint64_t m = nodes.children(node, at);
        if (!m || fallback) break;
        const int i = __ffsll(m) - 1;
        at = i + 1;
        if (wa.hi == 0.f && !gone && (at_once >> i & 1)) {
          if (lane == 0) s.path[count] = i;
          ++count;
          node = i;
          continue;
        }
        const float q = of_node(qz, i), p = of_node(pz, i), ui = of_node(u, i);
        Two w = {p, 0.f};
        if (Q) {
          const Weight2 y = weight(f2(p), f2(q), wa.hi, wa.lo);
          w = plus({y.hi.x, 0.f}, {y.lo.x, 0.f});
        } else if (gone && (gone & nodes.say(of_node(nodes.token, i)))) {
          w.hi = 0.f;
        }
        if (less(times(times({ui, 0.f}, {q, 0.f}), wz), w)) {
          if (lane == 0) s.path[count] = i;
          ++count;
          node = i;
          wa = {0.f, 0.f};
          wz = {1.f, 0.f};
          gone = 0;
        } else if (Q) {
          wa = plus(wa, wz);
          rejected = true;
          break;
        } else {
          wz = minus(wz, w);
          gone |= 1ull << i;
        }
      }
      const int n_lo = __popc((uint32_t)gone);
      if ((gone >> lane) & 1) s.gone[__popc((uint32_t)gone & ((1u << lane) - 1))] = nodes.token[0];
      if ((gone >> (lane + 32)) & 1) s.gone[n_lo + __popc((uint32_t)(gone >> 32) & ((1u << lane) - 1))] = nodes.token[1];
      if (lane == 0) {
        s.node = node;
        s.n_gone = __popcll(gone);
        s.a_hi = wa.hi;
        s.a_lo = wa.lo;
        s.done = 0;
      }
    }
    __syncthreads();
    const T* row = P + s.node * a.p_st;
    const float a_hi = s.a_hi, a_lo = s.a_lo;
    const T* qrow = Q && a_hi > 0.f ? Q + s.node * a.q_st : nullptr;
    const bool wide = (reinterpret_cast<uintptr_t>(row) & (4 * sizeof(T) - 1)) == 0 &&
                      (!qrow || (reinterpret_cast<uintptr_t>(qrow) & (4 * sizeof(T) - 1)) == 0);
    const int n_gone = s.n_gone;
    auto is_gone = [&](int v) {
      bool g = false;
      for (int k = 0; k < n_gone; ++k) g = g || s.gone[k] == v;
      return g;
    };
    // ---- sums of w over the block's chunks; a step's entries are on their way while the one before is added ----
    const int per = a.chunk / kStep, steps = warp < n_chunks ? ((n_chunks - 1 - warp) / kWarps + 1) * per : 0;
    uint32_t p[8], q[8], pn[8], qn[8];
    Sum2 sum = {f2(0.f), f2(0.f)};
    int at_v = 0, at_end = 0;  // the step that is added
#pragma unroll 1
    for (int k = 0; k <= steps; ++k) {
      const int c = warp + k / per * kWarps, c0 = v0 + c * a.chunk, v = c0 + k % per * kStep, end = min(v1, c0 + a.chunk);
      if (k < steps) {
        load8(row, v, end, lane, wide, pn);
        if (qrow) load8(qrow, v, end, lane, wide, qn);
      }
      if (k > 0) {
        if (qrow) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const Weight2 w = weight(pair_of<T>(p, i, wide), pair_of<T>(q, i, wide), a_hi, a_lo);
            sum.add(w.hi);
            sum.lo = __fadd2_rn(sum.lo, w.lo);
          }
        } else {
          float2 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = pair_of<T>(p, i, wide);
          for (int g = 0; g < n_gone; ++g) {
            const int t = s.gone[g];
            if (t < at_v || t >= min(at_end, at_v + kStep)) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (entry8(at_v, j, lane, wide) == t) (j & 1 ? x[j >> 1].y : x[j >> 1].x) = 0.f;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) sum.add(x[i]);
        }
        if (k % per == 0) {
          const Two t = warp_sum(sum.total());
          if (lane == 0) s.chunk[warp + (k - 1) / per * kWarps] = t;
          sum = {f2(0.f), f2(0.f)};
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = pn[i];
        q[i] = qn[i];
      }
      at_v = v;
      at_end = end;
    }
    __syncthreads();
    part.begin();
    // ---- warp 0: runs of chunks a lane, the block's total to every block ----
    const int run = (n_chunks + 31) / 32;
    Two upto = {0.f, 0.f};  // the block's sum up to the end of the lane's run
    if (warp == 0) {
      for (int c = lane * run; c < min(n_chunks, (lane + 1) * run); ++c) upto = plus(upto, s.chunk[c]);
      upto = scan(upto, lane, 32);
      const Two mine = shfl(upto, 31);
      if (lane < C) store_remote(&s.x.total[part.turn][rank], lane, bits(mine));
    }
    part.wait();
    Two target = {0.f, 0.f}, base = {0.f, 0.f};
    if (warp == 0) {
      Two end = {0.f, 0.f};  // the sum up to the end of block `lane`
      if (lane < C) end = two(s.x.total[part.turn][lane]);
      end = scan(end, lane, C);
      const Two total = shfl(end, C - 1);
      // a rejection with a later child left to test: on; else these are the draw's sums. A residual without mass: P's
      const bool more = rejected && nodes.children(node, at), empty = !more && !fallback && !(total.hi > 0.f);
      if (more) {
        wz = total;
      } else if (empty) {
        fallback = true;
        wa = {0.f, 0.f};
        gone = 0;
      } else {
        // ---- the draw: the block, the chunk, the entry in which the sums pass u total ----
        target = times({__shfl_sync(0xFFFFFFFFu, u[0], 0), 0.f}, total);
        // each block's end is the next one's beginning, so exactly one holds the target; without mass any token does
        const unsigned past = __ballot_sync(0xFFFFFFFFu, lane < C && less(target, end));
        const Two before = shfl(end, rank > 0 ? (int)rank - 1 : 0);
        if (rank == 0) {
          for (int i = lane; i < count; i += 32) a.path[(size_t)b * a.N + i] = s.path[i];
          if (lane == 0) {
            a.n_accept[b] = count;
            if (!past) a.next[b] = 0;
          }
        }
        if (past && __ffs(past) - 1 == (int)rank) {
          if (rank > 0) base = before;
          const unsigned in = __ballot_sync(0xFFFFFFFFu, less(target, plus(base, upto)));
          const int last_run = (n_chunks - 1) / run, hold = in ? min(__ffs(in) - 1, last_run) : last_run;
          const Two y = shfl(upto, hold > 0 ? hold - 1 : 0);
          if (hold > 0) base = plus(base, y);
          int c = hold * run;
          for (; c + 1 < min(n_chunks, (hold + 1) * run); ++c) {
            const Two e = plus(base, s.chunk[c]);
            if (less(target, e)) break;
            base = e;
          }
          if (lane == 0) {
            s.c0 = v0 + c * a.chunk;
            s.found = -1;
            s.done = 2;
          }
        } else if (lane == 0) {
          s.done = 1;
        }
      }
    }
    part.turn ^= 1;
    __syncthreads();
    if (s.done == 1) return;  // the last writes into this block's memory were those that the last barrier waited for
    if (s.done == 2) {
      // ---- the chunk that holds the target, 512 entries at a time: an entry a thread, then 16 a lane of warp 0 ----
      const int c1 = min(v1, s.c0 + a.chunk);
      int last = s.c0;  // the last entry with a weight, should roundings leave none past the target
      for (int v = s.c0; v < c1; v += 512) {
        for (int i = tid; i < 512; i += THREADS) {
          const int x = v + i;
          float p = x < c1 ? to_f(row[x]) : 0.f;
          const float q = qrow && x < c1 ? to_f(qrow[x]) : 0.f;
          if (n_gone && is_gone(x)) p = 0.f;
          const Weight2 w = weight(f2(p), f2(q), a_hi, a_lo);  // p without a row of Q
          const Two y = plus({w.hi.x, 0.f}, {w.lo.x, 0.f});
          s.w[0][i + (i >> 4)] = y.hi;
          s.w[1][i + (i >> 4)] = y.lo;
        }
        __syncthreads();
        if (warp == 0) {
          const float *hi = s.w[0] + 17 * lane, *lo = s.w[1] + 17 * lane;
          Two t = {0.f, 0.f};
#pragma unroll 4
          for (int j = 0; j < 16; ++j) {
            t = plus(t, {hi[j], lo[j]});
            if (hi[j] > 0.f) last = v + 16 * lane + j;
          }
          const Two upto16 = scan(t, lane, 32);
          const unsigned hit = __ballot_sync(0xFFFFFFFFu, less(target, plus(base, upto16)));
          if (hit) {  // that lane's entries, one a lane
            const int src = __ffs(hit) - 1;
            const float h = lane < 16 ? s.w[0][17 * src + lane] : 0.f, l = lane < 16 ? s.w[1][17 * src + lane] : 0.f;
            const Two e = scan({h, l}, lane, 16);
            const Two at16 = shfl(upto16, src > 0 ? src - 1 : 0), from = src > 0 ? plus(base, at16) : base;
            const unsigned some = __ballot_sync(0xFFFFFFFFu, lane < 16 && h > 0.f);
            const unsigned one = __ballot_sync(0xFFFFFFFFu, lane < 16 && h > 0.f && less(target, plus(from, e)));
            if (lane == 0) s.found = v + 16 * src + (one ? __ffs(one) - 1 : some ? 31 - __clz(some) : 0);
          }
          base = plus(base, shfl(upto16, 31));
        }
        __syncthreads();
        if (s.found >= 0) break;
      }
      if (warp == 0) {
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) last = max(last, __shfl_xor_sync(0xFFFFFFFFu, last, off));
        if (lane == 0) a.next[b] = s.found >= 0 ? s.found : last;
      }
      return;
    }
  }
}

template <typename T>
cudaError_t launch_typed(const VerifyArgs& args, cudaStream_t st) {
  VerifyArgs a = args;
  int C = 1;  // two blocks an SM at most; a slice of 2048 entries at least
  while (C < kMaxCluster && a.B * C * 2 <= 2 * device_sms() && a.V / (2 * C) >= 2048) C *= 2;
  a.blocks = C;
  a.slice = ((a.V + C - 1) / C + 511) / 512 * 512;
  a.chunk = 512;
  while ((a.slice + a.chunk - 1) / a.chunk > kMaxChunks) a.chunk *= 2;
  const bool few = a.B * C <= device_sms();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = (unsigned)(a.B * C);
  cfg.blockDim = !a.u ? kGreedyThreads : few ? 512 : 256;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (!a.u) return cudaLaunchKernelEx(&cfg, verify_greedy_kernel<T>, a);
  return few ? cudaLaunchKernelEx(&cfg, verify_kernel<T, 512>, a) : cudaLaunchKernelEx(&cfg, verify_kernel<T, 256>, a);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int dtype, cudaStream_t st) {
  if (dtype == KVQ_DT_FP32) return launch_typed<float>(a, st);
  if (dtype == KVQ_DT_BF16) return launch_typed<__nv_bfloat16>(a, st);
  return launch_typed<__half>(a, st);
}

}  // namespace kvq
