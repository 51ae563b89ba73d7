// Slots of a cache continue other slots: copying, forking, reordering, compacting and freeing requests.
//
// slot[b0 + i] := what slot[source[i]] was before the call, for all i at once. The arrays of a cache
// are [outer][slot][head][rows]: a slot's bytes lie at the same places relative to its start, so a
// thread takes one 16-byte unit of a (outer, head) line and moves it for every slot: what it writes is
// read by no other thread, and "all loads before all stores" is a matter of one thread (or, with many
// slots, of one block). Only a move whose source slot is itself overwritten (a hazard: permutations,
// chains) has to wait in shared memory; those of forks and of beams that replace dropped ones stream
// through registers. The blocks take equal shares of the units up to the longest slot that moves.
//
// Bound: HBM, each moved byte read once per distinct source and written once per slot.
#include <algorithm>

#include "kvq_common.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 128;
constexpr int kStage = 16;     // hazards that a full-width unit row stages (32 KB)
constexpr int kBatch = 8;      // moves whose loads are in flight together
constexpr int kBlocks = 5;     // an SM, as the staging leaves room for

// What a slot holds. KIVI: tokens, quantized keys, quantized values; LoopVQ: tokens, index pages.
struct Lens {
  int n, a, b;
};
struct Move {
  int dst, src;
  Lens len;
};

// 0: a move; else the error of a slot that cannot be one (-1: nothing to do, -2: to be freed)
__device__ __forceinline__ int judge(const CacheForkArgs& a, int i, Move& m) {
  const int s = a.source[i];
  m.dst = a.b0 + i;
  m.src = s;
  if (s == KVQ_SLOT_KEEP || (a.same && s == m.dst)) return -1;
  if (s == KVQ_SLOT_FREE) return -2;
  if (s < 0 || s >= a.from_batch) return KVQ_ERR_INVALID_ARG;
  Lens& L = m.len;
  L.n = a.from_len[0][s];
  L.a = a.from_len[1][s];
  L.b = a.from_len[2] ? a.from_len[2][s] : 0;
  if (a.format == KVQ_FMT_KIVI) {
    if (L.b < 0 || L.b > L.a || L.a > L.n || L.n - L.b > a.residual || L.a % 32 || L.a > a.from_room) return KVQ_ERR_INVALID_ARG;
    return L.a > a.room ? KVQ_ERR_CAPACITY : 0;
  }
  const int first = a.sink + kPage * L.a;  // the first token behind the pages
  if (L.n < 0 || L.a < 0 || L.a > a.from_room || (L.a > 0 && L.n < first) || L.n - first > a.ring) return KVQ_ERR_INVALID_ARG;
  return L.a > a.room || L.n > a.max_ctx ? KVQ_ERR_CAPACITY : 0;
}

// Bytes of a line up to the last one that a slot of these lengths may hold
__device__ __forceinline__ long long line_bytes(const CacheForkArgs& a, const ForkArray& x, const Lens& L) {
  switch (x.kind) {
    case kForkA: return (long long)L.a * x.row;
    case kForkGroups: return (long long)(L.a / 32) * x.row;
    case kForkB: return (long long)L.b * x.row;
    case kForkTail: return (long long)(L.n - L.a) * x.row;
    case kForkRing: return L.n > L.b ? (long long)a.ring * x.row : 0;
    default: return (long long)(a.sink + a.ring) * x.row;  // window
  }
}
// Bytes (16, 8 or 0) of the unit at `off` of a line that a slot of these lengths holds
__device__ __forceinline__ int unit_bytes(const CacheForkArgs& a, const ForkArray& x, const Lens& L, long long off, long long end) {
  if (off >= end) return 0;
  if (x.kind < kForkRing) return end - off >= 16 ? 16 : 8;  // rows are multiples of 8 bytes
  int r = (int)off / x.row;  // a few rows
  if (x.kind == kForkWindow) {
    if (r < a.sink) return r < L.n ? 16 : 0;
    r -= a.sink;
  }
  // tokens t0 .. n - 1 in rows t % ring (window: (t - sink) % ring)
  const int t0 = x.kind == kForkRing ? L.b : kPage * L.a, held = x.kind == kForkRing ? L.n - L.b : L.n - a.sink - t0;
  int d = r - t0 % a.ring;
  if (d < 0) d += a.ring;
  return d < held ? 16 : 0;
}

__global__ void __launch_bounds__(kThreads, kBlocks) cache_fork_kernel(const CacheForkArgs a) {
  __shared__ __align__(16) uint4 stage[kStage * kThreads];
  __shared__ Move moves[KVQ_FORK_MAX];
  __shared__ unsigned char is_move[KVQ_FORK_MAX], is_hazard[KVQ_FORK_MAX];
  __shared__ long long longest[kForkArrays], upto[kForkArrays + 1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, n = a.n;
  Move mine[KVQ_FORK_MAX / kThreads];
#pragma unroll
  for (int k = 0; k < KVQ_FORK_MAX / kThreads; ++k) {
    const int i = tid + k * kThreads;
    if (i < n) is_move[i] = judge(a, i, mine[k]) == 0;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < KVQ_FORK_MAX / kThreads; ++k) {
    const int i = tid + k * kThreads, s = i < n && is_move[i] ? mine[k].src - a.b0 : -1;
    if (i < n) is_hazard[i] = a.same && s >= 0 && s < n && is_move[s];
  }
  __syncthreads();
  // the list of moves, hazards first
  int hazards = 0, total = 0;
  for (int base = 0; base < n; base += 32) {
    const bool in = base + lane < n;
    const unsigned h = __ballot_sync(0xFFFFFFFFu, in && is_hazard[base + lane]);
    const unsigned m = __ballot_sync(0xFFFFFFFFu, in && is_move[base + lane]);
    hazards += __popc(h);
    total += __popc(m);
  }
  if (total == 0) return;
#pragma unroll
  for (int k = 0; k < KVQ_FORK_MAX / kThreads; ++k) {
    const int i = tid + k * kThreads;
    if (i >= n || !is_move[i]) continue;
    int at = is_hazard[i] ? 0 : hazards;
    for (int j = 0; j < i; ++j) at += is_move[j] && is_hazard[j] == is_hazard[i];
    moves[at] = mine[k];
  }
  __syncthreads();
  // units across: as many as the hazards of each leave room for; the rest of the threads takes other moves of theirs
  int width = kThreads;
  while (hazards * width > kStage * kThreads) width >>= 1;
  const int unit = tid & (width - 1), group = tid / width, groups = kThreads / width;
  for (int x = tid >> 5; x < a.n_arrays; x += kThreads / 32) {
    long long most = 0;
    for (int i = lane; i < total; i += 32) most = max(most, line_bytes(a, a.array[x], moves[i].len));
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, off));
    if (lane == 0) longest[x] = most;
  }
  __syncthreads();
  if (tid == 0) {
    upto[0] = 0;
    for (int x = 0; x < a.n_arrays; ++x)
      upto[x + 1] = upto[x] + (longest[x] + width * 16 - 1) / (width * 16) * a.array[x].outer * a.heads;
  }
  __syncthreads();
  const long long pieces = upto[a.n_arrays];
  for (long long p = blockIdx.x; p < pieces; p += gridDim.x) {
    int xi = 0;
    while (p >= upto[xi + 1]) ++xi;
    const ForkArray& x = a.array[xi];
    const int lines = x.outer * a.heads;
    const long long rel = p - upto[xi], piece = rel / lines;
    const int line = (int)(rel - piece * lines), o = line / a.heads, h = line - o * a.heads;
    const long long off = (piece * width + unit) * 16;
    const unsigned char* src = x.src + o * x.src_outer + h * x.src_head + off;
    unsigned char* dst = x.dst + o * x.dst_outer + h * x.dst_head + off;
    auto bytes = [&](const Move& m) { return unit_bytes(a, x, m.len, off, line_bytes(a, x, m.len)); };
    auto load = [&](const Move& m, int k) {
      const unsigned char* at = src + m.src * x.src_slot;
      if (k == 16) return *reinterpret_cast<const uint4*>(at);
      const uint2 u = *reinterpret_cast<const uint2*>(at);
      return make_uint4(u.x, u.y, 0u, 0u);
    };
    auto store = [&](const Move& m, int k, const uint4& v) {
      unsigned char* at = dst + m.dst * x.dst_slot;
      if (k == 16) *reinterpret_cast<uint4*>(at) = v;
      else *reinterpret_cast<uint2*>(at) = make_uint2(v.x, v.y);
    };
    if (hazards > 0) {
      int st = tid;
      for (int i = group; i < hazards; i += groups, st += kThreads) {
        const int k = bytes(moves[i]);
        if (k) stage[st] = load(moves[i], k);
      }
      if (groups > 1) __syncthreads();  // other threads write what these have read
    }
    for (int i0 = hazards + group; i0 < total; i0 += kBatch * groups) {
      uint4 v[kBatch];
      int k[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int i = i0 + e * groups;
        k[e] = i < total ? bytes(moves[i]) : 0;
        if (k[e]) v[e] = load(moves[i], k[e]);
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e)
        if (k[e]) store(moves[i0 + e * groups], k[e], v[e]);
    }
    int st = tid;
    for (int i = group; i < hazards; i += groups, st += kThreads) {
      const int k = bytes(moves[i]);
      if (k) store(moves[i], k, stage[st]);
    }
  }
}

// The lengths, once every block above has read them.
__global__ void __launch_bounds__(KVQ_FORK_MAX) cache_fork_lens_kernel(const CacheForkArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int i = threadIdx.x;
  Move m = {};
  const int st = i < a.n ? judge(a, i, m) : -1;
  if (st > 0) set_error(a.err, st);
  __syncthreads();
  if (st != 0 && st != -2) return;
  if (st == -2) m.len = {0, 0, 0};
  a.len[0][m.dst] = m.len.n;
  a.len[1][m.dst] = m.len.a;
  if (a.len[2]) a.len[2][m.dst] = m.len.b;
}

}  // namespace

cudaError_t launch_cache_fork(const CacheForkArgs& a, long long most_pieces, cudaStream_t st) {
  const int grid = (int)std::min(most_pieces, (long long)device_sms() * kBlocks);
  if (grid > 0) {
    cache_fork_kernel<<<grid, kThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = 1;
  cfg.blockDim = KVQ_FORK_MAX;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = grid > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, cache_fork_lens_kernel, a);
}

}  // namespace kvq
