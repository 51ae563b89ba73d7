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
// Bound: HBM, each moved byte read once per distinct source and written once per slot, behind a chain of dependent loads
// (sources, lengths, table, first units: about 5 us). A prompt of 4096 tokens to 16 slots (32 heads, 2 bits, 243 MB): 52 us,
// 4.7 TB/s, 69 % of the copy rate; 64 beams of 1531 tokens in place, about half of which move: 31; eight slots of 701 tokens in
// index pages: 16 - 18. The first form took 64, 39 and 20. Blocks of 256 threads, batches of 4 and 16
// moves, streaming stores and loads past L1 were not better. Moves with hazards, every unit by way of shared memory: 64 slots of
// 1531 tokens (8 heads, 4 bits) compacted to 43 57 us (floor 29), in another order 98 (42); 16 slots of 4096 (32 heads, 2 bits)
// in a ring 124 (67).
#include <algorithm>

#include "kvq_common.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 128;
constexpr int kStage = 8;      // hazards that a full-width row of units stages (16 KB)
constexpr int kBatch = 8;      // moves whose loads are in flight together
constexpr int kBlocks = 7;     // an SM, as the staging leaves room for

// What a slot holds. KIVI: tokens, quantized keys, quantized values; LoopVQ: tokens, index pages.
struct Lens {
  int n, a, b;
};
struct Move {
  int dst, src;
  Lens len;
};

// 0: a move; else the error of a slot that cannot be one (-1: nothing to do, -2: to be freed)
__device__ __forceinline__ int check_move(const CacheForkArgs& a, int i, Move& m) {
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

// Eighths of a line's bytes up to the last one that a slot of these lengths may hold (rows are multiples of 8 bytes)
__device__ __forceinline__ int line_eighths(const CacheForkArgs& a, const ForkArray& x, const Lens& L) {
  const int row = x.row / 8;
  switch (x.kind) {
    case kForkA: return L.a * row;
    case kForkGroups: return L.a / 32 * row;
    case kForkB: return L.b * row;
    case kForkTail: return (L.n - L.a) * row;
    case kForkRing: return L.n > L.b ? a.ring * row : 0;
    default: return (a.sink + a.ring) * row;  // window
  }
}
// Rows of a ring (of the window's: behind the sink): `held` of them from `first` on, around its end
struct Ring {
  int first, held;
};
__device__ __forceinline__ Ring ring_of(const CacheForkArgs& a, const Lens& L) {
  if (a.ring == 0) return {0, 0};
  if (a.format == KVQ_FMT_KIVI) return {L.b % a.ring, L.n - L.b};
  return {kPage * L.a % a.ring, L.n - a.sink - kPage * L.a};
}
__device__ __forceinline__ bool in_ring(const CacheForkArgs& a, int kind, int row, int n, const Ring& g) {
  if (kind == kForkWindow) {
    if (row < a.sink) return row < n;
    row -= a.sink;
  }
  int d = row - g.first;
  if (d < 0) d += a.ring;
  return d < g.held;
}

__global__ void __launch_bounds__(kThreads, kBlocks) cache_fork_kernel(const CacheForkArgs a) {
  __shared__ __align__(16) uint4 stage[kStage * kThreads];
  __shared__ int2 moves[KVQ_FORK_MAX];             // from, to
  __shared__ int tokens[KVQ_FORK_MAX];
  __shared__ Ring rings[KVQ_FORK_MAX];
  __shared__ int ends[kForkArrays][KVQ_FORK_MAX];  // eighths of a line that a move has
  __shared__ unsigned char is_move[KVQ_FORK_MAX];
  __shared__ int longest[kForkArrays], shortest[kForkArrays], upto[kForkArrays + 1];
  launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, n = a.n;
  constexpr int kMine = KVQ_FORK_MAX / kThreads, kWords = KVQ_FORK_MAX / 32;
  Move mine[kMine];
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int i = tid + k * kThreads;
    is_move[i] = i < n && check_move(a, i, mine[k]) == 0;
  }
  if (tid < kForkArrays) {
    longest[tid] = 0;
    shortest[tid] = 0x7FFFFFFF;
  }
  __syncthreads();
  // the list of moves, hazards first
  uint32_t moved[kWords], hazard[kWords];
  int hazards = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    moved[w] = hazard[w] = 0;
    if (32 * w < n) {
      const int i = 32 * w + lane, s = is_move[i] ? a.source[i] - a.b0 : -1;
      moved[w] = __ballot_sync(0xFFFFFFFFu, is_move[i]);
      hazard[w] = __ballot_sync(0xFFFFFFFFu, a.same && s >= 0 && s < n && is_move[s]);
      hazards += __popc(hazard[w]);
      total += __popc(moved[w]);
    }
  }
  if (total == 0) return;
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int i = tid + k * kThreads;
    if (!is_move[i]) continue;
    int before_h = 0, before_o = 0;
    bool h = false;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const uint32_t below = w < i >> 5 ? ~0u : w == i >> 5 ? (1u << (i & 31)) - 1 : 0u;
      before_h += __popc(hazard[w] & below);
      before_o += __popc(moved[w] & ~hazard[w] & below);
      if (w == i >> 5) h = (hazard[w] >> (i & 31)) & 1;
    }
    const int at = h ? before_h : hazards + before_o;
    moves[at] = make_int2(mine[k].src, mine[k].dst);
    tokens[at] = mine[k].len.n;
    rings[at] = ring_of(a, mine[k].len);
    for (int x = 0; x < a.n_arrays; ++x) {
      const int e = line_eighths(a, a.array[x], mine[k].len);
      ends[x][at] = e;
      atomicMax(&longest[x], e);
      atomicMin(&shortest[x], e);
    }
  }
  // units across: as many as the hazards of each leave room for; the rest of the threads takes other moves of theirs
  int width = kThreads;
  while (hazards * width > kStage * kThreads) width >>= 1;
  const int unit = tid & (width - 1), group = tid / width, groups = kThreads / width;
  __syncthreads();
  if (tid == 0) {
    upto[0] = 0;
    for (int x = 0; x < a.n_arrays; ++x)
      upto[x + 1] = upto[x] + (longest[x] + 2 * width - 1) / (2 * width) * a.array[x].outer * a.heads;
  }
  __syncthreads();
  // without hazards any moves of a piece may go to any block: kBatch of them each
  const int all_runs = (total + kBatch - 1) / kBatch, pieces = upto[a.n_arrays];
  const bool spread = hazards == 0 && (long long)pieces * all_runs < (1ll << 31);
  const IntDiv runs = {spread ? all_runs : 1, 0xFFFFFFFFu / (uint32_t)(spread ? all_runs : 1)};
  for (long long task = blockIdx.x, tasks = (long long)pieces * runs.d; task < tasks; task += gridDim.x) {
    const int p = div_by((int)task, runs), run = (int)task - p * runs.d;
    int xi = 0;
    while (p >= upto[xi + 1]) ++xi;
    const ForkArray& x = a.array[xi];
    const int kind = x.kind, rel = p - upto[xi], piece = div_by(rel, x.lines);
    const int line = rel - piece * x.lines.d, o = div_by(line, a.per_outer), h = line - o * a.heads;
    const int mine_at = 2 * (piece * width + unit);  // the thread's unit of the line, in eighths
    const unsigned char* src = x.src + o * x.src_outer + h * x.src_head + mine_at * 8ll;
    unsigned char* dst = x.dst + o * x.dst_outer + h * x.dst_head + mine_at * 8ll;
    const int ring_row = kind >= kForkRing ? mine_at / (x.row / 8) : 0;
    if (spread && kind < kForkRing && 2 * (piece + 1) * width <= shortest[xi] && (run + 1) * kBatch <= total) {
      // every move has the whole piece: no questions asked, a source that they share (a forked prompt) read once
      const uint32_t from = (uint32_t)(x.src_slot >> 4), to = (uint32_t)(x.dst_slot >> 4);
      int2 m[kBatch];
      bool one = true;
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        m[e] = moves[run * kBatch + e];
        one = one && m[e].x == m[0].x;
      }
      uint4 v[kBatch];
      const uint4* src16 = reinterpret_cast<const uint4*>(src);
      uint4* dst16 = reinterpret_cast<uint4*>(dst);
      if (one) {
        v[0] = src16[(uint64_t)(uint32_t)m[0].x * from];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) dst16[(uint64_t)(uint32_t)m[e].y * to] = v[0];
      } else {
#pragma unroll
        for (int e = 0; e < kBatch; ++e) v[e] = src16[(uint64_t)(uint32_t)m[e].x * from];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) dst16[(uint64_t)(uint32_t)m[e].y * to] = v[e];
      }
      continue;
    }
    // what move i has of the unit: 16 bytes (2), 8 (1) or none
    auto has = [&](int i) {
      const int left = ends[xi][i] - mine_at;
      if (left <= 0) return 0;
      if (kind >= kForkRing) return in_ring(a, kind, ring_row, tokens[i], rings[i]) ? 2 : 0;
      return left >= 2 ? 2 : 1;
    };
    auto load = [&](int i, int k) {
      const unsigned char* at = src + moves[i].x * x.src_slot;
      if (k == 2) return *reinterpret_cast<const uint4*>(at);
      const uint2 v = *reinterpret_cast<const uint2*>(at);
      return make_uint4(v.x, v.y, 0u, 0u);
    };
    auto store = [&](int i, int k, const uint4& v) {
      unsigned char* at = dst + moves[i].y * x.dst_slot;
      if (k == 2) *reinterpret_cast<uint4*>(at) = v;
      else *reinterpret_cast<uint2*>(at) = make_uint2(v.x, v.y);
    };
    if (hazards > 0) {
      int st = tid;
      for (int i = group; i < hazards; i += groups, st += kThreads) {
        const int k = has(i);
        if (k) stage[st] = load(i, k);
      }
      if (groups > 1) __syncthreads();  // other threads write what these have read
    }
    for (int i0 = hazards + run * kBatch + group; i0 < total; i0 += kBatch * groups) {
      uint4 v[kBatch];
      int k[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int i = i0 + e * groups;
        k[e] = i < total ? has(i) : 0;
        if (k[e]) v[e] = load(i, k[e]);
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e)
        if (k[e]) store(i0 + e * groups, k[e], v[e]);
      if (spread) break;  // the next ones are another task's
    }
    int st = tid;
    for (int i = group; i < hazards; i += groups, st += kThreads) {
      const int k = has(i);
      if (k) store(i, k, stage[st]);
    }
  }
}

// The lengths, once every block above has read them.
__global__ void __launch_bounds__(KVQ_FORK_MAX) cache_fork_lens_kernel(const CacheForkArgs a) {
  wait_behind();
  const int i = threadIdx.x;
  Move m = {};
  const int st = i < a.n ? check_move(a, i, m) : -1;
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
  // a piece's moves go to different blocks, kBatch each, and with many hazards pieces are smaller: a short slot's pieces alone
  // left most of the GPU idle (256 slots of 300 tokens, 8 heads, 2 bits: from one prompt 64 us, now 44; a permutation 301, now 117)
  const long long runs = (a.n + kBatch - 1) / kBatch;
  const int grid = (int)std::min(most_pieces * runs, (long long)device_sms() * kBlocks);
  if (grid > 0) {
    cache_fork_kernel<<<grid, kThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return launch_early(grid > 0, cache_fork_lens_kernel, dim3(1), KVQ_FORK_MAX, 0, st, a);
}

}  // namespace kvq
