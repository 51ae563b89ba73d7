// Attention of a tree of drafted tokens over a KIVI cache.
//
// Request b has n cached tokens and up to N <= 64 drafted ones with their own fp16 keys and
// values. Drafted token i attends every cached token and the drafted tokens j whose bit is set
// in its mask, with one softmax over both (scale 1/sqrt(D)):
//   o_i = sum_t p_it v_t / sum_t p_it,  p_it = exp(q_i k_t / sqrt(D) - m_i).
// The rows of a KV head are the N drafted tokens times its n_q_heads / n_heads query heads.
//
// Tokens (cached, then drafted) form tiles of 128, and a persistent grid takes equal contiguous
// shares of all tiles (segment by segment, a segment being a request, KV head and row tile).
// Operands enter the tensor cores as fp16, in two parts where one would cost more than the bound of
// attention allows; the sums, the running maxima and the normalisers are fp32. The running maximum of a row moves only when a score passes it by
// 2^kSlack. Segments that blocks share leave partial softmaxes in the workspace, which a second
// small kernel joins in block order, so the result does not depend on timing.
//
// Two kernels by the number of rows R of a KV head (tree_rows, where both sides are measured):
//  * R <= 16: warp-wide products. A warp takes a 32-token key group and unpacks the codes straight
//    into the A fragments of m16n8k16 products (tokens and channels are the 16 rows, query rows the
//    8 columns); scores and sums stay in registers, nothing goes through shared memory but the
//    stored tile, and warps meet only at the segment's end.
//  * more rows: tcgen05 on tiles of 32 or 64 rows. S^T [128 tokens x rows] = K . q^T and
//    O^T [128 channels x rows] += V^T . P^T keep all 128 lanes of every product busy; the unpacked
//    operands go through shared memory once for a tile's rows.
// HBM traffic is the codes and scales once per row tile; both kernels are bound on chip (below).
//
// What a block runs once or once per segment (its share, the queries, the last tile's drafts, the
// segment's end) is written for few instructions rather than few steps: rolled loops, divisions by
// the launch's constants as one product. Unrolled, that code was fetched cold in every block and
// took longer than the work in it (two requests, 1K context, 64 rows: 22.8 -> 20.2 us; 16 rows, 4K:
// 142 -> 123 in the form of then).
#include <cuda_fp16.h>

#include <cfloat>

#include "kivi_tree_join.h"
#include "kvq_common.cuh"
#include "kvq_internal.h"
#include "../../include/kvq.h"

namespace kvq {
namespace {

constexpr int kTile = 128;    // tokens per tile
constexpr int kGroupT = 32;   // tokens per key group, channels per value group
// A row's weights are exp2(x - m + kRaise), m its running maximum, which moves when a score passes it by kSlack (log2):
// weights stay below 2^15 and are held as fp16, where one below 2^-30 of the maximum's is lost (2^-25 without kRaise).
// Raising costs a pass over the sums; at a slack of 7 the peaked scores of outlier channels raise some row of a tile
// of 64 in most of a segment's first tiles.
constexpr float kSlack = 10.f, kRaise = 5.f;

// TOK stored tokens (a key group or a tile): key codes, scales and zeros [groups][128], value codes, scales and
// zeros [tokens][4]
template <int KB, int VB, int TOK>
struct StageLayout {
  static constexpr int kKRow = kD * KB / 8, kVRow = kD * VB / 8;   // code bytes per token
  static constexpr int kKs = TOK * kKRow, kKz = kKs + (TOK / kGroupT) * kD * 2;
  static constexpr int kVc = kKz + (TOK / kGroupT) * kD * 2;
  static constexpr int kVs = kVc + TOK * kVRow, kVz = kVs + TOK * (kD / kGroupT) * 2;
  static constexpr int kBytes = kVz + TOK * (kD / kGroupT) * 2;
};

__device__ __forceinline__ float th2f(uint32_t b) { return __half2float(__ushort_as_half((unsigned short)b)); }
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The work of a call, the same for every block: segment (b, h, row tile) has T_b tiles (its cached
// and drafted tokens), all segments in the order b, h, row tile form one list of P tile positions,
// and block k of G takes positions [k P / G, (k + 1) P / G); of fewer than G positions the first blocks take one each,
// so that the blocks of a segment are neighbours (two requests, 1K context, 64 rows: 20.2 -> 16.6 us).
struct TreeLens {
  int nqk, nqv, n, nd;  // quantized keys, quantized values, cached tokens, drafted tokens
  int tiles;
};
__device__ __forceinline__ TreeLens tree_lens(const KiviTreeArgs& a, int b) {
  TreeLens L;
  L.nqk = min(max(a.n_quant_k[b], 0), a.max_tokens) & -kGroupT;
  L.n = L.nqk + max(0, min(a.n_tok[b] - L.nqk, a.residual));
  // at least n - residual, as in every valid state: the ring holds no more values
  L.nqv = (a.residual > 0) ? min(max(a.n_quant_v[b], max(L.n - a.residual, 0)), L.nqk) : L.nqk;
  L.nd = a.n_draft ? min(max(a.n_draft[b], 0), a.N) : a.N;
  L.tiles = L.nd > 0 ? (int)((uint32_t)(L.n + L.nd + kTile - 1) / kTile) : 0;
  return L;
}
// where the share of block k of G begins, without leaving 32 bits (k <= G, G far below 2^15)
__device__ __forceinline__ int share_begin(int P, int k, const IntDiv& G) {
  if (P <= G.d) return min(k, P);
  const int q = div_by(P, G);
  return k * q + div_by(k * (P - q * G.d), G);
}

// A role's place in the block's share
struct Walk {
  int b, seg, tile;  // seg = h * row tiles + row tile
  TreeLens len;
  __device__ __forceinline__ bool last() const { return tile + 1 == len.tiles; }
  // to the next position; `more`: there is one in the share
  __device__ __forceinline__ void next(const KiviTreeArgs& a, int seg_per_b, bool more) {
    if (++tile < len.tiles || !more) return;
    tile = 0;
    if (++seg < seg_per_b) return;
    seg = 0;
    do len = tree_lens(a, ++b);
    while (len.tiles == 0);  // a position is left, so such a request exists
  }
};

// partial softmax of a segment: rows of o[128], then m, l per row
template <int ROWS>
__host__ __device__ constexpr size_t slot_floats() { return (size_t)ROWS * (kD + 2); }
// What block k did with the segments it shares, for the merge. first: its first segment (kSeg...). open: the segment
// that begins in the block and goes on (b * segments per request + seg), or -1; nd: that request's drafted tokens.
struct TreeShared {
  int first, open, nd, pad;
};

// The place in all positions where the block's share begins, and the share [p0, p1): each warp on its own, its lanes
// take equal runs of requests.
__device__ __forceinline__ int2 find_share(const KiviTreeArgs& a, int seg_per_b, int lane, Walk& w) {
  const int run = (a.B + 31) / 32, b0 = lane * run, b1 = min(a.B, b0 + run);
  TreeLens L = {};
  int upto = 0;  // tiles of this lane's requests, then of all up to it
#pragma unroll 1
  for (int b = b1 - 1; b >= b0; --b) {  // L: of the first one
    L = tree_lens(a, b);
    upto += L.tiles;
  }
  const int mine = upto;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, upto, off);
    if (lane >= off) upto += v;
  }
  const int P = __shfl_sync(0xFFFFFFFFu, upto, 31) * seg_per_b;
  const int p0 = share_begin(P, blockIdx.x, a.blocks), p1 = share_begin(P, blockIdx.x + 1, a.blocks);
  w = {};
  if (p0 < p1) {  // the first lane with p0 below its end
    const int src = __ffs(__ballot_sync(0xFFFFFFFFu, p0 < upto * seg_per_b)) - 1;
    if (lane == src) {
      int before = upto - mine;
      w.b = b0;
      while (p0 >= (before + L.tiles) * seg_per_b) {  // ends inside the run
        before += L.tiles;
        L = tree_lens(a, ++w.b);
      }
      const int off = p0 - before * seg_per_b;
      w.len = L;
      w.seg = off / L.tiles;
      w.tile = off - w.seg * L.tiles;
    }
    int* f = reinterpret_cast<int*>(&w);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Walk) / 4); ++i) f[i] = __shfl_sync(0xFFFFFFFFu, f[i], src);
  }
  return make_int2(p0, p1);
}

// The row of a token behind the quantized ones (token t, value: of the ring): residual, drafted, or none
__device__ __forceinline__ const uint16_t* fp16_key(const KiviTreeArgs& a, const TreeLens& L, int b, int h, int t) {
  if (t < L.n) return a.k_resid + (((size_t)b * a.H + h) * a.residual + (t - L.nqk)) * kD;
  if (t < L.n + L.nd) return a.k_draft + (((size_t)b * a.N + (t - L.n)) * a.H + h) * kD;
  return nullptr;
}
// place: t % residual for a token that is cached
__device__ __forceinline__ const uint16_t* fp16_value(const KiviTreeArgs& a, const TreeLens& L, int b, int h, int t, int place) {
  if (t < L.n) return a.v_resid + (((size_t)b * a.H + h) * a.residual + place) * kD;
  if (t < L.n + L.nd) return a.v_draft + (((size_t)b * a.N + (t - L.n)) * a.H + h) * kD;
  return nullptr;
}
// place of token t0 + i (i < 32) when t0's is p: the ring holds at least 32 rows, or none (no token is there then)
__device__ __forceinline__ int ring_place(int p, int i, int R) {
  p += i;
  if (p >= R) p -= R;
  return p;
}
// channels 8c .. 8c+7 of a row, zero without one
__device__ __forceinline__ uint4 row8(const uint16_t* p, int c) {
  return p ? __ldg(reinterpret_cast<const uint4*>(p + 8 * c)) : make_uint4(0u, 0u, 0u, 0u);
}
// halves of w that are infinite or NaN become 0
__device__ __forceinline__ void drop_nonfinite(uint32_t& w) {
  if ((w & 0x7C00u) == 0x7C00u) w &= 0xFFFF0000u;
  if ((w & 0x7C000000u) == 0x7C000000u) w &= 0xFFFFu;
}

// Channel order of the staged keys and queries. The contraction runs over all 128 channels, so any order serves
// that both share; this one is the order in which a code word's halves unpack: pairs (c, c + 8) of 16 channels
// (2 bits), (c, c + 4) of 8 (4 bits). lo, hi: channels 16 w .. + 7, 16 w + 8 .. + 15, natural order; out: the two
// 16-byte chunks of the block.
template <int KB>
__device__ __forceinline__ void pair_order(const uint4 lo, const uint4 hi, uint4& out0, uint4& out1) {
  if constexpr (KB == 2) {
    out0 = make_uint4(__byte_perm(lo.x, hi.x, 0x5410), __byte_perm(lo.x, hi.x, 0x7632), __byte_perm(lo.y, hi.y, 0x5410),
                      __byte_perm(lo.y, hi.y, 0x7632));
    out1 = make_uint4(__byte_perm(lo.z, hi.z, 0x5410), __byte_perm(lo.z, hi.z, 0x7632), __byte_perm(lo.w, hi.w, 0x5410),
                      __byte_perm(lo.w, hi.w, 0x7632));
  } else {
    out0 = make_uint4(__byte_perm(lo.x, lo.z, 0x5410), __byte_perm(lo.x, lo.z, 0x7632), __byte_perm(lo.y, lo.w, 0x5410),
                      __byte_perm(lo.y, lo.w, 0x7632));
    out1 = make_uint4(__byte_perm(hi.x, hi.z, 0x5410), __byte_perm(hi.x, hi.z, 0x7632), __byte_perm(hi.y, hi.w, 0x5410),
                      __byte_perm(hi.y, hi.w, 0x7632));
  }
}
// Token order of the staged values and weights: in odd octets neighbours change places, so that the two octets a
// warp reads at a time come from different banks.
__device__ __forceinline__ int token_place(int t) { return t ^ ((t >> 3) & 1); }

__device__ __forceinline__ __half2 as_h2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ uint32_t as_u(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
// Constants of the unpacking, held in registers, since an instruction has room for one immediate: the exponent of
// 2^10 in both halves (mask and insert are then one instruction), and the powers of two that bring codes unpacked in
// place back to their value.
struct CodeScale {
  uint32_t magic;
  uint32_t p[4];  // 2^-2, 2^-4, 2^-6, 2^-8 as packed halves
  __device__ __forceinline__ CodeScale() {
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));
    asm volatile("mov.b32 %0, 0x34003400;" : "=r"(p[0]));
    asm volatile("mov.b32 %0, 0x2C002C00;" : "=r"(p[1]));
    asm volatile("mov.b32 %0, 0x24002400;" : "=r"(p[2]));
    asm volatile("mov.b32 %0, 0x1C001C00;" : "=r"(p[3]));
  }
};
// Code j of both halves of w as fp16 (exact): masked in place under the exponent of 2^10, where it stands for
// 1024 + c 2^(b j), and scaled back by one FMA. Codes above the ten mantissa bits come from w shifted right.
// CENTRE: what is taken off the code.
template <int BITS, int CENTRE = 0>
__device__ __forceinline__ __half2 code_h2(const CodeScale& cs, uint32_t w, int j) {
  constexpr int kIn = (BITS == 2) ? 5 : 2;  // codes that fit in place
  const int jj = j < kIn ? j : j - kIn, k = BITS * jj / 2;
  uint32_t m;  // (w & mask) | magic
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
      : "=r"(m)
      : "r"(j < kIn ? w : w >> (BITS * kIn)), "r"((((1u << BITS) - 1u) << (BITS * jj)) * 0x10001u), "r"(cs.magic));
  if (k == 0) return __hadd2(as_h2(m), __float2half2_rn(-1024.f - CENTRE));
  return __hfma2(as_h2(m), as_h2(cs.p[k - 1]), __float2half2_rn(-1024.f / (float)(1 << (2 * k)) - CENTRE));
}
// What a stored element is made of: X = s (c - z) = s (c - c0) - (s z - c0 s). With the middle code c0 the first part
// is small and one fp16 (exact with 2 bits; with 4 off by 2^-11 of at most 8 s), however far the group lies from zero;
// the second is one number per group and is never added to it in fp16.
template <int BITS>
constexpr int kCentre = BITS == 2 ? 1 : 8;
// what the rounding of p = fp16(x y) left, exactly
__device__ __forceinline__ uint32_t product_rest(uint32_t x, uint32_t y, uint32_t p) {
  return as_u(__hfma2(as_h2(x), as_h2(y), __hneg2(as_h2(p))));
}
__device__ __forceinline__ uint32_t halved(uint32_t x) { return as_u(__hmul2(as_h2(x), __float2half2_rn(0.5f))); }
// s (c - c0) of eight codes (VB == 2: the low half of w), natural order
template <int VB>
__device__ __forceinline__ uint4 centred8(const CodeScale& cs, uint32_t w, __half2 s) {
  if constexpr (VB == 2) w = __byte_perm(w, 0, 0x4140);  // codes 0 .. 3 and 4 .. 7 in the two halves
  uint32_t x[4];  // codes j, j + 4
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = as_u(__hmul2(code_h2<VB, kCentre<VB>>(cs, w, j), s));
  return make_uint4(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410), __byte_perm(x[0], x[1], 0x7632),
                    __byte_perm(x[2], x[3], 0x7632));
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp_async16(unsigned char* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// The stored part of a tile into a stage by bulk copies of one thread: the keys of whole groups below n_quant_k, the
// values below n_quant_v. With nothing to copy the barrier completes at once.
template <int KB, int VB>
__device__ __forceinline__ void bulk_keys(const KiviTreeArgs& a, const TreeLens& len, size_t bh, int t0,
                                          unsigned char* stage, uint64_t* full) {
  using S = StageLayout<KB, VB, kTile>;
  const int nk = min(kTile, len.nqk - t0);
  if (nk <= 0) {
    mbar_arrive(full);
    return;
  }
  const size_t g = (bh * (a.max_tokens / kGroupT) + t0 / kGroupT) * kD;
  const uint32_t gb = nk / kGroupT * kD * 2;
  fence_proxy_async_smem();
  mbar_arrive_expect_tx(full, nk * S::kKRow + 2 * gb);
  bulk_g2s(stage, a.k_codes + (bh * a.max_tokens + t0) * S::kKRow, nk * S::kKRow, full);
  bulk_g2s(stage + S::kKs, a.k_scale + g, gb, full);
  bulk_g2s(stage + S::kKz, a.k_zero + g, gb, full);
}
template <int KB, int VB>
__device__ __forceinline__ void bulk_values(const KiviTreeArgs& a, const TreeLens& len, size_t bh, int t0,
                                            unsigned char* stage, uint64_t* full) {
  using S = StageLayout<KB, VB, kTile>;
  const int nv = (min(kTile, len.nqv - t0) + 1) & ~1;  // whole 16-byte pieces
  if (nv <= 0) {
    mbar_arrive(full);
    return;
  }
  const size_t tok = bh * a.max_tokens + t0;
  fence_proxy_async_smem();
  mbar_arrive_expect_tx(full, nv * (S::kVRow + 16));
  bulk_g2s(stage + S::kVc, a.v_codes + tok * S::kVRow, nv * S::kVRow, full);
  bulk_g2s(stage + S::kVs, a.v_scale + tok * (kD / kGroupT), nv * 8, full);
  bulk_g2s(stage + S::kVz, a.v_zero + tok * (kD / kGroupT), nv * 8, full);
}

// The fp16 rows of cached tokens t0 .. t1 - 1 into L2 (the warps read them with plain loads): the key residual's are
// contiguous, the value ring's wrap around at most once.
__device__ __forceinline__ void prefetch_fp16(const KiviTreeArgs& a, const TreeLens& len, size_t bh, int t0, int t1) {
  t1 = min(t1, len.n);
  const int tk = max(t0, len.nqk), tv = max(t0, len.nqv), R = a.residual;
  if (tk < t1) bulk_prefetch_l2(a.k_resid + (bh * R + (tk - len.nqk)) * kD, (t1 - tk) * kD * 2);
  if (tv < t1) {
    const int r = tv % R, first = min(t1 - tv, R - r);
    bulk_prefetch_l2(a.v_resid + (bh * R + r) * kD, first * kD * 2);
    if (first < t1 - tv) bulk_prefetch_l2(a.v_resid + bh * R * kD, (t1 - tv - first) * kD * 2);
  }
}

// A query row as fp16 times a power of two that puts its largest magnitude in [2^TOP, 2^(TOP + 1)): eight lanes, 16
// channels each (w: bf16 pairs; o: fp16 pairs). Returns what a score has to be multiplied with (scale: log2 units).
template <int TOP>
__device__ __forceinline__ float query_fp16(const uint32_t (&w)[8], uint32_t (&o)[8], float scale) {
  float mx = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
#pragma unroll
  for (int off = 4; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
  const int ex = (int)(__float_as_uint(mx) >> 23);  // biased exponent; 0: zero or subnormal, 255: not finite
  // times 2^(TOP - (ex - 127)) in two factors, since the power may pass the fp32 range
  const int sh = (ex == 0 || ex == 255) ? 0 : TOP + 127 - ex;
  const float f1 = __uint_as_float((uint32_t)(127 + sh / 2) << 23), f2 = __uint_as_float((uint32_t)(127 + sh - sh / 2) << 23);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 y = __fmul2_rn(__fmul2_rn(make_float2(bf16_lo(w[e]), bf16_hi(w[e])), make_float2(f1, f1)), make_float2(f2, f2));
    o[e] = pack_h2(y.x, y.y);
  }
  return scale / f1 / f2;
}
// 16 channels 16c .. of query row `row` of (b, KV head h), zero for padding
__device__ __forceinline__ bool load_query(const KiviTreeArgs& a, const TreeLens& len, int b, int h, int row, int c,
                                           uint32_t (&w)[8]) {
  const int di = div_by(row, a.rep);
  const bool real = row < a.N * a.rep.d && di < len.nd;
  uint4 u[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (real) {
    const uint4* src = reinterpret_cast<const uint4*>(
        a.q + (((size_t)b * a.N + di) * a.Hq + (size_t)h * a.rep.d + row - di * a.rep.d) * kD + 16 * c);
    u[0] = __ldg(src);
    u[1] = __ldg(src + 1);
  }
  w[0] = u[0].x; w[1] = u[0].y; w[2] = u[0].z; w[3] = u[0].w;
  w[4] = u[1].x; w[5] = u[1].y; w[6] = u[1].z; w[7] = u[1].w;
  return real;
}

// ======================================================================================
// Up to 16 rows: warp-wide products
// ======================================================================================
//
// Tokens (scores) and channels (values) are the 16 rows of an m16n8k16 product, the query rows its 8 columns:
//   S^T [16 tokens x 8 rows] = K . q^T,  O^T [16 channels x 8 rows] += V^T . P^T,
// so a row tile is 8 query rows (NT of them) and the unpacked codes are the A fragments. Fragment orders: the
// contraction over channels and the one over tokens may run in any order that both operands share, and output rows
// may be any channels; they are chosen so that a code word's halves are a fragment's register without moving single
// codes. Lane (n = lane / 4, q = lane % 4):
//  * Scores: the lane holds token rows n and n + 8 of a token tile and channels 32 q .. + 31 of those, i.e. its own
//    code words; k-step kk takes two channel pairs of them ((c, c + 8) at 2 bits, (c, c + 4) at 4 bits).
//  * Place n of eight is token n ^ (n >> 2 & 1): the four tokens a lane quartet reads for the value product then
//    lie in different banks.
//  * Values: the lane holds channels 16 n .. + 15, its own code word(s): rows n and n + 8 of channel tile t are
//    channels 16 n + 2 t and + 1.
//  * P^T turns from accumulator into B fragment by the 8 x 8 transposition of packed halves.
//  * Keys are not dequantized: sum_c q_c s_c (code_c - z_c) = sum_c (q_c s_c) code_c - sum_c (q_c s_c) z_c. A masked
//    half of a code word is the fp16 subnormal code 2^(k - 24), exact; the scales of the group go into the queries,
//    q s 2^-k = q' + q'' with q' its fp16 and q'' the exact rest as fp16, in both sums (with q' alone the output was off
//    by up to 7e-3, three times the bound of attention), and the second sum is a product with the zero-points as A.
//    The group's scales are taken times a power of two that puts the largest in [2^6, 2^7), the queries' rows likewise:
//    products reach 2^14, and scales down to 2^-20 of the largest keep their bits beside it (a dead channel has scale
//    1; times a fixed 2^10 for all groups of small scales, one such channel left errors of 0.17 at scales near 2^-16).
//  * Values: s (c - z) = s (c - c0) - (s z - c0 s) with the middle code c0: the first part is one fp16 (exact at 2 bits,
//    one rounding of at most 8 s at 4), the second one number per token and channel group. A product of its own has
//    the constants as its rows: s z as fp16, the exact rest of it, c0 s, and ones, whose sums are those of the rounded
//    weights, so that a weight's rounding leaves a row's weights a convex combination. Values are halved on the way in:
//    8 s passes the fp16 range for values near its end.
// Bound: instruction issue (53 % of the cycles) and fixed latencies. A group of 32 tokens costs a warp 940 instructions at
// 8 rows (counted over a launch, segment ends included): one a code pair for the keys, three for the values, 66 products.
// Measured (16 requests, 32 KV heads, 4K context, 2 bits): 102 us for 8 rows (208 MB, 2.0 TB/s, 30 % of the copy rate),
// 164 us for 16. Without q'' and with values dequantized to one fp16 it took 80 and 126 us, outside the bound of
// attention (max-abs 2e-3): worst error of random cases 7e-3, now 1.7e-3. Per-warp rings of two groups by cp.async
// (each lane copies what its warp reads, so no block barrier in the loop); four blocks of four warps an SM for 8 rows, two
// for 16, as the registers of the sums allow (three, with spills in the loop: 173 us). Five blocks of 96 registers for 8
// rows spilled in the loop: 105 us against 88 then.
constexpr int kMmaThreads = 128;
constexpr int kMmaWarps = kMmaThreads / 32;

// Bit position of pair j (of the 8 of 16 channels) inside the half it is masked in: 2-bit codes 0 .. 2, 3 .. 5 and 6, 7
// come from the word shifted by 0, 6 and 12, 4-bit codes 0, 1 and 2, 3 from shifts by 0 and 8.
template <int KB>
__host__ __device__ constexpr int pair_pos(int j) { return KB == 2 ? 2 * (j % 3) : 4 * (j % 2); }
template <int KB>
__device__ __forceinline__ uint32_t pair_codes(const uint32_t* w, int j) {  // w: the words of 16 channels
  const uint32_t u = KB == 2 ? w[0] >> (6 * (j / 3)) : w[j >> 2] >> (8 * ((j & 3) >> 1));
  return u & ((((1u << KB) - 1u) << pair_pos<KB>(j)) * 0x10001u);
}
// x 2^(SIGN pos) for pair j
template <int KB, int SIGN>
__device__ __forceinline__ uint32_t pos_scale(uint32_t x, int j) {
  const int k = pair_pos<KB>(j);
  return k == 0 ? x : as_u(__hmul2(as_h2(x), __float2half2_rn(SIGN > 0 ? (float)(1 << k) : 1.f / (float)(1 << k))));
}

template <int KB, int VB, int NT>  // NT: row tiles of 8
struct MmaLayout {
  using S = StageLayout<KB, VB, kGroupT>;
  static constexpr int kRows = 8 * NT;
  // resident blocks the registers (36 NT sums a thread) and the shared memory leave room for
  static constexpr int kBlocks = (NT == 1) ? 4 : 2;
  static constexpr int kStages = 2;            // of a warp's ring, one key group each
  static constexpr int kOffQ = kMmaWarps * kStages * S::kBytes;     // uint4 [4][NT][32 lanes]: B fragments of two k-steps
  static constexpr int kOffO = kOffQ + 4 * NT * 32 * 16;            // float [2][kRows][128]: sums on their way to a warp
  static constexpr int kOffMl = kOffO + 2 * kRows * kD * 4;         // float2 [4 warps][kRows]: m, l; [kRows]: the block's
  static constexpr int kOffMask = kOffMl + (kMmaWarps + 1) * kRows * 8;  // uint64 [kRows]
  static constexpr int kOffC = kOffMask + kRows * 8;                // float [kRows]: log2 units per score unit
  static constexpr int kOffAhead = kOffC + kRows * 4;               // Walk [4 warps]: the warp's next copy; Walk: the block's
  static constexpr int kOffFlag = kOffAhead + (kMmaWarps + 1) * 48;
  static constexpr int kSmem = kOffFlag + 16;
  static_assert(sizeof(Walk) <= 48, "a warp's place");
  static_assert(kSmem <= 232448 / kBlocks - 1024, "blocks per SM");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A fragments of the constants' product from a token pair's scales and zero-points of the lane's channel group: rows n
// (az) s z / 2 in an even lane row and what its rounding left in an odd one, rows n + 8 (ac) c0 s / 2 or 1. Returns s / 2.
template <int VB>
__device__ __forceinline__ __half2 constants(uint32_t s, uint32_t z, bool odd, uint32_t& az, uint32_t& ac) {
  const uint32_t s2 = halved(s), p = as_u(__hmul2(as_h2(s2), as_h2(z)));
  az = odd ? product_rest(s2, z, p) : p;
  ac = odd ? 0x3C003C00u : as_u(__hmul2(as_h2(s2), __float2half2_rn(kCentre<VB>)));
  return as_h2(s2);
}

template <int KB, int VB, int NT>
__global__ void __launch_bounds__(kMmaThreads, MmaLayout<KB, VB, NT>::kBlocks)
    kivi_tree_mma_kernel(const KiviTreeArgs a, const float scale_log2) {
  using L = MmaLayout<KB, VB, NT>;
  using S = StageLayout<KB, VB, kGroupT>;
  constexpr int kRows = L::kRows, kSt = L::kStages;
  extern __shared__ __align__(128) unsigned char sm[];
  uint4* qf = reinterpret_cast<uint4*>(sm + L::kOffQ);
  float* osum = reinterpret_cast<float*>(sm + L::kOffO);
  float2* ml = reinterpret_cast<float2*>(sm + L::kOffMl);
  float2* row_ml = ml + kMmaWarps * kRows;
  uint64_t* mask = reinterpret_cast<uint64_t*>(sm + L::kOffMask);
  float* rowc = reinterpret_cast<float*>(sm + L::kOffC);
  int* nonfinite = reinterpret_cast<int*>(sm + L::kOffFlag);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q4 = lane & 3, n8 = lane >> 2;
  const int rep = a.rep.d, rows_all = a.N * rep, seg_per_b = a.H;  // one row tile
  TreeShared* shared = reinterpret_cast<TreeShared*>(a.part);
  float* slots = reinterpret_cast<float*>(shared + gridDim.x);

  Walk& w = *reinterpret_cast<Walk*>(sm + L::kOffAhead + kMmaWarps * 48);  // the block's place, kept out of registers
  Walk& ahead = *reinterpret_cast<Walk*>(sm + L::kOffAhead + warp * 48);    // the warp's copies'
  int n;
  {
    Walk x;
    const int2 share = find_share(a, seg_per_b, lane, x);
    n = share.y - share.x;
    if (tid == 0) w = x;
    if (lane == 0) ahead = x;
  }
  TreeShared sh = {n > 0 ? kSegBegins : kSegNoWork, -1, 0, 0};
  if (n == 0) {
    if (tid == 0) shared[blockIdx.x] = sh;
    return;
  }
  // The warp's ring: its key group of tile i is in stage i % kSt, copied kSt - 1 tiles ahead by its own lanes.
  unsigned char* ring = sm + warp * kSt * S::kBytes;
  // the next copy: its first token among all tokens of the cache, its quantized keys and values (from there on), the
  // tiles left in its segment and in the share
  size_t c_tok = 0;
  int c_nk = 0, c_nv = 0, c_left = 0, c_all = n;
  auto aim = [&]() {
    c_tok = ((size_t)ahead.b * a.H + ahead.seg) * a.max_tokens + ahead.tile * kTile + 32 * warp;
    c_nk = ahead.len.nqk - ahead.tile * kTile - 32 * warp;
    c_nv = ahead.len.nqv - ahead.tile * kTile - 32 * warp;
    c_left = ahead.len.tiles - ahead.tile;
  };
  auto copy_next = [&](int stage) {  // one commit group per tile, also when there is nothing to copy
    if (c_all > 0) {
      unsigned char* st = ring + stage * S::kBytes + lane * 16;
      const int half = lane & 15;
      if (c_nk > 0) {  // a whole group or nothing
        const unsigned char* src = a.k_codes + c_tok * S::kKRow + lane * 16;
#pragma unroll
        for (int x = 0; x < S::kKRow / 16; ++x) cp_async16(st + x * 512, src + x * 512);
        cp_async16(st + S::kKs, (lane < 16 ? a.k_scale : a.k_zero) + c_tok / kGroupT * kD + half * 8);
      }
      if (c_nv > 0) {  // the rows behind n_quant_v are there, but not used
        const unsigned char* src = a.v_codes + c_tok * S::kVRow + lane * 16;
#pragma unroll
        for (int x = 0; x < S::kVRow / 16; ++x) cp_async16(st + S::kVc + x * 512, src + x * 512);
        cp_async16(st + S::kVs, (lane < 16 ? a.v_scale : a.v_zero) + c_tok * (kD / kGroupT) + half * 8);
      }
      c_tok += kTile;
      c_nk -= kTile;
      c_nv -= kTile;
      --c_all;
      if (--c_left == 0) {  // on to the next segment
        __syncwarp();
        if (lane == 0) {
          ahead.tile = ahead.len.tiles - 1;
          ahead.next(a, seg_per_b, c_all > 0);
          if (warp == 0 && c_all > 0) prefetch_fp16(a, ahead.len, (size_t)ahead.b * a.H + ahead.seg, 0, ahead.len.n);
        }
        __syncwarp();
        aim();
      }
    }
    cp_commit();
  };
  if (tid == 0) {
    *nonfinite = 0;
    prefetch_fp16(a, w.len, (size_t)w.b * a.H + w.seg, w.tile * kTile, w.len.n);
  }
  __syncwarp();
  aim();
#pragma unroll 1
  for (int i = 1; i < kSt; ++i) copy_next(i - 1);
  __syncthreads();  // w is there
  const CodeScale cs0;
  const int tok8 = n8 ^ ((n8 >> 2) & 1);                                       // the token at place n of eight
  const int ca = (2 * q4) ^ ((2 * q4 >> 2) & 1), cb = (2 * q4 + 1) ^ ((2 * q4 + 1) >> 2 & 1);  // at places 2 q, 2 q + 1

  int i = 0, st = 0;  // tiles done, the next one's stage
  while (i < n) {
    // ================= one segment's part: its queries =================
    const int h = w.seg;
#pragma unroll 1
    for (int x = tid; x < kRows * 8; x += kMmaThreads) {  // 8 lanes per row, 16 channels each
      const int r = x >> 3, c = x & 7;
      uint32_t u[8], o[8];
      const bool real = load_query(a, w.len, w.b, h, r, c, u);
      const float back = query_fp16<6>(u, o, scale_log2);
      uint4 x0, x1;
      pair_order<KB>(make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]), x0, x1);
      x0 = make_uint4(pos_scale<KB, -1>(x0.x, 0), pos_scale<KB, -1>(x0.y, 1), pos_scale<KB, -1>(x0.z, 2), pos_scale<KB, -1>(x0.w, 3));
      x1 = make_uint4(pos_scale<KB, -1>(x1.x, 4), pos_scale<KB, -1>(x1.y, 5), pos_scale<KB, -1>(x1.z, 6), pos_scale<KB, -1>(x1.w, 7));
      // lane (row % 8, c / 2); k-steps 4 (c % 2) .. + 3: (pair 0, pair 1) each, two steps a uint4
      uint4* dst = qf + (2 * (c & 1) * NT + (r >> 3)) * 32 + (r & 7) * 4 + (c >> 1);
      dst[0] = x0;
      dst[NT * 32] = x1;
      if (c == 0) {
        rowc[r] = back;
        mask[r] = real ? a.mask[(size_t)w.b * a.N + div_by(r, a.rep)] : 0ull;
      }
    }
    __syncthreads();  // queries staged
    float m[NT][2], cs[NT][2];  // of rows 8 nt + 2 q, + 1: maximum - kRaise, scale
    float o[NT][8][4], w0[NT][4];  // sums of s (c - c0), and of the constants and weights (below)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = -FLT_MAX;
        cs[nt][e] = rowc[8 * nt + 2 * q4 + e];
        w0[nt][e] = w0[nt][2 + e] = 0.f;
      }
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][t][e] = 0.f;
    }
    const int i_first = i, i_end = min(n, i + w.len.tiles - w.tile);
    // the warp's tokens of a tile: tw, .. + 31; how far it is from there to the ends of the quantized keys and values
    // and of the cached tokens
    int tw = w.tile * kTile + 32 * warp, to_k = w.len.nqk - tw, to_v = w.len.nqv - tw, to_n = w.len.n - tw;
    for (; i < i_end; ++i, tw += kTile, to_k -= kTile, to_v -= kTile, to_n -= kTile) {
      const unsigned char* stage = ring + st * S::kBytes;
      copy_next(st == 0 ? kSt - 1 : st - 1);  // into the stage of tile i - 1, which every lane has read
      st = st + 1 == kSt ? 0 : st + 1;
      cp_wait<kSt - 1>();
      __syncwarp();  // every lane's copies of tile i
      if (to_n > 0 || to_n + w.len.nd > 0) {
        // ---- scores: 2 tiles of 16 tokens ----
        float s[NT][2][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][t][e] = 0.f;
        if (__builtin_expect(to_k > 0, 1)) {
          uint32_t u[4][KB];  // code words of the lane's 32 channels, four tokens (octets of the group)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const unsigned char* p = stage + (8 * t + tok8) * S::kKRow + q4 * (4 * KB);
            if constexpr (KB == 2) {
              const uint2 v = *reinterpret_cast<const uint2*>(p);
              u[t][0] = v.x;
              u[t][1] = v.y;
            } else {
              const uint4 v = *reinterpret_cast<const uint4*>(p);
              u[t][0] = v.x;
              u[t][1] = v.y;
              u[t][2] = v.z;
              u[t][3] = v.w;
            }
          }
          float code_unit, zero_unit;  // what a sum of code products and one with the zero-points count
          {  // the group's scales and zero-points in pair order, in place: a lane takes 16 channels of one of them
            uint4* blk = reinterpret_cast<uint4*>(const_cast<unsigned char*>(stage) + S::kKs) + 2 * (lane & 15);
            uint4 x0, x1;
            pair_order<KB>(blk[0], blk[1], x0, x1);
            // The scales (lanes 0 .. 7) are taken times the power of two that puts the group's largest in [2^6, 2^7):
            // however small, and beside whatever larger ones, the others keep their bits in q' then.
            const __half2 t = __hmax2(__hmax2(__hmax2(__habs2(as_h2(x0.x)), __habs2(as_h2(x0.y))), __hmax2(__habs2(as_h2(x0.z)), __habs2(as_h2(x0.w)))),
                                      __hmax2(__hmax2(__habs2(as_h2(x1.x)), __habs2(as_h2(x1.y))), __hmax2(__habs2(as_h2(x1.z)), __habs2(as_h2(x1.w)))));
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, lane < 8 ? max(as_u(t) & 0xFFFFu, as_u(t) >> 16) : 0u);
            const int e = 21 - (int)(top >> 10);  // -10 .. 21
            if (lane < 8) {
              uint32_t* x[8] = {&x0.x, &x0.y, &x0.z, &x0.w, &x1.x, &x1.y, &x1.z, &x1.w};
              const __half2 f = as_h2((uint32_t)(min(e, 15) + 15) * 0x4000400u);
#pragma unroll
              for (int i = 0; i < 8; ++i) *x[i] = as_u(__hmul2(as_h2(*x[i]), f));
              if (e > 15) {  // the rest of a power past the largest fp16 one
                const __half2 f1 = as_h2((uint32_t)e * 0x4000400u);
#pragma unroll
                for (int i = 0; i < 8; ++i) *x[i] = as_u(__hmul2(as_h2(*x[i]), f1));
              }
            }
            code_unit = __uint_as_float((uint32_t)(127 + 24 - e) << 23);  // codes are 2^-24 of themselves in the products
            zero_unit = __uint_as_float((uint32_t)(127 - e) << 23);
            if (lane < 16) {
              blk[0] = x0;
              blk[1] = x1;
            }
            __syncwarp();
          }
          float zs[NT][4];  // sum q' z
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) zs[nt][e] = 0.f;
#pragma unroll
          for (int k2 = 0; k2 < 4; ++k2) {  // two k-steps: pairs j0 .. j0 + 3 of 16 channels
            const int j0 = 4 * (k2 & 1), hw = k2 >> 1;
            const uint4 sc = *reinterpret_cast<const uint4*>(stage + S::kKs + (32 * q4 + 8 * k2) * 2);
            const uint4 zp = *reinterpret_cast<const uint4*>(stage + S::kKz + (32 * q4 + 8 * k2) * 2);
            uint4 bq[NT][2];  // q s 2^-k and what its rounding left
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint4 x = qf[(k2 * NT + nt) * 32 + lane];
              bq[nt][0] = make_uint4(as_u(__hmul2(as_h2(x.x), as_h2(sc.x))), as_u(__hmul2(as_h2(x.y), as_h2(sc.y))),
                                     as_u(__hmul2(as_h2(x.z), as_h2(sc.z))), as_u(__hmul2(as_h2(x.w), as_h2(sc.w))));
              bq[nt][1] = make_uint4(product_rest(x.x, sc.x, bq[nt][0].x), product_rest(x.y, sc.y, bq[nt][0].y),
                                     product_rest(x.z, sc.z, bq[nt][0].z), product_rest(x.w, sc.w, bq[nt][0].w));
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                const uint4 y = bq[nt][p];
                mma_f16(zs[nt], zp.x, zp.x, zp.y, zp.y, pos_scale<KB, 1>(y.x, j0), pos_scale<KB, 1>(y.y, j0 + 1));
                mma_f16(zs[nt], zp.z, zp.z, zp.w, zp.w, pos_scale<KB, 1>(y.z, j0 + 2), pos_scale<KB, 1>(y.w, j0 + 3));
              }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const uint32_t* ua = u[2 * t] + hw * (KB / 2);
              const uint32_t* ub = u[2 * t + 1] + hw * (KB / 2);
#pragma unroll
              for (int kk = 0; kk < 2; ++kk) {
                const uint32_t a0 = pair_codes<KB>(ua, j0 + 2 * kk), a1 = pair_codes<KB>(ub, j0 + 2 * kk);
                const uint32_t a2 = pair_codes<KB>(ua, j0 + 2 * kk + 1), a3 = pair_codes<KB>(ub, j0 + 2 * kk + 1);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int p = 0; p < 2; ++p)
                    mma_f16(s[nt][t], a0, a1, a2, a3, kk ? bq[nt][p].z : bq[nt][p].x, kk ? bq[nt][p].w : bq[nt][p].y);
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e)  // the row's own factor last: with the units it may pass the fp32 range
                s[nt][t][e] = fmaf(s[nt][t][e], code_unit, -zs[nt][e & 1] * zero_unit) * cs[nt][e & 1];
        } else {  // fp16 rows: residual, drafted, or none
          const uint16_t* row[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) row[t] = fp16_key(a, w.len, w.b, h, tw + 8 * t + tok8);
#pragma unroll 1
          for (int hw = 0; hw < 2; ++hw) {
            uint4 x[4][2];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int e = 0; e < 2; ++e) x[t][e] = row8(row[t], 4 * q4 + 2 * hw + e);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              uint4 pa[2], pb[2];  // pairs of octets 2 t, 2 t + 1
              pair_order<KB>(x[2 * t][0], x[2 * t][1], pa[0], pa[1]);
              pair_order<KB>(x[2 * t + 1][0], x[2 * t + 1][1], pb[0], pb[1]);
#pragma unroll
              for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  const uint4 bq = qf[((2 * hw + k2) * NT + nt) * 32 + lane];
                  mma_f16(s[nt][t], pa[k2].x, pb[k2].x, pa[k2].y, pb[k2].y, pos_scale<KB, 1>(bq.x, 4 * k2), pos_scale<KB, 1>(bq.y, 4 * k2 + 1));
                  mma_f16(s[nt][t], pa[k2].z, pb[k2].z, pa[k2].w, pb[k2].w, pos_scale<KB, 1>(bq.z, 4 * k2 + 2), pos_scale<KB, 1>(bq.w, 4 * k2 + 3));
                }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[nt][t][e] *= cs[nt][e & 1];
        }
        // ---- softmax of the scores in log2 units; they are rounded before the maximum is taken from them, so that
        //      the largest one's weight is exact however large it is. Element e of tile t: octet 2 t + e / 2, row
        //      2 q + e % 2 ----
        const bool plain = to_n >= 32;
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) over = over || s[nt][t][e] - m[nt][e & 1] > kRaise + kSlack;
        if (!plain) {  // drafted tokens among the 32
          over = true;
          const uint64_t there = w.len.nd >= 64 ? ~0ull : (1ull << w.len.nd) - 1;
          const int dj = tok8 - to_n;  // the drafted token of the lane's first one (-31 .. : cached below 0)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint64_t mk = mask[8 * nt + 2 * q4 + e] & there;
              // bit 8 oct: the row sees the lane's token of that octet
              const uint32_t sees = dj >= 64 ? 0u : dj >= 0 ? (uint32_t)(mk >> dj) : ((uint32_t)(mk << -dj) | ((1u << -dj) - 1u));
#pragma unroll
              for (int oct = 0; oct < 4; ++oct)
                if (!((sees >> (8 * oct)) & 1u)) s[nt][oct >> 1][e + 2 * (oct & 1)] = -INFINITY;
            }
        }
        if (__builtin_expect(__any_sync(0xFFFFFFFFu, over), 0)) {
          // raise the maxima of the rows with a score past them
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = fmaxf(fmaxf(s[nt][0][e], s[nt][0][2 + e]), fmaxf(s[nt][1][e], s[nt][1][2 + e]));
#pragma unroll
              for (int off = 4; off <= 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
              if (mx - m[nt][e] > kRaise + kSlack) {
                const float f = exp2_approx(m[nt][e] - (mx - kRaise));
                m[nt][e] = mx - kRaise;
                w0[nt][e] *= f;
                w0[nt][2 + e] *= f;
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                  o[nt][t][e] *= f;
                  o[nt][t][2 + e] *= f;
                }
              }
            }
        }
        uint32_t pf[NT][4];  // weights: B fragments of the two 16-token steps
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int oc = 0; oc < 2; ++oc) {
              const float p0 = exp2_approx(s[nt][t][2 * oc] - m[nt][0]), p1 = exp2_approx(s[nt][t][2 * oc + 1] - m[nt][1]);
              pf[nt][2 * t + oc] = transpose8(pack_h2(p0, p1));
            }
        // ---- values: token pairs at places 2 q, 2 q + 1 of the four octets ----
        if (__builtin_expect(to_v >= 32, 1)) {
          const uint16_t* sp = reinterpret_cast<const uint16_t*>(stage + S::kVs) + (n8 >> 1);
          const uint16_t* zp = reinterpret_cast<const uint16_t*>(stage + S::kVz) + (n8 >> 1);
          const unsigned char* cw = stage + S::kVc + n8 * (2 * VB);
          __half2 sv[4];
          uint32_t az[4], ac[4];
          uint32_t wa[4][VB / 2], wb[4][VB / 2];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int ta = 8 * t + ca, tb = 8 * t + cb;
            if constexpr (VB == 2) {
              wa[t][0] = *reinterpret_cast<const uint32_t*>(cw + ta * S::kVRow);
              wb[t][0] = *reinterpret_cast<const uint32_t*>(cw + tb * S::kVRow);
            } else {
              const uint2 va = *reinterpret_cast<const uint2*>(cw + ta * S::kVRow), vb = *reinterpret_cast<const uint2*>(cw + tb * S::kVRow);
              wa[t][0] = va.x;
              wa[t][1] = va.y;
              wb[t][0] = vb.x;
              wb[t][1] = vb.y;
            }
            sv[t] = constants<VB>(sp[ta * 4] | ((uint32_t)sp[tb * 4] << 16), zp[ta * 4] | ((uint32_t)zp[tb * 4] << 16), n8 & 1, az[t], ac[t]);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(w0[nt], az[2 * k], ac[2 * k], az[2 * k + 1], ac[2 * k + 1], pf[nt][2 * k], pf[nt][2 * k + 1]);
          constexpr int kCodes = 16 / VB;  // channels of a half word
#pragma unroll
          for (int hw = 0; hw < VB; ++hw) {  // half words of the lane's 16 channels
            uint32_t x[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) x[t] = __byte_perm(wa[t][hw >> 1], wb[t][hw >> 1], (hw & 1) ? 0x7632 : 0x5410);
#pragma unroll
            for (int c = 0; c < kCodes; c += 2)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t af[4];
#pragma unroll
                for (int oc = 0; oc < 2; ++oc)
#pragma unroll
                  for (int f = 0; f < 2; ++f)
                    af[2 * oc + f] = as_u(__hmul2(code_h2<VB, kCentre<VB>>(cs0, x[2 * k + oc], c + f), sv[2 * k + oc]));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_f16(o[nt][(hw * kCodes + c) / 2], af[0], af[1], af[2], af[3], pf[nt][2 * k], pf[nt][2 * k + 1]);
              }
          }
        } else {  // fp16 rows, and the group in which the quantized values end
          const int place = a.residual > 0 ? tw - div_by(tw, a.ring) * a.residual : 0;
          {  // the stored tokens' constants; of the others none but the weights
            uint32_t az[4], ac[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              uint32_t s2 = 0, z2 = 0;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int tt = 8 * t + (e ? cb : ca), at = tt * 4 + (n8 >> 1);
                if (tt < to_v) {
                  s2 |= (uint32_t)reinterpret_cast<const uint16_t*>(stage + S::kVs)[at] << (16 * e);
                  z2 |= (uint32_t)reinterpret_cast<const uint16_t*>(stage + S::kVz)[at] << (16 * e);
                }
              }
              constants<VB>(s2, z2, n8 & 1, az[t], ac[t]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(w0[nt], az[2 * k], ac[2 * k], az[2 * k + 1], ac[2 * k + 1], pf[nt][2 * k], pf[nt][2 * k + 1]);
          }
#pragma unroll 1
          for (int hw = 0; hw < 2; ++hw) {  // channels 16 n8 + 8 hw .. + 7
            uint32_t x[8][4];  // octet y / 2, place 2 q + y % 2
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              const int tt = 8 * (y >> 1) + ((y & 1) ? cb : ca);
              const uint4 v = tt < to_v
                                  ? make_uint4(0u, 0u, 0u, 0u)
                                  : row8(fp16_value(a, w.len, w.b, h, tw + tt, ring_place(place, tt, a.residual)), 2 * n8 + hw);
              x[y][0] = halved(v.x);
              x[y][1] = halved(v.y);
              x[y][2] = halved(v.z);
              x[y][3] = halved(v.w);
            }
            if (to_v > 0) {
#pragma unroll
              for (int y = 0; y < 8; ++y) {
                const int tt = 8 * (y >> 1) + ((y & 1) ? cb : ca);
                if (tt < to_v) {
                  const uint32_t cwd = *reinterpret_cast<const uint32_t*>(stage + S::kVc + tt * S::kVRow + n8 * (2 * VB) + (VB == 4 ? 4 * hw : 0)) >> (VB == 2 ? 16 * hw : 0);
                  const int at = tt * 4 + (n8 >> 1);
                  const uint4 v = centred8<VB>(cs0, cwd, as_h2(halved(reinterpret_cast<const uint16_t*>(stage + S::kVs)[at] * 0x10001u)));
                  x[y][0] = v.x;
                  x[y][1] = v.y;
                  x[y][2] = v.z;
                  x[y][3] = v.w;
                }
              }
            }
            if (!plain) {
              // A drafted value is seen only by the rows whose mask has it, but the product multiplies it by
              // every row's weight, 0 for the others: one that is not finite is taken as 0 and added at the
              // end to the rows that see it.
              const __half2 nil = __float2half2_rn(0.f);
              __half2 z = nil;  // 0 times a number that is not finite is not 0
#pragma unroll
              for (int y = 0; y < 8; ++y)
                if (8 * (y >> 1) + ((y & 1) ? cb : ca) >= to_n) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) z = __hfma2(as_h2(x[y][e]), nil, z);
                }
              if (__builtin_expect(!__hbeq2(z, nil), 0)) {
                *nonfinite = 1;
#pragma unroll
                for (int y = 0; y < 8; ++y)
                  if (8 * (y >> 1) + ((y & 1) ? cb : ca) >= to_n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) drop_nonfinite(x[y][e]);
                  }
              }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)  // channels 2 c, 2 c + 1 of the eight
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t af[4];
#pragma unroll
                for (int oc = 0; oc < 2; ++oc)
#pragma unroll
                  for (int f = 0; f < 2; ++f)
                    af[2 * oc + f] = __byte_perm(x[4 * k + 2 * oc][c], x[4 * k + 2 * oc + 1][c], f ? 0x7632 : 0x5410);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  if (hw == 0) mma_f16(o[nt][c], af[0], af[1], af[2], af[3], pf[nt][2 * k], pf[nt][2 * k + 1]);
                  else mma_f16(o[nt][4 + c], af[0], af[1], af[2], af[3], pf[nt][2 * k], pf[nt][2 * k + 1]);
                }
              }
          }
        }
      }
      __syncwarp();  // the stage is read
    }

    // ================= the segment ends here (or the share does): hand its sums on =================
    const int tile_first = w.tile, t_end = tile_first + i - i_first;  // tiles of the segment that are done
    const bool last = t_end == w.len.tiles, earlier = tile_first > 0 && i_first == 0;
    const bool whole = last && !earlier;
    // the sum of weights, and the constants' part of the sums: lanes n and n ^ 1 hold them for their channel group
    float l[NT][2], wc[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float z = w0[nt][e] + __shfl_xor_sync(0xFFFFFFFFu, w0[nt][e], 4);
        const float y = __shfl_xor_sync(0xFFFFFFFFu, w0[nt][2 + e], 4);
        l[nt][e] = (n8 & 1) ? w0[nt][2 + e] : y;
        wc[nt][e] = ((n8 & 1) ? y : w0[nt][2 + e]) - z;
        if (n8 == 0) ml[warp * kRows + 8 * nt + 2 * q4 + e] = make_float2(m[nt][e], l[nt][e]);
      }
    __syncthreads();
    // every warp's sums against the block's maximum; warps 2, 3 hand theirs to 0, 1, which leave two for all to add
    auto top = [&](int r) {
      float x = ml[r].x;
#pragma unroll
      for (int k = 1; k < kMmaWarps; ++k) x = fmaxf(x, ml[k * kRows + r].x);
      return x;
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // values were halved
        const float f = l[nt][e] == 0.f ? 0.f : 2.f * exp2_approx(m[nt][e] - top(8 * nt + 2 * q4 + e));
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          o[nt][t][e] = f == 0.f ? 0.f : (o[nt][t][e] + wc[nt][e]) * f;
          o[nt][t][2 + e] = f == 0.f ? 0.f : (o[nt][t][2 + e] + wc[nt][e]) * f;
        }
      }
    if (tid < kRows) {
      const float mr = top(tid);
      float lr = 0.f;
#pragma unroll
      for (int k = 0; k < kMmaWarps; ++k) {
        const float2 v = ml[k * kRows + tid];
        if (v.y != 0.f) lr += v.y * exp2_approx(v.x - mr);  // 0: the row saw nothing there
      }
      row_ml[tid] = make_float2(mr, lr);
    }
    float* mine = osum + (warp & 1) * kRows * kD + lane;
    auto element = [](int nt, int t, int e) { return ((nt * 8 + t) * 4 + e) * 32; };
    if (warp >= 2) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) mine[element(nt, t, e)] = o[nt][t][e];
    }
    __syncthreads();
    if (warp < 2) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) mine[element(nt, t, e)] += o[nt][t][e];
    }
    __syncthreads();
    if (earlier) sh.first = last ? kSegEnds : kSegGoesOn;
    else if (!last) {
      sh.open = w.b * seg_per_b + w.seg;
      sh.nd = w.len.nd;
    }
    float* slot = slots + ((size_t)blockIdx.x * 2 + (earlier ? 0 : 1)) * slot_floats<kRows>();
    const bool fix = *nonfinite != 0;
#pragma unroll 1
    for (int x = 0; x < 2 * NT; ++x) {  // row 8 nt + 2 q + e, channels 16 n + 4 warp .. + 3: o[nt][2 warp + c / 2][e + 2 (c % 2)]
      const int nt = x >> 1, e = x & 1, r = 8 * nt + 2 * q4 + e, di = div_by(r, a.rep), ch = 16 * n8 + 4 * warp;
      if (r >= rows_all || di >= w.len.nd) continue;  // padding
      const float* s0 = osum + element(nt, 2 * warp, e) + lane;
      float v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = s0[64 * c] + s0[kRows * kD + 64 * c];
      if (fix) {  // of the drafted tokens in this block's tiles
        const int j1 = min(w.len.nd, t_end * kTile - w.len.n);
#pragma unroll 1
        for (int j = max(0, tile_first * kTile - w.len.n); j < j1; ++j) {
          if (!((mask[r] >> j) & 1ull)) continue;
          const uint16_t* d = a.v_draft + (((size_t)w.b * a.N + j) * a.H + h) * kD + ch;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if ((d[c] & 0x7C00u) == 0x7C00u) v[c] += th2f(d[c]);
        }
      }
      const float2 t = row_ml[r];
      float* to = slot + (size_t)r * kD + ch;
      if (whole) {
        const float inv = (t.y > 0.f || t.y != t.y) ? 1.f / t.y : 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = inv == 0.f ? 0.f : v[c] * inv;
        const size_t at = (((size_t)w.b * a.N + di) * a.Hq + (size_t)h * rep + r - di * rep) * kD + ch;
        to = reinterpret_cast<float*>(a.out) + at;
        if (!a.out_fp32)
          *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at) =
              make_uint2(f32_to_bf16(v[0]) | ((uint32_t)f32_to_bf16(v[1]) << 16), f32_to_bf16(v[2]) | ((uint32_t)f32_to_bf16(v[3]) << 16));
      } else if (n8 == 0 && warp == 0) {
        slot[(size_t)kRows * kD + r] = t.x;
        slot[(size_t)kRows * kD + kRows + r] = t.y;
      }
      if (!whole || a.out_fp32) *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
    }
    __syncthreads();  // the queries, the row state and the place are read before the next segment's
    if (tid == 0) {
      *nonfinite = 0;
      w.tile = t_end - 1;
      w.next(a, seg_per_b, i < n);
    }
    __syncthreads();
  }
  if (tid == 0) shared[blockIdx.x] = sh;
}

// ======================================================================================
// More rows: tcgen05 on tiles of 32 or 64 rows
// ======================================================================================
//
//   S^T [128 tokens x rows] = K [128 x 128] . q^T      K = s (c - c0) as fp16 in shared memory (4 bits: in two parts)
//   P^T = exp2(S^T c - m)                               a thread owns a token and half the rows
//   O^T [128 channels x rows] += V^T [128 x 128] . P^T  V^T = s (c - c0) as fp16 in shared memory
// The constants s (z - c0) of a key group's channels, of a token's channel groups, and the sum of a row's weights come
// from products of their own (kConst below). Whether a running maximum has to move is a block-wide vote.
//
// Two blocks an SM, so that one's products, copies and barriers run beside the other's unpacking and softmax. The next
// tile's stored keys and values are on their way (bulk copies) from the moment this tile's are unpacked, and its keys
// are unpacked into registers while this tile's value product still reads the weights, which lie where the keys were.
//
// Bound: no single unit (16 requests, 8 KV heads, 192 rows, 4K context, 4 bits: 247 us; issue 41 % of the cycles, ALU
// 28 %, tensor 22 %, shared-memory wavefronts 58 %, DRAM 6 %), but the chain of a tile: unpacking, the
// products, the softmax with what raises maxima, barriers. 175 us of it are the same kernel with keys and values dequantized
// to one fp16, outside the bound of attention (max-abs 2e-3): worst error of random cases 3.7e-2, now 1.2e-3. Of the rest
// the constants' products cost 24, reading the keys' ones back 10, the keys' second parts and the constants themselves 38.
// Measured with the one-fp16 form and not kept: four more warps a block (64 registers, 234 us against 191 then), copies and
// products issued by warps of their own with the registers that costs (238; four roles with code of their own 463),
// the softmax in pieces of 16 rows with the scores read twice (212), weights before the vote (194).
constexpr int kTreeThreads = 256;

// V^T is staged in 8 channel x 8 token core matrices: the 16 of a row group (8 channels) are contiguous, row
// groups 2064 bytes apart, so that eight threads with eight row groups store to different banks
constexpr int kVRowGrp = (kTile / 8) * 128 + 16;

// The constants of a tile's keys (s z - c0 s of each channel) and values (of each token) as rows of a product of their
// own: 16 rows of 8 elements for each 8 channels or tokens, kConst bytes apart. Row 4 g + i is constant i of group g; with
// 16 bytes from row group to row group of the 128 the tensor core takes, lane 32 g + i of the result is that row, for
// i < 8, so that a group's constants come out beside its tokens or channels. The other lanes' sums are not used.
constexpr int kConst = 16 * 16 + 16;            // (+ 16: neighbours in different banks)
constexpr int kConstBytes = 16 * kConst + 128;  // with what the last row groups reach past them

struct Place : Walk {
  int h, row0;  // KV head, first row
};

template <int KB, int VB, int ROWS>
struct TreeLayout {
  static constexpr int kOffQ = 0;                                  // fp16 [ROWS x 128], K-major
  static constexpr int kOffK = kOffQ + ROWS * kD * 2;              // fp16 [128 tokens x 128], K-major; then P
  static constexpr int kOffV = kOffK + kTile * kD * 2;             // fp16 [128 channels x 128 tokens], K-major
  static constexpr int kOffZ = (kOffV + (kD / 8) * kVRowGrp + 127) / 128 * 128;  // constants of the keys
  static constexpr int kOffW = kOffZ + kConstBytes;                // and of the values
  static constexpr int kOffStage = kOffW + kConstBytes;
  static constexpr int kOffMask = kOffStage + StageLayout<KB, VB, kTile>::kBytes;  // uint64 [ROWS]
  static constexpr int kOffC = kOffMask + ROWS * 8;                // float [ROWS]: log2 units per score unit
  static constexpr int kOffM = kOffC + ROWS * 4;                   // float [ROWS]: kRaise - running maximum (log2)
  static constexpr int kOffF = kOffM + ROWS * 4;                   // float [ROWS]: rescale factor
  static constexpr int kOffRed = kOffF + ROWS * 4;                 // float [2][4][ROWS]: per lane quadrant
  static constexpr int kOffUnit = kOffRed + 8 * ROWS * 4;          // float [2][4]: what a key group's sums count
  static constexpr int kOffWalk = kOffUnit + 32;                   // Place [2]: this position's and the next one's
  static constexpr int kOffBar = kOffWalk + 96;                    // mbarriers, TMEM address, flags
  static constexpr int kSmem = kOffBar + 64;
  static constexpr uint32_t kCols = 4 * ROWS;  // TMEM: S^T, O^T, and the sums of the keys' and values' constants
  static_assert(ROWS * 256 <= kTile * kD * 2, "P fits in the key tile");
  static_assert((kD / 8) * kVRowGrp >= kTile * kD * 2, "the keys' second parts fit in the value tile");
  static_assert(kSmem <= 232448 / 2 - 1024, "two blocks per SM");
};

// shared-memory matrix descriptor, no swizzle. K-major: lbo steps 8 elements along K, sbo 8 rows;
// MN-major: lbo steps 8 along K, sbo 8 along N
__device__ __forceinline__ uint64_t tree_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}
// instruction descriptor, kind::f16: fp32 D, fp16 A (K-major) and B, M = 128
__host__ __device__ constexpr uint32_t tree_idesc(int n, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void umma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tree_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// eight consecutive fp32 columns of this thread's TMEM lane (valid after tmem_wait_ld)
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
  tmem_wait_ld();
  return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(v)) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}

// the largest of the lanes' values that are numbers
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(x));
  return r;
}
// ---- keys of a tile. A lane takes token lane % 8 of an octet and a code word (2 bits: 16 channels, 4 bits: 8);
//      a warp one key group and half of the words, so a lane unpacks four tokens per scale. Groups behind the
//      quantized keys are fp16 rows.
//      A stored key enters as s (c - c0), exact in one fp16 at 2 bits and in two at 4 (`rest`), the scales times a power
//      of two that puts the group's largest in [2^11, 2^12); its constants s (z - c0), times one of their own, as two
//      rows of `consts`. unit: what their sums count.
//      free() waits until the tile may be written: the codes are unpacked into registers before. ----
template <int KB, typename F>
__device__ __forceinline__ void unpack_keys(const CodeScale& cs0, const KiviTreeArgs& a, const TreeLens& len, int b, int h, int t0,
                                            const unsigned char* codes, const unsigned char* scale,
                                            const unsigned char* zero, unsigned char* dst0, unsigned char* rest0,
                                            unsigned char* consts, float* unit, int warp, int lane, F free) {
  constexpr int kRow = kD * KB / 8;
  const int g = warp & 3, tok = 32 * g + (lane & 7);
  if (t0 + 32 * g < len.nqk) {
    constexpr int kBlocks = (KB == 2) ? 1 : 2;   // of four words
    constexpr int kPairs = (KB == 2) ? 8 : 4;    // channel pairs of a word
    const int w0 = (warp >> 2) * 4 * kBlocks + (lane >> 3);
    scale += g * kD * 2;
    zero += g * kD * 2;
    const uint2 four = *reinterpret_cast<const uint2*>(scale + 8 * lane);
    const __half2 t = __hmax2(__habs2(as_h2(four.x)), __habs2(as_h2(four.y)));
    const int e = 26 - (int)(__reduce_max_sync(0xFFFFFFFFu, max(as_u(t) & 0xFFFFu, as_u(t) >> 16)) >> 10);  // -5 .. 26
    if (warp < 4) {
      // the lane's pairs j, j + 1 of 16 channels, j = 2 (lane % 4), in pair order
      const int j = lane & 3, ch = 16 * (lane >> 2) + (KB == 2 ? 2 * j : 8 * (j >> 1) + 2 * (j & 1));
      constexpr int kTo = KB == 2 ? 8 : 4;  // channels of a pair are kTo apart
      float2 y[2];
      float most = 0.f;
      {
        const float2 sa = __half22float2(as_h2(*reinterpret_cast<const uint32_t*>(scale + 2 * ch)));
        const float2 sb = __half22float2(as_h2(*reinterpret_cast<const uint32_t*>(scale + 2 * (ch + kTo))));
        const float2 za = __half22float2(as_h2(*reinterpret_cast<const uint32_t*>(zero + 2 * ch)));
        const float2 zb = __half22float2(as_h2(*reinterpret_cast<const uint32_t*>(zero + 2 * (ch + kTo))));
        constexpr float c0 = kCentre<KB>;
        y[0] = make_float2(sa.x * (za.x - c0), sb.x * (zb.x - c0));
        y[1] = make_float2(sa.y * (za.y - c0), sb.y * (zb.y - c0));
      }
      most = fmaxf(fmaxf(fabsf(y[0].x), fabsf(y[0].y)), fmaxf(fabsf(y[1].x), fabsf(y[1].y)));
      // the largest in [2^13, 2^14)
      const int top = (int)(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most)) >> 23), sh = min(140 - top, 64);
      const float f = __uint_as_float((uint32_t)(127 + sh) << 23);
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        y[i] = __fmul2_rn(y[i], make_float2(f, f));
        hi[i] = pack_h2(y[i].x, y[i].y);
        const float2 back = __half22float2(as_h2(hi[i]));
        lo[i] = pack_h2(y[i].x - back.x, y[i].y - back.y);
      }
      unsigned char* at = consts + (2 * (lane >> 2) + (j >> 1)) * kConst + 4 * g * 16 + (j & 1) * 8;
      *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(at + 16) = make_uint2(lo[0], lo[1]);
      if (lane == 0) {
        unit[g] = __uint_as_float((uint32_t)(127 - e) << 23);
        unit[4 + g] = __uint_as_float((uint32_t)(127 - sh) << 23);
      }
    }
    uint32_t o[kBlocks][4][kPairs], r[KB == 4 ? kBlocks : 1][4][kPairs];
    const __half2 f0 = as_h2((uint32_t)(min(e, 15) + 15) * 0x4000400u), f1 = as_h2((uint32_t)(max(e, 15)) * 0x4000400u);
#pragma unroll
    for (int blk = 0; blk < kBlocks; ++blk) {
      const int w = w0 + 4 * blk;
      __half2 s[kPairs];
      const uint4* sp = reinterpret_cast<const uint4*>(scale + 2 * kPairs * w * 2);
      {
        uint4 s0, s1;
        pair_order<KB>(sp[0], sp[KB == 2 ? 1 : 0], s0, s1);
        const uint32_t sw[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int j = 0; j < kPairs; ++j) s[j] = __hmul2(as_h2(sw[j]), f0);
        if (e > 15) {  // the rest of a power past the largest fp16 one
#pragma unroll
          for (int j = 0; j < kPairs; ++j) s[j] = __hmul2(s[j], f1);
        }
      }
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const uint32_t*>(codes + (tok + 8 * i) * kRow + 4 * w);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const __half2 c = code_h2<KB, kCentre<KB>>(cs0, u[i], j);
          o[blk][i][j] = as_u(__hmul2(c, s[j]));
          if constexpr (KB == 4) r[blk][i][j] = product_rest(as_u(c), as_u(s[j]), o[blk][i][j]);
        }
    }
    free();
#pragma unroll
    for (int blk = 0; blk < kBlocks; ++blk)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = tok + 8 * i, at = (t >> 3) * 2048 + (w0 + 4 * blk) * (kPairs * 32) + (t & 7) * 16;
        const uint32_t(&x)[kPairs] = o[blk][i];
        *reinterpret_cast<uint4*>(dst0 + at) = make_uint4(x[0], x[1], x[2], x[3]);
        if constexpr (KB == 2) {
          *reinterpret_cast<uint4*>(dst0 + at + 128) = make_uint4(x[4], x[5], x[6], x[7]);
        } else {
          const uint32_t(&y)[kPairs] = r[blk][i];
          *reinterpret_cast<uint4*>(rest0 + at) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
  } else {
    const int c = (warp >> 2) * 4 + (lane >> 3);  // 16 channels c
    uint4 x[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint16_t* row = fp16_key(a, len, b, h, t0 + tok + 8 * i);
      x[i][0] = row8(row, 2 * c);
      x[i][1] = row8(row, 2 * c + 1);
    }
    free();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = tok + 8 * i, at = (t >> 3) * 2048 + c * 256 + (t & 7) * 16;
      uint4 x0, x1;
      pair_order<KB>(x[i][0], x[i][1], x0, x1);
      *reinterpret_cast<uint4*>(dst0 + at) = x0;
      *reinterpret_cast<uint4*>(dst0 + at + 128) = x1;
      if constexpr (KB == 4) {
        *reinterpret_cast<uint4*>(rest0 + at) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(rest0 + at + 128) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
}

// ---- values of a tile, transposed. A thread takes a token octet and eight channels; octets with tokens behind
//      the quantized values mix stored tokens and fp16 rows. Stored values enter as s (c - c0), their constants as rows
//      of `consts` (of four threads with one channel group each writes one: s z, the rest of it, c0 s, and ones, which
//      stay), all of them halved: 8 s passes the fp16 range for values near its end.
//      free() waits until the tile may be written. ----
template <int VB, typename F>
__device__ __forceinline__ void unpack_values(const CodeScale& cs0, const KiviTreeArgs& a, const TreeLens& len, int b, int h, int t0,
                                              const unsigned char* codes, const unsigned char* scale,
                                              const unsigned char* zero, unsigned char* dst0, unsigned char* consts,
                                              int* nonfinite, int warp, int lane, F free) {
  constexpr int kRow = kD * VB / 8;
  const int c = lane & 15, oct = 2 * warp + (lane >> 4), flip = oct & 1;
  unsigned char* dst = dst0 + c * kVRowGrp + oct * 128;
  const unsigned char* cw = codes + 8 * oct * kRow + ((VB == 2) ? (c >> 1) : c) * 4;
  const uint16_t* sp = reinterpret_cast<const uint16_t*>(scale) + 8 * oct * 4 + (c >> 2);
  const uint16_t* zp = reinterpret_cast<const uint16_t*>(zero) + 8 * oct * 4 + (c >> 2);
  const int n = len.nqv - t0 - 8 * oct;  // stored tokens from the octet's first
  uint32_t w[8], s2[4], y[4];  // place i of the octet: token i ^ flip
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const uint32_t*>(cw + (i ^ flip) * kRow);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int ta = (2 * i) ^ flip, tb = (2 * i + 1) ^ flip;
    uint32_t z2;
    s2[i] = z2 = 0;  // of tokens behind the stored ones
    if (ta < n) {
      s2[i] = sp[4 * ta];
      z2 = zp[4 * ta];
    }
    if (tb < n) {
      s2[i] |= (uint32_t)sp[4 * tb] << 16;
      z2 |= (uint32_t)zp[4 * tb] << 16;
    }
    s2[i] = halved(s2[i]);
    const uint32_t p = as_u(__hmul2(as_h2(s2[i]), as_h2(z2)));
    y[i] = (c & 3) == 0 ? p : (c & 3) == 1 ? product_rest(s2[i], z2, p) : as_u(__hmul2(as_h2(s2[i]), __float2half2_rn(kCentre<VB>)));
  }
  free();
  if ((c & 3) < 3) *reinterpret_cast<uint4*>(consts + oct * kConst + c * 16) = make_uint4(y[0], y[1], y[2], y[3]);
  if (n > 0) {
    if constexpr (VB == 2) {
      const uint32_t sel = (c & 1) ? 0x7632u : 0x5410u;
      uint32_t x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __byte_perm(w[2 * i], w[2 * i + 1], sel);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = as_u(__hmul2(code_h2<2, kCentre<2>>(cs0, x[i], e), as_h2(s2[i])));
        *reinterpret_cast<uint4*>(dst + e * 16) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    } else {
#pragma unroll
      for (int hw = 0; hw < 2; ++hw) {
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __byte_perm(w[2 * i], w[2 * i + 1], hw ? 0x7632 : 0x5410);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = as_u(__hmul2(code_h2<4, kCentre<4>>(cs0, x[i], e), as_h2(s2[i])));
          *reinterpret_cast<uint4*>(dst + (4 * hw + e) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
  }
  if (t0 + 8 * oct + 8 > len.nqv) {
    // tokens behind the quantized values, over what was unpacked for them from the end of the stage
    const int t8 = t0 + 8 * oct, place = a.residual > 0 ? t8 - div_by(t8, a.ring) * a.residual : 0;
#pragma unroll 1
    for (int i = 0; i < 8; i += 4) {
      uint4 u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = make_uint4(0u, 0u, 0u, 0u);
        if (t8 + i + e >= len.nqv) u[e] = row8(fp16_value(a, len, b, h, t8 + i + e, ring_place(place, i + e, a.residual)), c);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = t8 + i + e;
        if (t < len.nqv) continue;
        uint32_t x[4] = {halved(u[e].x), halved(u[e].y), halved(u[e].z), halved(u[e].w)};
        // A drafted value is seen only by the rows whose mask has it, but the product multiplies it by every row's
        // weight, 0 for the others: one that is not finite is staged as 0 and added at the end to the rows that see it.
        if (t >= len.n) {
          const __half2 nil = __float2half2_rn(0.f);
          const __half2 z = __hfma2(as_h2(x[0]), nil, __hfma2(as_h2(x[1]), nil, __hfma2(as_h2(x[2]), nil, __hmul2(as_h2(x[3]), nil))));
          if (!__hbeq2(z, nil)) {  // 0 times a number that is not finite is not 0
#pragma unroll
            for (int y = 0; y < 4; ++y) drop_nonfinite(x[y]);
            *nonfinite = 1;
          }
        }
        unsigned char* at = dst + ((i + e) ^ flip) * 2;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          *reinterpret_cast<uint16_t*>(at + 32 * y) = (uint16_t)x[y];
          *reinterpret_cast<uint16_t*>(at + 32 * y + 16) = (uint16_t)(x[y] >> 16);
        }
      }
    }
  }
}

template <int KB, int VB, int ROWS>
__global__ void __launch_bounds__(kTreeThreads, 2) kivi_tree_kernel(const KiviTreeArgs a, const float scale_log2) {
  using L = TreeLayout<KB, VB, ROWS>;
  using S = StageLayout<KB, VB, kTile>;
  extern __shared__ __align__(128) unsigned char sm[];
  uint64_t* mask = reinterpret_cast<uint64_t*>(sm + L::kOffMask);
  float* rowc = reinterpret_cast<float*>(sm + L::kOffC);
  float* rowm = reinterpret_cast<float*>(sm + L::kOffM);
  float* rowf = reinterpret_cast<float*>(sm + L::kOffF);
  float* red = reinterpret_cast<float*>(sm + L::kOffRed);
  float* unit = reinterpret_cast<float*>(sm + L::kOffUnit);
  uint64_t* bar_s = reinterpret_cast<uint64_t*>(sm + L::kOffBar);  // scores done
  uint64_t* bar_o = bar_s + 1;                                      // value product done
  uint64_t* bar_k = bar_s + 2;                                      // the tile's stored keys landed
  uint64_t* bar_v = bar_s + 3;                                      // its stored values
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_s + 4);
  volatile int* failed = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* nonfinite = reinterpret_cast<int*>(tmem_slot + 2);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rep = a.rep.d, rows_all = a.N * rep;
  const int seg_per_b = a.segs.d;

  TreeShared* shared = reinterpret_cast<TreeShared*>(a.part);
  float* slots = reinterpret_cast<float*>(shared + gridDim.x);
  Place* place = reinterpret_cast<Place*>(sm + L::kOffWalk);  // of position p in place[p & 1] (kept out of registers)
  auto place_of = [&](const Walk& x) {
    const int h = div_by(x.seg, a.row_tiles);
    return Place{x, h, (x.seg - h * a.row_tiles.d) * ROWS};
  };
  int p0, p1;
  {
    Walk x;
    const int2 share = find_share(a, seg_per_b, lane, x);
    p0 = share.x;
    p1 = share.y;
    if (tid == 0) place[p0 & 1] = place_of(x);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge's blocks take places that become free
  TreeShared sh = {p0 < p1 ? kSegBegins : kSegNoWork, -1, 0, 0};
  if (p0 >= p1) {
    if (tid == 0) shared[blockIdx.x] = sh;
    return;
  }

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(L::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  unsigned char* stage = sm + L::kOffStage;
  // by one thread each, of warps that issue no products
  auto keys_of = [&](const Place& x) {
    bulk_keys<KB, VB>(a, x.len, (size_t)x.b * a.H + x.h, x.tile * kTile, stage, bar_k);
  };
  auto values_of = [&](const Place& x) {
    const size_t bh = (size_t)x.b * a.H + x.h;
    bulk_values<KB, VB>(a, x.len, bh, x.tile * kTile, stage, bar_v);
    prefetch_fp16(a, x.len, bh, x.tile * kTile, (x.tile + 1) * kTile);
  };
  if (tid == 0) {
    mbar_init(bar_s, 1);
    mbar_init(bar_o, 1);
    mbar_init(bar_k, 1);
    mbar_init(bar_v, 1);
    *failed = 0;
    *nonfinite = 0;
    fence_mbar_init();
  }
  // the rows of ones among the values' constants: their sums are those of the weights
  if (tid < 64) *reinterpret_cast<uint4*>(sm + L::kOffW + (tid & 15) * kConst + (4 * (tid >> 4) + 3) * 16) = make_uint4(0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u);
  tmem_before();
  __syncthreads();
  tmem_after();
  if (tid == 96) keys_of(place[p0 & 1]);
  if (tid == 224) values_of(place[p0 & 1]);
  const uint32_t tmem = *tmem_slot;
  const int quad = warp & 3, half = warp >> 2;            // TMEM lane quadrant, half of the rows
  const uint32_t t_lane = tmem + ((uint32_t)(32 * quad) << 16);
  constexpr int kHR = ROWS / 2;                            // rows a thread works on
  const int r0 = half * kHR;
  uint32_t phase = 0;    // of the barriers: one completion each per tile
  // the operands' descriptors; a k-step further on is 256 bytes (16 units) further on, 2 kConst in the constants
  const uint64_t desc_k = tree_desc(smem_u32(sm + L::kOffK), 128, 2048), desc_q = tree_desc(smem_u32(sm + L::kOffQ), 128, 2048);
  const uint64_t desc_v = tree_desc(smem_u32(sm + L::kOffV), 128, kVRowGrp), desc_p = desc_k;  // P lies where K was
  const uint64_t desc_kr = tree_desc(smem_u32(sm + L::kOffV), 128, 2048);  // the keys' second parts, before the values
  const uint64_t desc_z = tree_desc(smem_u32(sm + L::kOffZ), kConst, 16), desc_w = tree_desc(smem_u32(sm + L::kOffW), kConst, 16);
  const CodeScale cs0;
  bool first = true;    // of the segment's tiles in this block
  int tile_first = 0;   // that tile
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!mbar_wait_bounded(bar, parity)) {
      *failed = 1;
      set_error(a.err, KVQ_ERR_TIMEOUT);
    }
  };

  for (int p = p0; p < p1; ++p) {
    const Place& w = place[p & 1];
    const Place& nw = place[(p + 1) & 1];
    const TreeLens& len = w.len;
    const int b = w.b, h = w.h, row0 = w.row0, tile = w.tile, t0 = tile * kTile;
    const bool last = w.last(), more = p + 1 < p1;
    if (tid == 32 && more) {  // shown to the others by the next barrier
      Walk x = w;
      x.next(a, seg_per_b, true);
      place[(p + 1) & 1] = place_of(x);
    }
    if (first) {
      // ---- the segment's query rows, masks and running state (8 lanes a row) ----
#pragma unroll 1  // run once per segment: fewer instructions to fetch
      for (int i = tid; i < ROWS * 8; i += kTreeThreads) {
        const int r = i >> 3, c = i & 7;
        uint32_t u[8], o[8];
        const bool real = load_query(a, len, b, h, row0 + r, c, u);
        const uint64_t sees = real ? a.mask[(size_t)b * a.N + div_by(row0 + r, a.rep)] : 0ull;
        const float back = query_fp16<14>(u, o, scale_log2);
        uint4 x0, x1;
        pair_order<KB>(make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]), x0, x1);
        unsigned char* dst = sm + L::kOffQ + (r >> 3) * 2048 + c * 256 + (r & 7) * 16;
        *reinterpret_cast<uint4*>(dst) = x0;
        *reinterpret_cast<uint4*>(dst + 128) = x1;
        if (c == 0) {
          rowc[r] = back;
          rowm[r] = FLT_MAX;
          mask[r] = sees;
        }
      }
      if (tid == 0) *nonfinite = 0;
      tile_first = tile;
    }
    wait(bar_k, phase);
    unpack_keys<KB>(cs0, a, len, b, h, t0, stage, stage + S::kKs, stage + S::kKz, sm + L::kOffK, sm + L::kOffV, sm + L::kOffZ, unit, warp, lane, [&]() {
      if (p > p0) wait(bar_o, phase ^ 1);  // the value product before has read its weights
      tmem_after();
    });
    fence_proxy_async_smem();
    tmem_before();
    if (__syncthreads_or(*failed)) break;
    if (tid == 0) {
      tmem_after();
#pragma unroll
      for (int k = 0; k < 8; ++k) umma_f16(tmem, desc_k + 16 * k, desc_q + 16 * k, tree_idesc(ROWS, false), k > 0);
      if constexpr (KB == 4) {
#pragma unroll
        for (int k = 0; k < 8; ++k) umma_f16(tmem, desc_kr + 16 * k, desc_q + 16 * k, tree_idesc(ROWS, false), 1);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        umma_f16(tmem + 2 * ROWS, desc_z + k * (2 * kConst / 16), desc_q + 16 * k, tree_idesc(ROWS, false), k > 0);
      tree_commit(bar_s);
    }
    if (tid == 96 && more) keys_of(nw);  // every thread has read this tile's
    wait(bar_v, phase);
    unpack_values<VB>(cs0, a, len, b, h, t0, stage + S::kVc, stage + S::kVs, stage + S::kVz, sm + L::kOffV, sm + L::kOffW, nonfinite, warp, lane, [&]() {
      if constexpr (KB == 4) wait(bar_s, phase);  // the score product has read the keys' second parts
    });
    wait(bar_s, phase);
    tmem_after();
    // ---- the constants' part of the scores of the warp's key group, negative: lanes 0 and 1 hold its two sums ----
    float* nz = red + quad * ROWS + r0;
    const bool stored = t0 + 32 * quad < len.nqk;
    if (stored) {
      uint32_t zr[kHR];
#pragma unroll
      for (int i = 0; i < kHR; i += 8) tmem_ld8(t_lane + 2 * ROWS + r0 + i, zr + i);
      tmem_wait_ld();
      if (lane < 2) {
#pragma unroll
        for (int i = 0; i < kHR; i += 4)
          *reinterpret_cast<uint4*>(nz + 4 * ROWS * lane + i) = make_uint4(zr[i], zr[i + 1], zr[i + 2], zr[i + 3]);
      }
      __syncwarp();
      if (lane < kHR) nz[lane] = -(nz[lane] + nz[4 * ROWS + lane]) * unit[4 + quad];
    } else if (lane < kHR) {
      nz[lane] = 0.f;
    }
    __syncwarp();
    // ---- weights: this thread's token against rows r0 .. r0 + kHR - 1, two rows an operation. x is rounded
    //      before the maximum is taken from it, so that the largest score's weight is exact however large it is ----
    const int tt = 32 * quad + lane;
    float2 x[kHR / 2];
    {
      const float un = stored ? unit[quad] : 1.f;
      uint32_t xr[kHR];
#pragma unroll
      for (int i = 0; i < kHR; i += 8) tmem_ld8(t_lane + r0 + i, xr + i);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < kHR; i += 4) {
        const float4 c4 = *reinterpret_cast<const float4*>(rowc + r0 + i), z4 = *reinterpret_cast<const float4*>(nz + i);
        const float2 u2 = make_float2(un, un);
        x[i / 2] = __fmul2_rn(__ffma2_rn(make_float2(__uint_as_float(xr[i]), __uint_as_float(xr[i + 1])), u2, make_float2(z4.x, z4.y)), make_float2(c4.x, c4.y));
        x[i / 2 + 1] = __fmul2_rn(__ffma2_rn(make_float2(__uint_as_float(xr[i + 2]), __uint_as_float(xr[i + 3])), u2, make_float2(z4.z, z4.w)), make_float2(c4.z, c4.w));
      }
    }
    if (t0 + kTile > len.n) {  // drafted tokens in the tile, or none at all behind the last one
      const int dj = t0 + tt - len.n;
      uint32_t sees = dj < 0 ? 0xFFFFFFFFu : 0u;  // rows that see this thread's token
      if (dj >= 0 && dj < len.nd) {
#pragma unroll 4
        for (int i = 0; i < kHR; ++i) sees |= (uint32_t)((mask[r0 + i] >> dj) & 1ull) << i;
      }
#pragma unroll
      for (int i = 0; i < kHR / 2; ++i) {
        if (!((sees >> (2 * i)) & 1u)) x[i].x = -INFINITY;
        if (!((sees >> (2 * i + 1)) & 1u)) x[i].y = -INFINITY;
      }
    }
    float most = -INFINITY;
#pragma unroll
    for (int i = 0; i < kHR; i += 4) {
      const float4 m4 = *reinterpret_cast<const float4*>(rowm + r0 + i);
      const float2 d0 = __fadd2_rn(x[i / 2], make_float2(m4.x, m4.y)), d1 = __fadd2_rn(x[i / 2 + 1], make_float2(m4.z, m4.w));
      most = fmaxf(most, fmaxf(d0.x, d0.y));
      most = fmaxf(most, fmaxf(d1.x, d1.y));
    }
    tmem_before();
    const bool raise = __syncthreads_or(most > kSlack + kRaise);
    if (tid == 224 && more) values_of(nw);  // every thread has read this tile's
    if (raise) {
      // ---- raise the running maxima of the rows with a score past them ----
      {
        float mine = 0.f;
#pragma unroll
        for (int i = 0; i < kHR; ++i) {
          const float v = warp_max((i & 1) ? x[i >> 1].y : x[i >> 1].x);
          if (lane == i) mine = v;
        }
        if (lane < kHR) red[quad * ROWS + r0 + lane] = mine;
      }
      __syncthreads();
      for (int r = tid; r < ROWS; r += kTreeThreads) {
        const float mt = fmaxf(fmaxf(red[r], red[ROWS + r]), fmaxf(red[2 * ROWS + r], red[3 * ROWS + r]));
        const bool up = mt + rowm[r] > kSlack + kRaise;
        rowf[r] = up ? exp2_approx((kRaise - mt) - rowm[r]) : 1.f;
        if (up) rowm[r] = kRaise - mt;
      }
      __syncthreads();
      if (!first) {  // the sums: the value product of the tile before is done (waited for above)
        tmem_after();
#pragma unroll
        for (int y = ROWS; y < 4 * ROWS; y += 2 * ROWS)  // O^T, and the constants' and weights'
#pragma unroll
          for (int i = 0; i < kHR; i += 8) {
            uint32_t u[8];
            float o[8];
            tmem_ld8(t_lane + y + r0 + i, u);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __uint_as_float(u[e]) * rowf[r0 + i + e];
            tmem_st8(t_lane + y + r0 + i, o);
          }
        tmem_wait_st();
      }
    }
#pragma unroll
    for (int i = 0; i < kHR; i += 8) {  // P^T over the key tile, which the score product has read
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 m4 = *reinterpret_cast<const float4*>(rowm + r0 + i + e);
        const int y = (i + e) / 2;
        float2 d0 = __fadd2_rn(x[y], make_float2(m4.x, m4.y)), d1 = __fadd2_rn(x[y + 1], make_float2(m4.z, m4.w));
        d0 = make_float2(exp2_approx(d0.x), exp2_approx(d0.y));
        d1 = make_float2(exp2_approx(d1.x), exp2_approx(d1.y));
        o[e / 2] = pack_h2(d0.x, d0.y);
        o[e / 2 + 1] = pack_h2(d1.x, d1.y);
      }
      *reinterpret_cast<uint4*>(sm + L::kOffK + ((r0 + i) >> 3) * 2048 + token_place(tt) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    fence_proxy_async_smem();
    tmem_before();
    __syncthreads();
    if (tid == 0) {
      tmem_after();
#pragma unroll
      for (int k = 0; k < 8; ++k) umma_f16(tmem + ROWS, desc_v + 16 * k, desc_p + 16 * k, tree_idesc(ROWS, true), !first || k > 0);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        umma_f16(tmem + 3 * ROWS, desc_w + k * (2 * kConst / 16), desc_p + 16 * k, tree_idesc(ROWS, true), !first || k > 0);
      tree_commit(bar_o);
    }
    first = false;

    // ---- the segment ends here (or the share does): hand its sums on ----
    if (last || p + 1 == p1) {
      const bool earlier = p - tile < p0;  // the segment began in an earlier block
      const bool whole = last && !earlier;
      if (earlier) sh.first = last ? kSegEnds : kSegGoesOn;
      else if (!last) {
        sh.open = b * seg_per_b + w.seg;
        sh.nd = len.nd;
      }
      float* slot = slots + ((size_t)blockIdx.x * 2 + (earlier ? 0 : 1)) * slot_floats<ROWS>();
      wait(bar_o, phase);
      tmem_after();
      // the sums of the constants of the warp's channel group and of the weights, lanes 0 .. 3, where the weights lay
      float* wc = reinterpret_cast<float*>(sm + L::kOffK) + 4 * ROWS * quad;
      {
        uint32_t u[kHR];
#pragma unroll
        for (int i = 0; i < kHR; i += 8) tmem_ld8(t_lane + 3 * ROWS + r0 + i, u + i);
        tmem_wait_ld();
        if (lane < 4) {
#pragma unroll
          for (int i = 0; i < kHR; i += 4)
            *reinterpret_cast<uint4*>(wc + ROWS * lane + r0 + i) = make_uint4(u[i], u[i + 1], u[i + 2], u[i + 3]);
        }
        __syncwarp();
        if (lane < kHR) {
          const int r = r0 + lane;
          wc[r] = wc[2 * ROWS + r] - (wc[r] + wc[ROWS + r]);
          if (quad == 0) red[r] = wc[3 * ROWS + r];
        }
      }
      __syncthreads();
      // each row's place in the output or the slot (-1: padding) and factor, once for all channels
      int* at_row = reinterpret_cast<int*>(rowc);
      if (tid < ROWS) {
        const int r = tid, row = row0 + r, di = div_by(row, a.rep);
        const float lt = red[r];
        const bool real = row < rows_all && di < len.nd;
        if (real && !whole) {
          slot[(size_t)ROWS * kD + r] = -rowm[r];
          slot[(size_t)ROWS * kD + ROWS + r] = lt;
        }
        at_row[r] = !real ? -1 : whole ? di * a.Hq + h * rep + row - di * rep : r;
        rowf[r] = !whole ? 2.f : (lt > 0.f || lt != lt) ? 2.f / lt : 0.f;  // values were halved
      }
      __syncthreads();
      const int ch = 32 * quad + lane;
      if (*nonfinite != 0) {  // of the drafted tokens in this block's tiles
        const int j0 = max(0, tile_first * kTile - len.n), j1 = min(len.nd, (tile + 1) * kTile - len.n);
#pragma unroll 1
        for (int r = r0; r < r0 + kHR; ++r) {
          if (at_row[r] < 0) continue;
          float o = tmem_ld1(t_lane + ROWS + r);
#pragma unroll 1
          for (int j = j0; j < j1; ++j) {
            if (!((mask[r] >> j) & 1ull)) continue;
            const uint16_t v = a.v_draft[(((size_t)b * a.N + j) * a.H + h) * kD + ch];
            if ((v & 0x7C00u) == 0x7C00u) o += th2f(v);
          }
          tmem_st1(t_lane + ROWS + r, o);
        }
        tmem_wait_st();
      }
      const bool f32 = !whole || a.out_fp32;
      const size_t out0 = (size_t)b * a.N * a.Hq * kD + ch;
      float* to32 = whole ? reinterpret_cast<float*>(a.out) + out0 : slot + ch;
      uint16_t* to16 = reinterpret_cast<uint16_t*>(a.out) + out0;
#pragma unroll 1
      for (int i = r0; i < r0 + kHR; i += 4) {
        uint32_t u[4];
        tmem_ld4(t_lane + ROWS + i, u);
        const float4 f4 = *reinterpret_cast<const float4*>(rowf + i), w4 = *reinterpret_cast<const float4*>(wc + i);
        const int4 at4 = *reinterpret_cast<const int4*>(at_row + i);
        const float f[4] = {f4.x, f4.y, f4.z, f4.w}, y[4] = {w4.x, w4.y, w4.z, w4.w};
        const int at[4] = {at4.x, at4.y, at4.z, at4.w};
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float o = f[e] == 0.f ? 0.f : (__uint_as_float(u[e]) + y[e]) * f[e];
          if (at[e] < 0) continue;
          if (f32) to32[(size_t)at[e] * kD] = o;
          else to16[(size_t)at[e] * kD] = f32_to_bf16(o);
        }
      }
      tmem_before();
      __syncthreads();  // the row state is read before the next segment resets it
      first = true;
    }
    phase ^= 1;
  }
  if (tid == 0) {
    shared[blockIdx.x] = sh;
    if (*failed) {  // a wait that ran out leaves the loop at the next barrier: let this block's copies and products end first
      mbar_wait_bounded(bar_k, phase, 10000000ull);
      mbar_wait_bounded(bar_v, phase, 10000000ull);
      mbar_wait_bounded(bar_o, phase ^ 1, 10000000ull);  // and its last value product, which the others came before
    }
  }
  tmem_before();
  __syncthreads();
  if (warp == 0) {
    tmem_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kCols) : "memory");
  }
}

// Joins the partials of a segment that several blocks shared, in block order. Block (k, rows): the segment that
// block k of the attention began and left open; a warp takes a row, a lane four channels.
constexpr int kMergeThreads = 128;
template <int ROWS>
__global__ void __launch_bounds__(kMergeThreads, ROWS <= 16 ? 6 : 9) kivi_tree_merge_kernel(const KiviTreeArgs a, const int G) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched ahead of the attention's end
  const int lane = threadIdx.x & 31, k = blockIdx.x, r = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5);
  const TreeShared* shared = reinterpret_cast<const TreeShared*>(a.part);
  const float* slots = reinterpret_cast<const float*>(shared + G);
  const int seg_all = shared[k].open;
  int f = k + 1 + lane < G ? shared[k + 1 + lane].first : kSegNoWork;
  if (seg_all < 0) return;
  const int rep = a.rep.d, rows_all = a.N * rep;
  const int b = div_by(seg_all, a.segs), seg = seg_all - b * a.segs.d, h = div_by(seg, a.row_tiles);
  const int row = (seg - h * a.row_tiles.d) * ROWS + r, di = div_by(row, a.rep);
  if (row >= rows_all || di >= shared[k].nd) return;
  const size_t mo = (size_t)ROWS * kD + r, lo = mo + ROWS;
  const float* own = slots + ((size_t)k * 2 + 1) * slot_floats<ROWS>();
  float M = own[mo], lt = own[lo];
  float4 o = *reinterpret_cast<const float4*>(own + (size_t)r * kD + 4 * lane);
  if (lt == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);  // the row saw nothing there
  // the blocks behind k that hold a part, 32 at a time: slot 0 of those, up to the one it ends in
  constexpr int kBatch = ROWS <= 16 ? 8 : 4;  // parts whose sums are on their way at once
  for (int base = k + 1;; base += 32) {
    const JoinParts join = join_parts(__ballot_sync(0xFFFFFFFFu, f == kSegGoesOn), __ballot_sync(0xFFFFFFFFu, f == kSegEnds));
    if (join.state == 2) return;  // a block's wait ran out (reported): the row is left as it was
    uint32_t parts = join.parts;
    const float* s = slots + (size_t)(base + lane) * 2 * slot_floats<ROWS>();
    const bool has = (parts >> lane) & 1u;
    float m = has ? s[mo] : -FLT_MAX, l = has ? s[lo] : 0.f;
    float4 v[kBatch];
    int at[kBatch];
    auto load = [&]() {
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        at[e] = parts ? __ffs(parts) - 1 : -1;
        parts &= parts - 1;
        v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (at[e] >= 0)
          v[e] = *reinterpret_cast<const float4*>(slots + (size_t)(base + at[e]) * 2 * slot_floats<ROWS>() + (size_t)r * kD + 4 * lane);
      }
    };
    load();
    float top = l == 0.f ? -FLT_MAX : m;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
    top = fmaxf(M, top);
    // a part that saw nothing stays out; one with a score that is not a number says so in the result
    auto weight = [&](float l, float m) { return l == 0.f ? 0.f : l != l ? 1.f : exp2_approx(m - top); };
    const float w0 = weight(lt, M), w = weight(l, m);
    M = top;
    l = w == 0.f ? 0.f : l * w;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, off);
    lt = (w0 == 0.f ? 0.f : lt * w0) + l;
    o = w0 == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * w0, o.y * w0, o.z * w0, o.w * w0);
    for (;;) {
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const float we = __shfl_sync(0xFFFFFFFFu, w, at[e] & 31);
        if (at[e] < 0 || we == 0.f) continue;
        o.x = fmaf(we, v[e].x, o.x);
        o.y = fmaf(we, v[e].y, o.y);
        o.z = fmaf(we, v[e].z, o.z);
        o.w = fmaf(we, v[e].w, o.w);
      }
      if (!parts) break;
      load();
    }
    if (join.state == 1) break;
    f = base + 32 + lane < G ? shared[base + 32 + lane].first : kSegNoWork;
  }
  const bool none = !(lt > 0.f || lt != lt);
  const size_t at = (((size_t)b * a.N + di) * a.Hq + (size_t)h * rep + row - di * rep) * kD + 4 * lane;
  float val[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) val[e] = none ? 0.f : val[e] / lt;
  if (a.out_fp32) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = make_float4(val[0], val[1], val[2], val[3]);
  } else {
    uint2 u;
    u.x = f32_to_bf16(val[0]) | ((uint32_t)f32_to_bf16(val[1]) << 16);
    u.y = f32_to_bf16(val[2]) | ((uint32_t)f32_to_bf16(val[3]) << 16);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at) = u;
  }
}

// Rows of a tile, which also choose the kernel: the warp-wide products for 8 or 16 rows, tcgen05 with 32 or 64. Of
// a tile's cost most is the same for any number of rows (the codes are unpacked once), so the smallest tile that holds
// all rows wins, and 64 above that. Measured with one kernel and the other (16 requests, 32 KV heads, 4K context, 2
// bits): 8 rows on the tile of 8 / 16 / 32: 102 / 159 / 221 us; 16 rows on 16 / 32: 164 / 223; 32 rows on 32 / 64:
// 228 / 274; 64 rows on 32 / 64: 448 / 288. A tile of 96 does not fit two blocks an SM: a thread's 48 scores would not
// stay in its registers.
int tree_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }
// resident blocks
int tree_blocks(int r) {
  return device_sms() * (r == 8 ? 4 : r == 16 ? MmaLayout<2, 2, 2>::kBlocks : 2);
}

template <int ROWS>
cudaError_t launch_merge(const KiviTreeArgs& a, int G, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(G, ROWS / (kMergeThreads / 32));
  cfg.blockDim = kMergeThreads;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kivi_tree_merge_kernel<ROWS>, a, G);
}
template <int ROWS, typename K>
cudaError_t launch_with(K kernel, int threads, int smem, const KiviTreeArgs& args, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int G = tree_blocks(ROWS), rep = args.Hq / args.H, row_tiles = (args.N * rep + ROWS - 1) / ROWS;
  KiviTreeArgs a = args;
  a.rep = int_div(rep);
  a.row_tiles = int_div(row_tiles);
  a.segs = int_div(a.H * row_tiles);
  a.blocks = int_div(G);
  a.ring = int_div(a.residual);
  kernel<<<G, threads, smem, st>>>(a, 1.4426950408889634f / sqrtf((float)kD));
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_merge<ROWS>(a, G, st);
}
template <int KB, int VB>
cudaError_t launch_tree_rows(const KiviTreeArgs& a, cudaStream_t st) {
  const int r = tree_rows(a.N * (a.Hq / a.H));
  if (r == 8) return launch_with<8>(kivi_tree_mma_kernel<KB, VB, 1>, kMmaThreads, MmaLayout<KB, VB, 1>::kSmem, a, st);
  if (r == 16) return launch_with<16>(kivi_tree_mma_kernel<KB, VB, 2>, kMmaThreads, MmaLayout<KB, VB, 2>::kSmem, a, st);
  if (r == 32) return launch_with<32>(kivi_tree_kernel<KB, VB, 32>, kTreeThreads, TreeLayout<KB, VB, 32>::kSmem, a, st);
  return launch_with<64>(kivi_tree_kernel<KB, VB, 64>, kTreeThreads, TreeLayout<KB, VB, 64>::kSmem, a, st);
}

}  // namespace

int device_sms() {
  static int cached[64] = {};
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return sms;
  if (cached[dev] == 0 && cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) cached[dev] = sms;
  return cached[dev] ? cached[dev] : sms;
}

size_t kivi_tree_ws_bytes(int B, int N, int H, int Hq, int k_bits, int v_bits) {
  const int r = tree_rows(N * (Hq / H));
  return (size_t)tree_blocks(r) * (sizeof(TreeShared) + 2 * r * (kD + 2) * sizeof(float));
}
long long kivi_tree_positions(int B, int N, int H, int Hq, int max_tokens, int residual) {
  const int rows = N * (Hq / H), r = tree_rows(rows);
  return (long long)B * H * ((rows + r - 1) / r) * (((long long)max_tokens + residual + N + kTile - 1) / kTile);
}

cudaError_t launch_kivi_tree(const KiviTreeArgs& a, cudaStream_t st) {
  if (a.k_bits == 2 && a.v_bits == 2) return launch_tree_rows<2, 2>(a, st);
  if (a.k_bits == 2) return launch_tree_rows<2, 4>(a, st);
  if (a.v_bits == 2) return launch_tree_rows<4, 2>(a, st);
  return launch_tree_rows<4, 4>(a, st);
}

}  // namespace kvq
