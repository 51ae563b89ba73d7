// Attention of a batch whose requests share a prefix that is cached once.
//
// Row r (request, drafted token, query head) attends the prefix's tokens and its request's own: with
// (o0, L0) the normalised output and the log2 of the sum of 2^score over the prefix, (o1, L1) over the
// request's cache and drafts,
//   o = (2^(L0 - M) o0 + 2^(L1 - M) o1) / (2^(L0 - M) + 2^(L1 - M)),  M = max(L0, L1).
// Over the prefix the rows of all requests are rows of one matrix per KV head; over its own tokens a
// request is a tree without the prefix (kivi_tree.cu), which writes fp32 outputs and L into the
// workspace; with one row a KV head and many requests it is the decode's (kivi.cu). Up to 32 rows a KV
// head the prefix, too, is one request of the tree kernels; more rows take the kernel below, which unpacks
// a tile of the prefix once for 256 of them.
#include <cfloat>

#include "kivi_tc.cuh"

namespace kvq {
namespace {

// ======================================================================================
// More than 32 rows: tcgen05 on tiles of 96 tokens and 2 x 128 rows
// ======================================================================================
//
//   S [128 rows x 112] = q [128 x 128] . K'^T      K' = 96 tokens s (c - c0) and rows of the groups' constants
//                                                  s (z - c0)
//   P = exp2(S c - m)                              a thread owns a row; P takes the columns of S
//   O [128 rows x 144] += P [128 x 96] . V'        V' = 128 channels s (c - c0), and columns of the tokens'
//                                                  constants s z, c0 s and of ones, whose sums are the weights'
// The constants enter as further tokens and channels of the same two products, so what a group lies off
// from zero is never rounded to fp16 (as in the tree kernels). 96 tokens: 2 (112 + 144) fp32 columns are
// the 512 of TMEM.
// s (c - c0) is exact in one fp16 at 2 bits. At 4 bits it takes two (kRest: a second product with what the rounding left),
// as in the tree kernels, so that a row's precision does not depend on how many others share the prefix. Rounded once it is
// off by 2^-11, which moves outputs by up to 6e-3 (queries as they come; by 4.6e-2 with eight times larger ones) against a
// bf16 rounding of 3e-2 at most. 512 rows over 32768 tokens: 142 us rounded, 159 in two parts; 256 rows over 8191 tokens 75
// and 81.
//
// Roles: warps 0 - 7 softmax (two row tiles, a thread a row); 8 - 15 unpack keys, four warps a 32-token group; 16 - 21
// unpack values, two warps a group; 22 issues the products; 23 copies what is stored of the groups ahead. Products and
// softmax of the two row tiles alternate: a tile's scores take the columns of its weights, so the score product waits for
// the value product. A row's maximum moves only when a score passes it by 2^kSlack, so rescaling O is rare and left to the
// softmax warps.
//
// Bound: the chain of a row tile (16 requests x 8 drafts x 4 heads, 32768 tokens, 4 and 2 bits, 126 us of the call's 158): 36
// tiles a block, 5700 cycles each with the begins and ends of segments (SMs are active 205 k cycles; the launch's 250 k under
// the profiler have its own begin and end): score product 500 cycles a part, softmax 1700 - 2300, value product 450, the
// barriers between them 900. Of the active cycles the tensor pipe has 44 %, issue 47 %, ALU 30 %, FMA 27 %. What it took (the
// same case, whole call with L2 flushed before it): the tree kernels, four row tiles of 64 that unpack the prefix each, 360 us;
// unpacking by four warps in unrolled code 220 (as many stalls on instruction fetch as issues); rolled loops by group 187;
// products issued by a warp that walks together 193 -> 182 with one part of the keys; two warps a group of values 179; loops of
// four code words 170; a room of 14 for kSlack's 10, with 1 for kRaise, 163; copies by a warp of their own 157; passes launched
// early 144; the join 140 (142 as measured since); kSlack and kRaise again 146, as 14 and 1 lose what lies below 2^-26 of a
// row's largest weight, 2^-30 elsewhere, and thousands of such tokens add up beside one large score; two parts of the keys 159.
// Tried and dropped: the softmax in pieces with the scores read twice (204 against 187), loads of codes two groups ahead into
// registers (192: their moves wait for them), spinning on barriers (266).
constexpr int kTok = 96, kGroups = kTok / kGroupT;
constexpr int kRows = 256;                       // of a segment: two row tiles
constexpr int kThreads = 768;
constexpr uint32_t kColS = 112, kColO = 144;     // TMEM columns of S and of O
constexpr int kVSbo = kTok * 16 + 16;            // V': from eight channels to the next (+ 16: other banks)
template <int KB, int VB>
struct PrefixLayout {
  static constexpr bool kRest = KB == 4;                   // the keys have second parts
  static constexpr int kVTiles = kRest ? 1 : 2;            // tiles of unpacked values
  // Groups whose stored keys are on their way; a warp's values. What is left of shared memory beside the second parts goes
  // to two stages of values first: 512 rows over 32768 tokens 159 us with (6, 2) to (8, 2), 196 with (9, 1), 200 with (5, 1).
  static constexpr int kKStages = kRest ? 6 : 9, kVStages = 2;
  // a group's stored keys or values: codes, scales, zero-points
  static constexpr int kKCode = kGroupT * kD * KB / 8, kVCode = kGroupT * kD * VB / 8, kPart = kD * 2;
  static constexpr int kKStage = kKCode + 2 * kPart, kVStage = kVCode + 2 * kPart;
  static constexpr int kK = (kTok + 16) * kD * 2, kKr = kRest ? kTok * kD * 2 : 0, kV = 18 * kVSbo;
  static constexpr int kOffQ = 0;                          // fp16 [2][128 x 128], K-major
  static constexpr int kOffK = kOffQ + 2 * 128 * kD * 2;   // [2] K' of a tile (112 rows), K-major
  static constexpr int kOffKr = kOffK + 2 * kK;            // [2] second parts of the keys
  static constexpr int kOffV = kOffKr + 2 * kKr;           // [kVTiles] V' of a tile, tokens within eight channels
  static constexpr int kOffKs = kOffV + kVTiles * kV;       // [kKStages] stored keys of a group
  static constexpr int kOffVs = kOffKs + kKStages * kKStage;
  static constexpr int kOffUnit = kOffVs + kGroups * kVStages * kVStage;  // float [4][8]: what a group's sums count, constants' from 4
  static constexpr int kOffBar = kOffUnit + 4 * 8 * 4;
  // A barrier of landed groups is waited on by the set of warps that unpacks the group. With an even number of stages a stage is
  // one set's. With an odd one the two sets take it by turns, and a warp that waits for group i must not meet the phase of group
  // i - kKStages, the other set's, unfinished: its tile of K' is free, so all groups of the tile before the last one are
  // unpacked, those up to i - 6 (kGroups = 3).
  static_assert(kKStages % 2 == 0 || kKStages >= 2 * kGroups, "phases that a set of warps does not see");
  static constexpr int kBars = 8 + 4 + 2 * kVTiles + 2 * kKStages + 2 * kGroups * kVStages;
  static constexpr int kSmem = kOffBar + kBars * 8 + 16;
  static_assert(kSmem <= 232448, "shared memory of a block");
};

// Registers: 80 a thread at launch, of which the softmax warps, with 96 scores each, take from the others.
constexpr int kRegsLaunch = 80, kRegsSoftmax = 128, kRegsOther = 56;
static_assert(256 * kRegsSoftmax + 512 * kRegsOther <= kThreads * kRegsLaunch, "registers of a block");
template <int N>
__device__ __forceinline__ void set_regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void set_regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// partial softmax of a segment: o [32 chunks of four channels][kRows][4], then m, l of each row
constexpr size_t kSlotFloats = (size_t)kRows * (kD + 2);

struct PrefixPlace {
  int P, T, p0, p1;  // positions of the launch, tiles of a segment, the block's share
};
__device__ __forceinline__ PrefixPlace prefix_place(const KiviTreeArgs& a, const TreeLens& len, int block) {
  PrefixPlace x;
  x.T = (int)((uint32_t)(len.n + kTok - 1) / kTok);
  x.P = x.T * a.segs.d;
  x.p0 = share_begin(x.P, block, a.blocks);
  x.p1 = share_begin(x.P, block + 1, a.blocks);
  return x;
}

// ---- keys of a 32-token group, by four warps: warp w takes channels 32 w .. + 31 of every token. A lane takes token
//      lane % 8 of an octet and a code word (2 bits: 16 channels, two octets; 4 bits: 8 channels, four octets). ----
// t: the group's first token; g: its place in the tile; stage: what is stored of it
template <int KB>
__device__ __forceinline__ void unpack_keys(const CodeScale& cs0, const KiviTreeArgs& a, const TreeLens& len, int h, int t, int g,
                                            int w, int lane, const unsigned char* stage, unsigned char* dst, unsigned char* rest,
                                            float* unit) {
  constexpr bool kRest = KB == 4;
  constexpr int kPairs = KB == 2 ? 8 : 4, kOct = KB == 2 ? 2 : 4, kRow = kD * KB / 8;
  const int word = KB == 2 ? 2 * w + ((lane >> 3) & 1) : 4 * w + (lane >> 3), oct = KB == 2 ? 2 * (lane >> 4) : 0;
  const int at0 = (4 * g + oct) * 2048 + word * (kPairs * 32) + (lane & 7) * 16;
  unsigned char* cdst = dst + kTok * kD * 2 + 2 * (lane >> 2) * 128 + ((lane & 3) >> 1) * 128 + 2 * g * 16 + (lane & 1) * 8;
  if (t < len.nqk) {
    const unsigned char* scale = stage + kGroupT * kRow;
    const uint2 four = *reinterpret_cast<const uint2*>(scale + 8 * lane);
    const __half2 most2 = __hmax2(__habs2(as_h2(four.x)), __habs2(as_h2(four.y)));
    const int e = 26 - (int)(__reduce_max_sync(0xFFFFFFFFu, max(as_u(most2) & 0xFFFFu, as_u(most2) >> 16)) >> 10);  // -5 .. 26
    if (w == g) {
      // constants: the lane's pairs j, j + 1 of 16 channels, j = 2 (lane % 4), in pair order
      const int j = lane & 3, ch = 16 * (lane >> 2) + (KB == 2 ? 2 * j : 8 * (j >> 1) + 2 * (j & 1));
      constexpr int kTo = KB == 2 ? 8 : 4;  // channels of a pair are kTo apart
      const unsigned char* zero = scale + kD * 2;
      float2 y[2];
      const float2 sa = __half22float2(as_h2(*reinterpret_cast<const uint32_t*>(scale + 2 * ch)));
      const float2 sb = __half22float2(as_h2(*reinterpret_cast<const uint32_t*>(scale + 2 * (ch + kTo))));
      const float2 za = __half22float2(as_h2(*reinterpret_cast<const uint32_t*>(zero + 2 * ch)));
      const float2 zb = __half22float2(as_h2(*reinterpret_cast<const uint32_t*>(zero + 2 * (ch + kTo))));
      constexpr float c0 = kCentre<KB>;
      y[0] = make_float2(sa.x * (za.x - c0), sb.x * (zb.x - c0));
      y[1] = make_float2(sa.y * (za.y - c0), sb.y * (zb.y - c0));
      const float most = fmaxf(fmaxf(fabsf(y[0].x), fabsf(y[0].y)), fmaxf(fabsf(y[1].x), fabsf(y[1].y)));
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
      *reinterpret_cast<uint2*>(cdst) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(cdst + 16) = make_uint2(lo[0], lo[1]);
      if (lane == 0) {
        unit[g] = __uint_as_float((uint32_t)(127 - e) << 23);
        unit[4 + g] = __uint_as_float((uint32_t)(127 - sh) << 23);
      }
    }
    // the scales times the power of two that puts the group's largest in [2^11, 2^12)
    const __half2 f0 = as_h2((uint32_t)(min(e, 15) + 15) * 0x4000400u), f1 = as_h2((uint32_t)(max(e, 15)) * 0x4000400u);
    __half2 s[kPairs];
    uint4 s0, s1;
    const uint4* sp = reinterpret_cast<const uint4*>(scale + 4 * kPairs * word);
    pair_order<KB>(sp[0], sp[KB == 2 ? 1 : 0], s0, s1);
    const uint32_t sw[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int j = 0; j < kPairs; ++j) s[j] = __hmul2(as_h2(sw[j]), f0);
    if (e > 15) {  // the rest of a power past the largest fp16 one
#pragma unroll
      for (int j = 0; j < kPairs; ++j) s[j] = __hmul2(s[j], f1);
    }
    const unsigned char* src = stage + (8 * oct + (lane & 7)) * kRow + 4 * word;
    uint32_t next = *reinterpret_cast<const uint32_t*>(src);
#pragma unroll 1  // short loops: the roles' unrolled code does not stay in the instruction cache
    for (int i = 0; i < kOct; ++i) {
      const uint32_t code = next;
      src += 8 * kRow;
      if (i + 1 < kOct) next = *reinterpret_cast<const uint32_t*>(src);
      uint32_t x[kPairs], y[kPairs];
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const __half2 c = code_h2<KB, kCentre<KB>>(cs0, code, j);
        x[j] = as_u(__hmul2(c, s[j]));
        if constexpr (kRest) y[j] = product_rest(as_u(c), as_u(s[j]), x[j]);
      }
      *reinterpret_cast<uint4*>(dst + at0 + 2048 * i) = make_uint4(x[0], x[1], x[2], x[3]);
      if constexpr (KB == 2) *reinterpret_cast<uint4*>(dst + at0 + 2048 * i + 128) = make_uint4(x[4], x[5], x[6], x[7]);
      if constexpr (kRest) *reinterpret_cast<uint4*>(rest + at0 + 2048 * i) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  } else {  // fp16 rows, or none
    if (w == g) {
      *reinterpret_cast<uint2*>(cdst) = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(cdst + 16) = make_uint2(0u, 0u);
      if (lane == 0) unit[g] = unit[4 + g] = 1.f;
    }
#pragma unroll 1
    for (int i = 0; i < kOct; ++i) {
      const uint16_t* row = fp16_key(a, len, 0, h, t + 8 * (oct + i) + (lane & 7));
      uint4 x0, x1;
      if constexpr (KB == 2) {
        pair_order<2>(row8(row, 2 * word), row8(row, 2 * word + 1), x0, x1);
        *reinterpret_cast<uint4*>(dst + at0 + 2048 * i + 128) = x1;
      } else {
        const uint4 v = row8(row, word);
        pair_order<4>(v, v, x0, x1);
        *reinterpret_cast<uint4*>(rest + at0 + 2048 * i) = make_uint4(0u, 0u, 0u, 0u);
      }
      *reinterpret_cast<uint4*>(dst + at0 + 2048 * i) = x0;
    }
  }
}

// ---- values of a 32-token group, by two warps: a lane a token, two value groups (32 channels each) a warp ----
// t: the group's first token; w0: the warp's first value group; dst: V' of the group
template <int VB>
__device__ __forceinline__ void unpack_values(const CodeScale& cs0, const KiviTreeArgs& a, const TreeLens& len, int h, int t, int w0,
                                              int lane, const unsigned char* stage, unsigned char* dst) {
  constexpr int kRow = kD * VB / 8;
  t += lane;
  dst += lane * 16;
  const bool stored = t < len.nqv;
  const unsigned char* codes = stage + lane * kRow;
  const uint16_t* scale = reinterpret_cast<const uint16_t*>(stage + kGroupT * kRow) + 4 * lane;
  const uint16_t* row = nullptr;
  if (!stored && t < len.n) row = fp16_value(a, len, 0, h, t, t - div_by(t, a.ring) * a.residual);
#pragma unroll 1
  for (int w = w0; w < w0 + 2; ++w) {
    // columns of the constants: s z, what its rounding left, c0 s (all halved as the values), 1
    uint2 c = make_uint2(0u, 0x3C000000u);
    if (stored) {
      const uint32_t z = scale[w + kGroupT * 4] * 0x10001u;
      const __half2 s2 = as_h2(halved(scale[w] * 0x10001u));
      const unsigned char* src = codes + 4 * VB * w;
      unsigned char* to = dst + 4 * w * kVSbo;
      auto eight = [&](int i) -> uint32_t {  // codes of channels 8 i .. + 7
        return VB == 2 ? (uint32_t)*reinterpret_cast<const uint16_t*>(src + 2 * i) : *reinterpret_cast<const uint32_t*>(src + 4 * i);
      };
      uint32_t next = eight(0);
#pragma unroll 1
      for (int i = 0; i < 4; ++i, to += kVSbo) {
        const uint32_t word = next;
        if (i < 3) next = eight(i + 1);
        *reinterpret_cast<uint4*>(to) = centred8<VB>(cs0, word, s2);
      }
      const uint32_t p = as_u(__hmul2(s2, as_h2(z))), left = product_rest(as_u(s2), z, p);
      c.x = (p & 0xFFFFu) | (left << 16);
      c.y |= as_u(__hmul2(s2, __float2half2_rn(kCentre<VB>))) & 0xFFFFu;
    } else {
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const uint4 v = row8(row, 4 * w + i);
        *reinterpret_cast<uint4*>(dst + (4 * w + i) * kVSbo) = make_uint4(halved(v.x), halved(v.y), halved(v.z), halved(v.w));
      }
    }
    *reinterpret_cast<uint2*>(dst + (16 + (w >> 1)) * kVSbo + (w & 1) * 8) = c;
  }
}

// What is stored of a group into a stage, by one thread; with nothing to copy the barrier completes at once.
template <int KB, int VB>
__device__ __forceinline__ void copy_keys(const KiviTreeArgs& a, const TreeLens& len, int h, int t, unsigned char* stage, uint64_t* full) {
  using L = PrefixLayout<KB, VB>;
  if (t >= len.nqk) {
    mbar_arrive(full);
    return;
  }
  const size_t tok = (size_t)h * a.max_tokens + t, g = tok / kGroupT * kD;
  mbar_arrive_expect_tx(full, L::kKStage);
  bulk_g2s(stage, a.k_codes + tok * (kD * KB / 8), L::kKCode, full);
  bulk_g2s(stage + L::kKCode, a.k_scale + g, L::kPart, full);
  bulk_g2s(stage + L::kKCode + L::kPart, a.k_zero + g, L::kPart, full);
}
template <int KB, int VB>
__device__ __forceinline__ void copy_values(const KiviTreeArgs& a, const TreeLens& len, int h, int t, unsigned char* stage, uint64_t* full) {
  using L = PrefixLayout<KB, VB>;
  if (t >= len.nqv) {
    mbar_arrive(full);
    return;
  }
  const size_t tok = (size_t)h * a.max_tokens + t;  // the rows behind n_quant_v are there, but not used
  mbar_arrive_expect_tx(full, L::kVStage);
  bulk_g2s(stage, a.v_codes + tok * (kD * VB / 8), L::kVCode, full);
  bulk_g2s(stage + L::kVCode, a.v_scale + tok * (kD / kGroupT), L::kPart, full);
  bulk_g2s(stage + L::kVCode + L::kPart, a.v_zero + tok * (kD / kGroupT), L::kPart, full);
}

// The groups of the block's share in order: group i of them, the g-th of tile p
struct Groups {
  int i, p, seg, tile, h, t, g;  // t: the group's first token
  __device__ __forceinline__ Groups(const KiviTreeArgs& a, const PrefixPlace& at, int seg_, int tile_)
      : i(0), p(at.p0), seg(seg_), tile(tile_), h(div_by(seg_, a.row_tiles)), t(tile_ * kTok), g(0) {}
  // d < kGroups groups on
  __device__ __forceinline__ void next(const KiviTreeArgs& a, const PrefixPlace& at, int d) {
    i += d;
    t += d * kGroupT;
    if ((g += d) < kGroups) return;
    g -= kGroups;
    ++p;
    if (++tile == at.T) {
      tile = 0;
      t = g * kGroupT;
      h = div_by(++seg, a.row_tiles);
    }
  }
};

template <int KB, int VB>
__global__ void __launch_bounds__(kThreads, 1) kivi_prefix_kernel(const KiviTreeArgs a, const float scale_log2) {
  using L = PrefixLayout<KB, VB>;
  constexpr int kVTiles = L::kVTiles, kKStages = L::kKStages, kVStages = L::kVStages;
  extern __shared__ __align__(128) unsigned char sm[];
  float* unit = reinterpret_cast<float*>(sm + L::kOffUnit);
  uint64_t* bar_q = reinterpret_cast<uint64_t*>(sm + L::kOffBar);  // [2] a row tile's queries are there
  uint64_t* bar_s = bar_q + 2;                                      // [2] its scores
  uint64_t* bar_p = bar_q + 4;                                      // [2] its weights
  uint64_t* bar_o = bar_q + 6;                                      // [2] its value product is done
  uint64_t* k_full = bar_q + 8;                                     // [2] a tile's keys are unpacked
  uint64_t* k_empty = bar_q + 10;                                   // [2] and read
  uint64_t* v_full = bar_q + 12;                                    // [kVTiles] a tile's values are unpacked
  uint64_t* v_empty = v_full + kVTiles;                             // [kVTiles] and read
  uint64_t* ks_full = v_empty + kVTiles;                            // [kKStages] a group's stored keys landed
  uint64_t* ks_empty = ks_full + kKStages;                          // [kKStages] and are unpacked
  uint64_t* vs_full = ks_empty + kKStages;                          // [kGroups][kVStages] a tile's group's stored values landed
  uint64_t* vs_empty = vs_full + kGroups * kVStages;                // and are unpacked
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_q + L::kBars);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const TreeLens len = tree_lens(a, 0, kTok);
  const PrefixPlace at = prefix_place(a, len, blockIdx.x);
  launch_dependents();
  if (at.p0 >= at.p1) return;
  const int rows_all = a.N * a.rep.d;
  if (warp == 16 + 2 * kGroups) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_q + i, 4);
      mbar_init(bar_s + i, 1);
      mbar_init(bar_p + i, 4);
      mbar_init(bar_o + i, 1);
      mbar_init(k_full + i, 4 * kGroups);
      mbar_init(k_empty + i, 1);
    }
    for (int i = 0; i < kVTiles; ++i) {
      mbar_init(v_full + i, 2 * kGroups);
      mbar_init(v_empty + i, 1);
    }
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(ks_full + i, 1);
      mbar_init(ks_empty + i, 4);
    }
    for (int i = 0; i < kGroups * kVStages; ++i) {
      mbar_init(vs_full + i, 1);
      mbar_init(vs_empty + i, 2);
    }
    fence_mbar_init();
  }
  tmem_before();
  __syncthreads();
  tmem_after();
  const uint32_t tmem = *tmem_slot;
  // a wait that runs out ends its role, and with it the waits of the others
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_wait_bounded_sleep(bar, parity & 1)) return true;
    set_error(a.err, KVQ_ERR_TIMEOUT);
    return false;
  };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity)) != 0; };
  // of a warp: one arrival
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  int seg = at.p0 / at.T, tile = at.p0 - seg * at.T;
  // row tiles of the segment: the second one may hold no row
  auto second = [&](int sg) { return rows_all - (sg - div_by(sg, a.row_tiles) * a.row_tiles.d) * kRows > 128; };

  if (warp < 8) {
    // ================= softmax: row tile r, a thread a row =================
    set_regs_up<kRegsSoftmax>();
    const int r = warp >> 2, row_t = tid & 127;
    const uint32_t t_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t t_s = t_lane + r * kColS, t_o = t_lane + 2 * kColS + r * kColO;
    uint32_t n = 0;                 // tiles done
    bool first = true;
    float rowc = 0.f, nm = FLT_MAX;  // log2 units per score unit; kRaise - running maximum
    for (int p = at.p0; p < at.p1; ++p) {
      const bool last = tile + 1 == at.T;
      if (r == 0 || second(seg)) {
        const int h = div_by(seg, a.row_tiles), rt = seg - h * a.row_tiles.d, row0 = rt * kRows + 128 * r;
        if (first) {
          // the tile's queries, every row on its way before the first is waited for: 8 lanes a row, four rows a warp at a time
          {
            const int row = row0 + row_t, di = div_by(row, a.rep);
            if (row < rows_all) {
              const uint16_t* src = a.q + ((size_t)di * a.Hq + (size_t)h * a.rep.d + row - di * a.rep.d) * kD;
              asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
              asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 64));
            }
          }
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const int rr = 32 * (warp & 3) + 4 * i + (lane >> 3), c = lane & 7;
            uint32_t u[8], o[8];
            load_query(a, len, 0, h, row0 + rr, c, u);
            const float back = query_fp16<14>(u, o, scale_log2);
            uint4 x0, x1;
            pair_order<KB>(make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]), x0, x1);
            unsigned char* dst = sm + L::kOffQ + r * (128 * kD * 2) + (rr >> 3) * 2048 + c * 256 + (rr & 7) * 16;
            *reinterpret_cast<uint4*>(dst) = x0;
            *reinterpret_cast<uint4*>(dst + 128) = x1;
            const float b = __shfl_sync(0xFFFFFFFFu, back, 8 * (lane & 3));
            if ((lane >> 2) == i) rowc = b;
          }
          nm = FLT_MAX;
          fence_proxy_async_smem();
          arrive(bar_q + r);
        }
        if (!wait_warp(bar_s + r, n)) break;
        tmem_after();
        // ---- scores, in units of 1 / rowc log2 ----
        float2 x[kTok / 2];
        {
          const float* un = unit + (p & 3) * 8;
          uint32_t cr[8];
          tmem_ld8(t_s + kTok, cr);
#pragma unroll
          for (int g = 0; g < kGroups; ++g) tmem_ld32(t_s + 32 * g, reinterpret_cast<uint32_t*>(x) + 32 * g);
          tmem_wait_ld();
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            const float z = -(__uint_as_float(cr[2 * g]) + __uint_as_float(cr[2 * g + 1])) * un[4 + g], f = un[g];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[16 * g + i] = __ffma2_rn(x[16 * g + i], make_float2(f, f), make_float2(z, z));
          }
        }
        if (last && len.n - tile * kTok < kTok) {  // none behind the last token
          const int there = len.n - tile * kTok;
#pragma unroll
          for (int i = 0; i < kTok / 2; ++i) {
            if (2 * i >= there) x[i].x = -INFINITY;
            if (2 * i + 1 >= there) x[i].y = -INFINITY;
          }
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kTok / 2; ++i) m4[i & 3] = fmaxf(m4[i & 3], fmaxf(x[i].x, x[i].y));
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * rowc;
        const bool up = mx + nm > kSlack + kRaise;
        if (__any_sync(0xFFFFFFFFu, up)) {
          const float f = up ? exp2_approx((kRaise - mx) - nm) : 1.f;
          if (up) nm = kRaise - mx;
          if (!first) {  // the sums, once the value product of the tile before is done
            if (!wait_warp(bar_o + r, n - 1)) break;
            tmem_after();
#pragma unroll 1
            for (int i = 0; i < (int)kColO; i += 16) {
              uint32_t u[16];
              tmem_ld8(t_o + i, u);
              tmem_ld8(t_o + i + 8, u + 8);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * f);
              tmem_st16(t_o + i, u);
            }
          }
        }
        // ---- weights, into the scores' columns. A weight is exp2(x rowc + nm) by one FMA: what the rounding of the maximum
        //      leaves in nm is common to the row. Scores so large that this is no longer small are rounded first, so that
        //      the largest one's weight is exact. ----
        float rc = rowc;
        if (__any_sync(0xFFFFFFFFu, !(fabsf(mx) < 1048576.f) || (nm != FLT_MAX && !(fabsf(nm) < 1048576.f)))) {
#pragma unroll
          for (int i = 0; i < kTok / 2; ++i) x[i] = __fmul2_rn(x[i], make_float2(rowc, rowc));
          rc = 1.f;
        }
#pragma unroll
        for (int c = 0; c < kTok / 32; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 d = __ffma2_rn(x[16 * c + i], make_float2(rc, rc), make_float2(nm, nm));
            w[i] = pack_h2(exp2_approx(d.x), exp2_approx(d.y));
          }
          tmem_st16(t_s + 16 * c, w);
        }
        tmem_wait_st();
        tmem_before();
        arrive(bar_p + r);
        first = false;
        if (last || p + 1 == at.p1) {
          // ---- the segment ends here (or the share does): hand its sums on ----
          if (!wait_warp(bar_o + r, n)) break;
          tmem_after();
          float* slot = a.part + (size_t)(blockIdx.x + seg) * kSlotFloats;
          const bool real = row0 + row_t < rows_all;
          float4* to = reinterpret_cast<float4*>(slot) + 128 * r + row_t;
          float wc[4], lt;
          {
            uint32_t u[16];
            tmem_ld8(t_o + kD, u);
            tmem_ld8(t_o + kD + 8, u + 8);
            tmem_wait_ld();
#pragma unroll
            for (int g = 0; g < 4; ++g)
              wc[g] = __uint_as_float(u[4 * g + 2]) - (__uint_as_float(u[4 * g]) + __uint_as_float(u[4 * g + 1]));
            lt = __uint_as_float(u[3]);
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint32_t u[32];
            tmem_ld32(t_o + 32 * g, u);
            tmem_wait_ld();
            if (real) {
#pragma unroll
              for (int i = 0; i < 8; ++i)  // values were halved
                to[(8 * g + i) * kRows] = make_float4(2.f * (__uint_as_float(u[4 * i]) + wc[g]), 2.f * (__uint_as_float(u[4 * i + 1]) + wc[g]),
                                                      2.f * (__uint_as_float(u[4 * i + 2]) + wc[g]), 2.f * (__uint_as_float(u[4 * i + 3]) + wc[g]));
            }
          }
          if (real) {
            slot[(size_t)kRows * kD + 128 * r + row_t] = -nm;
            slot[(size_t)kRows * (kD + 1) + 128 * r + row_t] = lt;
          }
          first = true;
        }
        ++n;
      }
      if (last) {
        tile = 0;
        ++seg;
        first = true;
      } else {
        ++tile;
      }
    }
  } else {
    set_regs_down<kRegsOther>();
    if (warp < 16) {
      // ================= keys: four warps a group, two such sets in turn =================
      const CodeScale cs0;
      const int set = (warp - 8) >> 2;
      Groups x(a, at, seg, tile);
      const int n = (at.p1 - at.p0) * kGroups;
      if (set) x.next(a, at, 1);
      int seen = 1;  // tiles whose stage was found empty (the first two are)
#pragma unroll 1
      while (x.i < n) {
        const int it = x.p - at.p0, st = it & 1, sg = x.i % kKStages;
        if (it > seen) {
          if (!wait_warp(k_empty + st, (it >> 1) + 1)) break;
          seen = it;
        }
        if (!wait_warp(ks_full + sg, x.i / kKStages)) break;
        unpack_keys<KB>(cs0, a, len, x.h, x.t, x.g, warp & 3, lane, sm + L::kOffKs + sg * L::kKStage,
                              sm + L::kOffK + st * L::kK, sm + L::kOffKr + st * L::kKr, unit + (x.p & 3) * 8);
        fence_proxy_async_smem();
        arrive(ks_empty + sg);
        if (lane == 0) mbar_arrive(k_full + st);
        x.next(a, at, 2);
      }
    } else if (warp < 16 + 2 * kGroups) {
      // ================= values: two warps every third group =================
      const CodeScale cs0;
      const int g = (warp - 16) >> 1, n = at.p1 - at.p0;
      int h = div_by(seg, a.row_tiles), t = tile * kTok;         // the tile's
      const unsigned char* stages = sm + L::kOffVs + g * kVStages * L::kVStage;
      uint64_t *landed = vs_full + g * kVStages, *taken = vs_empty + g * kVStages;
#pragma unroll 1
      for (int it = 0; it < n; ++it) {
        const int sg = it % kVStages;
        const int sv = it % kVTiles;
        if (it >= kVTiles && !wait_warp(v_empty + sv, it / kVTiles + 1)) break;
        if (!wait_warp(landed + sg, it / kVStages)) break;
        unpack_values<VB>(cs0, a, len, h, t + g * kGroupT, 2 * (warp & 1), lane, stages + sg * L::kVStage,
                          sm + L::kOffV + sv * L::kV + g * kGroupT * 16);
        fence_proxy_async_smem();
        arrive(taken + sg);
        if (lane == 0) mbar_arrive(v_full + sv);
        t += kTok;
        if (++tile == at.T) {
          tile = t = 0;
          h = div_by(++seg, a.row_tiles);
        }
      }
    } else if (warp == 17 + 2 * kGroups) {
      // ================= copies: the stored keys and values of each group in turn, as stages become free =================
      Groups x(a, at, seg, tile);
      const int n = (at.p1 - at.p0) * kGroups;
      int copied = 0;
#pragma unroll 1
      for (; x.i < n; x.next(a, at, 1)) {
        const int it = x.p - at.p0, sg = x.i % kKStages, sv = x.g * kVStages + it % kVStages;
        if (x.i >= kKStages && !wait_warp(ks_empty + sg, x.i / kKStages + 1)) break;
        if (lane == 0) copy_keys<KB, VB>(a, len, x.h, x.t, sm + L::kOffKs + sg * L::kKStage, ks_full + sg);
        copied = x.i + 1;  // of its values at most
        if (it >= kVStages && !wait_warp(vs_empty + sv, it / kVStages + 1)) break;
        if (lane == 0) copy_values<KB, VB>(a, len, x.h, x.t, sm + L::kOffVs + sv * L::kVStage, vs_full + sv);
      }
      // nothing is in flight when the block ends, also where a wait ran out: the last copy into every stage
      for (int i = max(0, copied - kKStages); i < copied; ++i) mbar_wait_bounded(ks_full + i % kKStages, (i / kKStages) & 1, 10000000ull);
      for (int i = max(0, copied - kGroups * kVStages); i < copied; ++i)
        mbar_wait_bounded(vs_full + i % kGroups * kVStages + i / kGroups % kVStages, (i / kGroups / kVStages) & 1, 10000000ull);
    } else if (warp == 16 + 2 * kGroups) {
      // ================= products: the warp walks together, one lane issues =================
      const uint32_t leader = elect_one();
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const uint32_t q0 = desc_lo(sm + L::kOffQ, 128), k0 = desc_lo(sm + L::kOffK, 128), kr0 = desc_lo(sm + L::kOffKr, 128);
      const uint32_t v0 = desc_lo(sm + L::kOffV, 128);
      constexpr uint32_t kHi = desc_hi(2048), kHiV = desc_hi(kVSbo);
      uint32_t n[2] = {0, 0}, parts[2] = {0, 0};  // tiles, and parts of segments, of each row tile
      // the scores of row tile r for the tile in stage st; starts: the part's first
      auto scores = [&](int r, int st, bool starts) {
        if (starts && !wait_warp(bar_q + r, parts[r]++)) return false;
        tmem_after();
        const uint32_t q = q0 + r * (128 * kD * 2 / 16), k = k0 + st * (L::kK / 16), d = tm + r * kColS;
#pragma unroll
        for (int i = 0; i < 8; ++i) umma_lo<kHi, kHi, tree_idesc(kColS, false)>(leader, d, q + 16 * i, k + 16 * i, i > 0);
        if constexpr (L::kRest) {
          const uint32_t kk = kr0 + st * (L::kKr / 16);
#pragma unroll
          for (int i = 0; i < 8; ++i) umma_lo<kHi, kHi, tree_idesc(kTok, false)>(leader, d, q + 16 * i, kk + 16 * i, 1);
        }
        commit_if(leader, bar_s + r);
        return true;
      };
      bool ok = true, starts = true;
      int last_r = second(seg) ? 1 : 0;
      ok = wait_warp(k_full, 0);
      for (int r = 0; ok && r <= last_r; ++r) ok = scores(r, 0, true);
      if (ok) commit_if(leader, k_empty);
#pragma unroll 1
      for (int p = at.p0; ok && p < at.p1; ++p) {
        const int it = p - at.p0, st = it & 1;
        const bool ends = tile + 1 == at.T, more = p + 1 < at.p1;
        const int nseg = ends ? seg + 1 : seg, next_r = !more ? -1 : ends ? (second(nseg) ? 1 : 0) : last_r;
        const int sv = it % kVTiles;
        ok = wait_warp(v_full + sv, it / kVTiles);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (ok && r <= last_r) {
            if (!(ok = wait_warp(bar_p + r, n[r]))) break;
            tmem_after();
#pragma unroll
            for (int i = 0; i < 2 * kGroups; ++i)
              umma_lo_ta<kHiV, tree_idesc(kColO, true)>(leader, tm + 2 * kColS + r * kColO, tm + r * kColS + 8 * i,
                                                        v0 + sv * (L::kV / 16) + 16 * i, i > 0 || !starts);
            commit_if(leader, bar_o + r);
            if (r == last_r) commit_if(leader, v_empty + sv);
            // the scores of the next tile take the columns that this product reads
            if (r <= next_r && !(ok = wait_warp(bar_o + r, n[r]))) break;
            ++n[r];
          }
          if (ok && r <= next_r) {
            if (r == 0 && !(ok = wait_warp(k_full + (st ^ 1), (it + 1) >> 1))) break;
            if (!(ok = scores(r, st ^ 1, ends))) break;
            if (r == next_r) commit_if(leader, k_empty + (st ^ 1));
          }
        }
        starts = ends;
        last_r = next_r;
        seg = nseg;
        tile = ends ? 0 : tile + 1;
      }
      const int done = at.p1 - at.p0 - 1;  // the last arrival there is
      if (ok) wait_warp(v_empty + done % kVTiles, done / kVTiles);
      if (!ok && leader) {  // let what was issued end before the memory goes
        mbar_wait_bounded(bar_s, n[0] & 1, 10000000ull);
        mbar_wait_bounded(bar_s + 1, n[1] & 1, 10000000ull);
        mbar_wait_bounded(bar_o, n[0] & 1, 10000000ull);
        mbar_wait_bounded(bar_o + 1, n[1] & 1, 10000000ull);
      }
    }
  }
  __syncwarp();
  tmem_before();
  __syncthreads();
  if (warp == 16 + 2 * kGroups) {
    tmem_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// ======================================================================================
// Joining the two sides
// ======================================================================================

// One side of a row: its four channels o, L the log2 of its sum of 2^score
struct Side {
  float l;
  float4 o;
};
__device__ __forceinline__ Side side(const KiviTreeArgs& t, size_t row, size_t at) {
  return {t.lse[row], *reinterpret_cast<const float4*>(static_cast<const float*>(t.out) + at)};
}
// The drafted token of a request with one row (`apart`): its value, and the score q k / sqrt(D) of the four channels at c
// (log2 units). -infinity: the row does not see it.
__device__ __forceinline__ bool sees_draft(const KiviPrefixArgs& a, int b) { return a.apart && a.own.mask && (a.own.mask[b] & 1ull); }
__device__ __forceinline__ Side draft(const KiviPrefixArgs& a, size_t row, int b, int h, int c) {
  const size_t at = ((size_t)b * a.own.H + h) * kD + 4 * c;
  const uint2 q = *reinterpret_cast<const uint2*>(a.own.q + row * kD + 4 * c);
  const uint2 k = *reinterpret_cast<const uint2*>(a.own.k_draft + at), v = *reinterpret_cast<const uint2*>(a.own.v_draft + at);
  const float2 k0 = __half22float2(as_h2(k.x)), k1 = __half22float2(as_h2(k.y)), v0 = __half22float2(as_h2(v.x)), v1 = __half22float2(as_h2(v.y));
  const float s = fmaf(bf16_hi(q.y), k1.y, fmaf(bf16_lo(q.y), k1.x, fmaf(bf16_hi(q.x), k0.y, bf16_lo(q.x) * k0.x)));
  return {s * (1.4426950408889634f * 0.08838834764831845f), make_float4(v0.x, v0.y, v1.x, v1.y)};
}
__device__ __forceinline__ void combine_row(const KiviPrefixArgs& a, size_t at, const Side& x, const Side& y, const Side& z) {
  // a side that saw nothing stays out, whatever its row holds; one that is not a number says so in the result
  const float top = fmaxf(fmaxf(fmaxf(x.l, y.l), z.l), -FLT_MAX);
  auto weight = [&](float l) { return l != l ? l : exp2f(l - top); };
  float w0 = weight(x.l), w1 = weight(y.l), w2 = weight(z.l);
  const float sum = w0 + w1 + w2, inv = sum == 0.f ? 0.f : 1.f / sum;
  w0 *= inv;
  w1 *= inv;
  w2 *= inv;
  auto mix = [&](float p, float q, float r) { return (w0 == 0.f ? 0.f : w0 * p) + (w1 == 0.f ? 0.f : w1 * q) + (w2 == 0.f ? 0.f : w2 * r); };
  const float v[4] = {mix(x.o.x, y.o.x, z.o.x), mix(x.o.y, y.o.y, z.o.y), mix(x.o.z, y.o.z, z.o.z), mix(x.o.w, y.o.w, z.o.w)};
  if (a.out_fp32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
        make_uint2(f32_to_bf16(v[0]) | ((uint32_t)f32_to_bf16(v[1]) << 16), f32_to_bf16(v[2]) | ((uint32_t)f32_to_bf16(v[3]) << 16));
}

// A warp a row, a lane four channels.
constexpr int kCombineThreads = 128;
__global__ void __launch_bounds__(kCombineThreads) kivi_prefix_combine_kernel(const KiviPrefixArgs a, const int rows) {
  wait_behind();
  const int row = blockIdx.x * (kCombineThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= rows) return;
  const int tok = div_by(row, a.heads), b = div_by(tok, a.tokens);
  if (a.own.n_draft && tok - b * a.own.N >= a.own.n_draft[b]) return;  // padding
  const size_t at = (size_t)row * kD + 4 * lane;
  Side z = {-INFINITY, make_float4(0.f, 0.f, 0.f, 0.f)};
  if (sees_draft(a, b)) {
    z = draft(a, row, b, div_by(row - tok * a.own.Hq, a.prefix.rep), lane);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) z.l += __shfl_xor_sync(0xFFFFFFFFu, z.l, off);
  }
  combine_row(a, at, side(a.prefix, row, at), side(a.own, row, at), z);
}

// The same behind the kernel above: the parts of a segment lie in the slots block + segment of the blocks that shared
// it. A block takes eight rows of a KV head, a thread four channels of one of them.
constexpr int kJoinThreads = 256, kJoinRows = 8;
__global__ void __launch_bounds__(kJoinThreads) kivi_prefix_join_kernel(const KiviPrefixArgs a) {
  const KiviTreeArgs& t = a.prefix;
  const int lane = threadIdx.x & 31, c = 4 * (threadIdx.x >> 5) + (lane >> 3), h = blockIdx.y;
  const int row = min(blockIdx.x * kJoinRows + (lane & 7), t.N * t.rep.d - 1);  // of the KV head; of the last block the last ones again
  const int tok = div_by(row, t.rep), b = div_by(tok, a.tokens);
  const bool real = !a.own.n_draft || tok - b * a.own.N < a.own.n_draft[b];  // no padding
  const size_t out_row = (size_t)tok * t.Hq + h * t.rep.d + row - tok * t.rep.d;
  Side z = {-INFINITY, make_float4(0.f, 0.f, 0.f, 0.f)};
  if (a.apart) {  // each warp has four of a row's 32 pieces
    __shared__ float score[kJoinThreads / 32][kJoinRows];
    const bool sees = real && sees_draft(a, b);
    float s = 0.f;
    if (sees) {
      z = draft(a, out_row, b, h, c);
      s = z.l;
    }
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
    if (lane < kJoinRows) score[threadIdx.x >> 5][lane] = s;
    __syncthreads();
    if (sees) {
      z.l = 0.f;
#pragma unroll
      for (int w = 0; w < kJoinThreads / 32; ++w) z.l += score[w][lane & 7];
    }
  }
  const TreeLens len = tree_lens(t, 0, kTok);
  const int T = (int)((uint32_t)(len.n + kTok - 1) / kTok), P = T * t.segs.d;
  const int seg = h * t.row_tiles.d + row / kRows, r = row & (kRows - 1);
  int k = 0, last = -1;
  if (T > 0) {  // the blocks that hold positions of the segment
    const int begin = seg * T, end = begin + T;
    k = P <= t.blocks.d ? begin : (int)((long long)begin * t.blocks.d / P);
    while (k > 0 && share_begin(P, k, t.blocks) > begin) --k;
    while (share_begin(P, k + 1, t.blocks) <= begin) ++k;
    last = P <= t.blocks.d ? end - 1 : (int)((long long)(end - 1) * t.blocks.d / P);
    while (last > 0 && share_begin(P, last, t.blocks) >= end) --last;
    while (last + 1 < t.blocks.d && share_begin(P, last + 1, t.blocks) < end) ++last;
  }
  wait_behind();  // what was read so far is the caller's
  if (!real) return;
  const size_t at = out_row * kD + 4 * c;
  const Side own = side(a.own, out_row, at);
  float top = -FLT_MAX, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kBatch = 10;  // parts on their way at once (256 rows, 8191 tokens, 20 parts a row: 8 of them 76.8 us a call, 10 and 12 74.7)
  for (; k <= last; k += kBatch) {
    float m[kBatch], lp[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const float* slot = t.part + (size_t)(min(k + e, last) + seg) * kSlotFloats;
      m[e] = slot[(size_t)kRows * kD + r];
      lp[e] = k + e <= last ? slot[(size_t)kRows * (kD + 1) + r] : 0.f;
      v[e] = reinterpret_cast<const float4*>(slot)[c * kRows + r];
    }
    float up = top;
#pragma unroll
    for (int e = 0; e < kBatch; ++e) up = lp[e] == 0.f ? up : fmaxf(up, m[e]);  // 0: the row saw nothing there
    const float f = l == 0.f ? 0.f : exp2_approx(top - up);
    top = up;
    l = f == 0.f ? 0.f : l * f;
    o = f == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const float w = lp[e] == 0.f ? 0.f : lp[e] != lp[e] ? 1.f : exp2_approx(m[e] - up);
      if (w == 0.f) continue;
      l = fmaf(lp[e], w, l);
      o = make_float4(fmaf(v[e].x, w, o.x), fmaf(v[e].y, w, o.y), fmaf(v[e].z, w, o.z), fmaf(v[e].w, w, o.w));
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  combine_row(a, at, {l == 0.f ? -INFINITY : top + __log2f(l), make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv)}, own, z);
}

template <int KB, int VB>
cudaError_t launch_prefix_rows(const KiviTreeArgs& a, cudaStream_t st) {
  auto kernel = kivi_prefix_kernel<KB, VB>;
  constexpr int kSmem = PrefixLayout<KB, VB>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<a.blocks.d, kThreads, kSmem, st>>>(a, 1.4426950408889634f / sqrtf((float)kD));
  return cudaGetLastError();
}
cudaError_t launch_prefix_bits(const KiviTreeArgs& a, cudaStream_t st) {
  if (a.k_bits == 2) return a.v_bits == 2 ? launch_prefix_rows<2, 2>(a, st) : launch_prefix_rows<2, 4>(a, st);
  return a.v_bits == 2 ? launch_prefix_rows<4, 2>(a, st) : launch_prefix_rows<4, 4>(a, st);
}

// Rows of a KV head from which on the kernel above takes the prefix. Measured with it and with the tree kernels (whole call, 4
// bits): 8 KV heads, 36 rows over 1024, 4096 and 8192 tokens 26 / 28 us, 36 / 33, 40 / 43; 64 rows 24 / 29, 36 / 40, 40 / 44; 128
// rows 26 / 31, 38 / 42, 41 / 51; 32 KV heads, 33 rows 45 / 44, 58 / 58, 79 / 75; 64 rows 58 / 60, 74 / 75, 93 / 93; 128 rows
// 95 / 95, 112 / 122, 130 / 159. 2 bits alike. Up to 32 rows the tree kernels have a tile for all of them: 32 rows over 8192
// tokens, 8 KV heads, 40 / 39.
bool many_rows(int rows) { return rows > 32; }
// Requests with one row a KV head attend their own caches as the decode does, unsplit, if that makes two blocks an SM (a
// drafted token is joined apart): it spends a third of the tree kernel's instructions on one row. Measured with it and
// without (whole call, 32 KV heads, 2 bits): 16 requests of 512 tokens 54 / 60 us, 64 requests of 40 tokens 66 / 79, 128
// 95 / 114. Four query heads a KV head, 64 requests of 640 tokens, 4 bits: 89 / 75, so not there.
// One block walks a (request, head) to its end, so a long request holds up a call of short ones, which the tree kernels split.
// The host knows the caches' capacity alone: up to 2048 tokens of it (16 requests, 32 heads over 1024 tokens: all of 2048 75 /
// 85, one of 2048 among 64s 48 / 46; beyond, all of 4096 112 / 122 and of 8192 187 / 198, but one of 4096 69 / 54, of 16384
// 183 / 98; 64 requests, 8 heads, one of 16384: 138 / 54).
constexpr int kAloneTokens = 2048;
bool alone(const KiviTreeArgs& a, int rep) {
  return a.N == 1 && rep == 1 && a.max_tokens <= kAloneTokens && (long long)a.B * a.H >= 2ll * device_sms();
}
int row_tiles(int rows) { return (rows + kRows - 1) / kRows; }

}  // namespace

size_t kivi_prefix_ws_bytes(int rows_n, int H, int Hq, int k_bits, int v_bits) {
  const int rows = rows_n * (Hq / H);
  if (!many_rows(rows)) return kivi_tree_ws_bytes(1, rows_n, H, Hq, k_bits, v_bits);
  return ((size_t)device_sms() + (size_t)H * row_tiles(rows)) * kSlotFloats * sizeof(float);
}
long long kivi_prefix_positions(int rows_n, int H, int Hq, int max_tokens, int residual) {
  const int rows = rows_n * (Hq / H);
  if (!many_rows(rows)) return kivi_tree_positions(1, rows_n, H, Hq, max_tokens, residual);
  return (long long)H * row_tiles(rows) * (((long long)max_tokens + residual + kTok - 1) / kTok);
}

cudaError_t launch_kivi_prefix(const KiviPrefixArgs& args, cudaStream_t st) {
  cudaError_t e;
  KiviPrefixArgs a = args;
  a.heads = int_div(a.own.Hq);
  a.tokens = int_div(a.own.N);
  KiviTreeArgs& t = a.prefix;
  const int rep = t.Hq / t.H, rows = t.N * rep;
  const bool many = many_rows(rows);
  if (many) {
    t.rep = int_div(rep);
    t.row_tiles = int_div(row_tiles(rows));
    t.segs = int_div(t.H * t.row_tiles.d);
    t.blocks = int_div(device_sms());
    t.ring = int_div(t.residual);
    e = launch_prefix_bits(t, st);
  } else {
    t.chained = kChainedFirst;
    e = launch_kivi_tree(t, st, kTreeAttend);
  }
  // every further launch is early: the blocks of both passes share the GPU, and what joins them is there when they end
  KiviTreeArgs& o = a.own;
  a.apart = alone(o, rep);
  o.chained = kChainedBehind;
  t.rep = int_div(rep);
  if (e == cudaSuccess && a.apart) {
    KiviAttnArgs d{};
    d.k_codes = o.k_codes; d.k_scale = o.k_scale; d.k_zero = o.k_zero;
    d.v_codes = o.v_codes; d.v_scale = o.v_scale; d.v_zero = o.v_zero;
    d.k_resid = o.k_resid; d.v_resid = o.v_resid;
    d.n_tok = o.n_tok; d.n_quant_k = o.n_quant_k; d.n_quant_v = o.n_quant_v;
    d.q = o.q; d.out = o.out; d.out_fp32 = 1; d.lse = o.lse; d.err = o.err;
    d.B = o.B; d.H = o.H; d.Hq = o.Hq; d.k_bits = o.k_bits; d.v_bits = o.v_bits;
    d.max_tokens = o.max_tokens; d.residual = o.residual; d.group = kGroupT;
    d.n_split = 1;
    d.tok_per_split = max(o.max_tokens, kGroupT);
    e = launch_kivi_attn(d, st);
  } else if (e == cudaSuccess) {
    e = launch_kivi_tree(o, st, kTreeAttend);
  }
  if (e == cudaSuccess && !many) e = launch_kivi_tree(t, st, kTreeMerge);
  if (e == cudaSuccess && !a.apart) e = launch_kivi_tree(o, st, kTreeMerge);
  if (e != cudaSuccess) return e;
  if (many) return launch_early(true, kivi_prefix_join_kernel, dim3((rows + kJoinRows - 1) / kJoinRows, t.H), kJoinThreads, 0, st, a);
  const int all = a.own.B * a.own.N * a.own.Hq, per = kCombineThreads / 32;
  return launch_early(true, kivi_prefix_combine_kernel, dim3((all + per - 1) / per), kCombineThreads, 0, st, a, all);
}

}  // namespace kvq
