// Attention of a batch whose requests share a prefix that is cached once.
//
// Row r (request, drafted token, query head) attends the prefix's tokens and its request's own: with
// (o0, L0) the normalised output and the log2 of the sum of 2^score over the prefix, (o1, L1) over the
// request's cache and drafts,
//   o = (2^(L0 - M) o0 + 2^(L1 - M) o1) / (2^(L0 - M) + 2^(L1 - M)),  M = max(L0, L1).
// Over the prefix the rows of all requests are rows of one matrix per KV head; over its own tokens a
// request is a tree without the prefix (kivi_tree.cu), which writes fp32 outputs and L into the
// workspace. Up to 64 rows a KV head the prefix, too, is one request of the tree kernels; more rows take
// the kernel below, which unpacks a tile of the prefix once for 256 of them.
#include <cfloat>

#include "kivi_tc.cuh"

namespace kvq {
namespace {

// ======================================================================================
// More than 64 rows: tcgen05 on tiles of 96 tokens and 2 x 128 rows
// ======================================================================================
//
//   S [128 rows x 112] = q [128 x 128] . K'^T      K' = 96 tokens s (c - c0), exact in one fp16 at 2 bits and in
//                                                  two at 4, and rows of the groups' constants s (z - c0)
//   P = exp2(S c - m)                              a thread owns a row; P takes the columns of S
//   O [128 rows x 144] += P [128 x 96] . V'        V' = 128 channels s (c - c0), and columns of the tokens'
//                                                  constants s z, c0 s and of ones, whose sums are the weights'
// The constants enter as further tokens and channels of the same two products, so what a group lies off
// from zero is never rounded to fp16 (as in the tree kernels). 96 tokens: 2 (112 + 144) fp32 columns are
// the 512 of TMEM.
// Roles: warps 0 - 7 softmax (two row tiles, a thread a row), 8 - 11 unpack keys and 12 - 14 values into
// two stages of shared memory, warp 15 issues the products. A row's maximum moves only when a score passes it by
// 2^kSlack, so rescaling O is rare and left to the softmax warps.
constexpr int kTok = 96, kGroups = kTok / kGroupT;
constexpr int kRows = 256;                       // of a segment: two row tiles
constexpr int kThreads = 512;
constexpr uint32_t kColS = 112, kColO = 144;     // TMEM columns of S and of O
constexpr int kVSbo = kTok * 16 + 16;            // V': from eight channels to the next (+ 16: other banks)

template <int KB>
struct PrefixLayout {
  static constexpr int kK = (kTok + 16) * kD * 2, kKr = KB == 4 ? kTok * kD * 2 : 0, kV = (18 * kVSbo + 127) / 128 * 128;
  static constexpr int kOffQ = 0;                          // fp16 [2][128 x 128], K-major
  static constexpr int kOffK = kOffQ + 2 * 128 * kD * 2;   // [2 stages] K' (112 rows), K-major
  static constexpr int kOffKr = kOffK + 2 * kK;            // [2 stages] second parts of the keys (4 bits)
  static constexpr int kOffV = kOffKr + 2 * kKr;           // [2 stages] V', tokens within eight channels
  static constexpr int kOffUnit = kOffV + 2 * kV;          // float [4][8]: what a group's sums count, constants' from 4
  static constexpr int kOffBar = kOffUnit + 4 * 8 * 4;
  static constexpr int kSmem = kOffBar + 160;
  static_assert(kSmem <= 232448, "shared memory of a block");
};

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
template <int KB>
struct KeyRegs {
  static constexpr int kOct = KB == 2 ? 2 : 4;
  uint32_t code[kOct];
  uint4 scale[KB == 2 ? 2 : 1];           // of the lane's word
  uint2 four;                             // of channels 4 lane .., for the group's largest
  uint32_t cs[2], cz[2];                  // scales and zeros of the constants the lane makes (one warp of the four)
};
template <int KB>
struct KeyLane {
  int w, lane, word, oct;
  __device__ __forceinline__ KeyLane(int w_, int lane_) : w(w_), lane(lane_) {
    word = KB == 2 ? 2 * w + ((lane >> 3) & 1) : 4 * w + (lane >> 3);
    oct = KB == 2 ? 2 * (lane >> 4) : 0;
  }
  // constants: the lane's pairs j, j + 1 of 16 channels, j = 2 (lane % 4), in pair order: channels ch, ch + 1, and kTo on
  static constexpr int kTo = KB == 2 ? 8 : 4;
  __device__ __forceinline__ int ch() const {
    const int j = lane & 3;
    return 16 * (lane >> 2) + (KB == 2 ? 2 * j : 8 * (j >> 1) + 2 * (j & 1));
  }
};
// t: the group's first token; g: its place in the tile
template <int KB>
__device__ __forceinline__ void load_keys(const KiviTreeArgs& a, const TreeLens& len, int h, int t, int g, const KeyLane<KB>& l,
                                          KeyRegs<KB>& r) {
  if (t >= len.nqk) return;
  constexpr int kRow = kD * KB / 8;
  const size_t tok = (size_t)h * a.max_tokens + t, grp = tok / kGroupT * kD;
  const uint8_t* codes = a.k_codes + (tok + 8 * l.oct + (l.lane & 7)) * kRow + 4 * l.word;
#pragma unroll
  for (int i = 0; i < KeyRegs<KB>::kOct; ++i) r.code[i] = __ldg(reinterpret_cast<const uint32_t*>(codes + 8 * i * kRow));
  const uint4* sp = reinterpret_cast<const uint4*>(a.k_scale + grp + (KB == 2 ? 16 : 8) * l.word);
  r.scale[0] = __ldg(sp);
  if constexpr (KB == 2) r.scale[1] = __ldg(sp + 1);
  r.four = __ldg(reinterpret_cast<const uint2*>(a.k_scale + grp) + l.lane);
  if (l.w == g) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r.cs[i] = __ldg(reinterpret_cast<const uint32_t*>(a.k_scale + grp + l.ch() + i * l.kTo));
      r.cz[i] = __ldg(reinterpret_cast<const uint32_t*>(a.k_zero + grp + l.ch() + i * l.kTo));
    }
  }
}
template <int KB>
__device__ __forceinline__ void store_keys(const CodeScale& cs0, const KiviTreeArgs& a, const TreeLens& len, int h, int t, int g,
                                           const KeyLane<KB>& l, const KeyRegs<KB>& r, unsigned char* dst,
                                           unsigned char* rest, float* unit) {
  constexpr int kPairs = KB == 2 ? 8 : 4;
  const int at0 = (4 * g + l.oct) * 2048 + l.word * (kPairs * 32) + (l.lane & 7) * 16;
  unsigned char* cdst = dst + kTok * kD * 2 + 2 * (l.lane >> 2) * 128 + ((l.lane & 3) >> 1) * 128 + 2 * g * 16 + (l.lane & 1) * 8;
  if (t < len.nqk) {
    const __half2 most2 = __hmax2(__habs2(as_h2(r.four.x)), __habs2(as_h2(r.four.y)));
    const int e = 26 - (int)(__reduce_max_sync(0xFFFFFFFFu, max(as_u(most2) & 0xFFFFu, as_u(most2) >> 16)) >> 10);  // -5 .. 26
    if (l.w == g) {
      float2 y[2];
      const float2 sa = __half22float2(as_h2(r.cs[0])), sb = __half22float2(as_h2(r.cs[1]));
      const float2 za = __half22float2(as_h2(r.cz[0])), zb = __half22float2(as_h2(r.cz[1]));
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
      if (l.lane == 0) {
        unit[g] = __uint_as_float((uint32_t)(127 - e) << 23);
        unit[4 + g] = __uint_as_float((uint32_t)(127 - sh) << 23);
      }
    }
    // the scales times the power of two that puts the group's largest in [2^11, 2^12)
    const __half2 f0 = as_h2((uint32_t)(min(e, 15) + 15) * 0x4000400u), f1 = as_h2((uint32_t)(max(e, 15)) * 0x4000400u);
    __half2 s[kPairs];
    uint4 s0, s1;
    pair_order<KB>(r.scale[0], r.scale[KB == 2 ? 1 : 0], s0, s1);
    const uint32_t sw[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int j = 0; j < kPairs; ++j) s[j] = __hmul2(as_h2(sw[j]), f0);
    if (e > 15) {  // the rest of a power past the largest fp16 one
#pragma unroll
      for (int j = 0; j < kPairs; ++j) s[j] = __hmul2(s[j], f1);
    }
#pragma unroll
    for (int i = 0; i < KeyRegs<KB>::kOct; ++i) {
      uint32_t x[kPairs], y[kPairs];
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const __half2 c = code_h2<KB, kCentre<KB>>(cs0, r.code[i], j);
        x[j] = as_u(__hmul2(c, s[j]));
        if constexpr (KB == 4) y[j] = product_rest(as_u(c), as_u(s[j]), x[j]);
      }
      *reinterpret_cast<uint4*>(dst + at0 + 2048 * i) = make_uint4(x[0], x[1], x[2], x[3]);
      if constexpr (KB == 2) *reinterpret_cast<uint4*>(dst + at0 + 2048 * i + 128) = make_uint4(x[4], x[5], x[6], x[7]);
      else *reinterpret_cast<uint4*>(rest + at0 + 2048 * i) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  } else {  // fp16 rows, or none
    if (l.w == g) {
      *reinterpret_cast<uint2*>(cdst) = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(cdst + 16) = make_uint2(0u, 0u);
      if (l.lane == 0) unit[g] = unit[4 + g] = 1.f;
    }
#pragma unroll 1
    for (int i = 0; i < KeyRegs<KB>::kOct; ++i) {
      const uint16_t* row = fp16_key(a, len, 0, h, t + 8 * (l.oct + i) + (l.lane & 7));
      uint4 x0, x1;
      if constexpr (KB == 2) {
        pair_order<2>(row8(row, 2 * l.word), row8(row, 2 * l.word + 1), x0, x1);
        *reinterpret_cast<uint4*>(dst + at0 + 2048 * i + 128) = x1;
      } else {
        const uint4 v = row8(row, l.word);
        pair_order<4>(v, v, x0, x1);
        *reinterpret_cast<uint4*>(rest + at0 + 2048 * i) = make_uint4(0u, 0u, 0u, 0u);
      }
      *reinterpret_cast<uint4*>(dst + at0 + 2048 * i) = x0;
    }
  }
}

// ---- values of 32 tokens and a value group w (32 channels), by one warp: a lane a token ----
template <int VB>
struct ValueRegs {
  uint32_t code[VB];
  uint16_t s, z;
};
template <int VB>
__device__ __forceinline__ void load_values(const KiviTreeArgs& a, const TreeLens& len, int h, int t, int w, ValueRegs<VB>& r) {
  if (t >= len.nqv) return;
  const size_t tok = (size_t)h * a.max_tokens + t;
  const uint8_t* src = a.v_codes + tok * (kD * VB / 8) + 4 * VB * w;
  if constexpr (VB == 2) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(src));
    r.code[0] = u.x; r.code[1] = u.y;
  } else {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(src));
    r.code[0] = u.x; r.code[1] = u.y; r.code[2] = u.z; r.code[3] = u.w;
  }
  r.s = __ldg(a.v_scale + tok * (kD / kGroupT) + w);
  r.z = __ldg(a.v_zero + tok * (kD / kGroupT) + w);
}
// t: the lane's token; dst: its place in V'
template <int VB>
__device__ __forceinline__ void store_values(const CodeScale& cs0, const KiviTreeArgs& a, const TreeLens& len, int h, int t, int w,
                                             const ValueRegs<VB>& r, unsigned char* dst) {
  // columns of the constants: s z, what its rounding left, c0 s (all halved as the values), 1
  uint2 c = make_uint2(0u, 0x3C000000u);
  if (t < len.nqv) {
    const __half2 s2 = as_h2(halved(r.s * 0x10001u));
    const uint32_t p = as_u(__hmul2(s2, as_h2(r.z * 0x10001u))), left = product_rest(as_u(s2), r.z * 0x10001u, p);
    c.x = (p & 0xFFFFu) | (left << 16);
    c.y |= as_u(__hmul2(s2, __float2half2_rn(kCentre<VB>))) & 0xFFFFu;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t word = VB == 4 ? r.code[i & (VB - 1)] : r.code[i >> 1] >> (16 * (i & 1));
      *reinterpret_cast<uint4*>(dst + (4 * w + i) * kVSbo) = centred8<VB>(cs0, word, s2);
    }
  } else {
    const uint16_t* row = nullptr;
    if (t < len.n) row = fp16_value(a, len, 0, h, t, t - div_by(t, a.ring) * a.residual);
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const uint4 v = row8(row, 4 * w + i);
      *reinterpret_cast<uint4*>(dst + (4 * w + i) * kVSbo) = make_uint4(halved(v.x), halved(v.y), halved(v.z), halved(v.w));
    }
  }
  *reinterpret_cast<uint2*>(dst + (16 + (w >> 1)) * kVSbo + (w & 1) * 8) = c;
}

// the stored part of a tile into L2, by one thread
template <int KB, int VB>
__device__ __forceinline__ void prefetch_tile(const KiviTreeArgs& a, const TreeLens& len, int h, int t0) {
  const size_t tok = (size_t)h * a.max_tokens + t0, g = tok / kGroupT * kD;
  const int nk = min(kTok, len.nqk - t0), nv = (min(kTok, len.nqv - t0) + 1) & ~1;  // whole 16-byte pieces
  if (nk > 0) {
    bulk_prefetch_l2(a.k_codes + tok * (kD * KB / 8), nk * (kD * KB / 8));
    bulk_prefetch_l2(a.k_scale + g, nk / kGroupT * kD * 2);
    bulk_prefetch_l2(a.k_zero + g, nk / kGroupT * kD * 2);
  }
  if (nv > 0) {
    bulk_prefetch_l2(a.v_codes + tok * (kD * VB / 8), nv * (kD * VB / 8));
    bulk_prefetch_l2(a.v_scale + tok * (kD / kGroupT), nv * 8);
    bulk_prefetch_l2(a.v_zero + tok * (kD / kGroupT), nv * 8);
  }
}

template <int KB, int VB>
__global__ void __launch_bounds__(kThreads, 1) kivi_prefix_kernel(const KiviTreeArgs a, const float scale_log2) {
  using L = PrefixLayout<KB>;
  extern __shared__ __align__(128) unsigned char sm[];
  float* unit = reinterpret_cast<float*>(sm + L::kOffUnit);
  uint64_t* bar_q = reinterpret_cast<uint64_t*>(sm + L::kOffBar);  // [2] a row tile's queries are there
  uint64_t* bar_s = bar_q + 2;                                      // [2] its scores
  uint64_t* bar_p = bar_q + 4;                                      // [2] its weights
  uint64_t* bar_o = bar_q + 6;                                      // [2] its value product is done
  uint64_t* k_full = bar_q + 8;                                     // [2] a stage's keys are unpacked
  uint64_t* k_empty = bar_q + 10;                                   // [2] and read
  uint64_t* v_full = bar_q + 12;
  uint64_t* v_empty = bar_q + 14;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_q + 16);
  volatile int* failed = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const TreeLens len = tree_lens(a, 0, kTok);
  const PrefixPlace at = prefix_place(a, len, blockIdx.x);
  if (at.p0 >= at.p1) return;
  const int rows_all = a.N * a.rep.d;
  if (warp == 15) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_q + i, 128);
      mbar_init(bar_s + i, 1);
      mbar_init(bar_p + i, 128);
      mbar_init(bar_o + i, 1);
      mbar_init(k_full + i, 128);
      mbar_init(k_empty + i, 1);
      mbar_init(v_full + i, 32 * kGroups);
      mbar_init(v_empty + i, 1);
    }
    *failed = 0;
    fence_mbar_init();
  }
  tmem_before();
  __syncthreads();
  tmem_after();
  const uint32_t tmem = *tmem_slot;
  // a wait that runs out ends its role, and with it the waits of the others
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_wait_bounded_sleep(bar, parity & 1)) return true;
    *failed = 1;
    set_error(a.err, KVQ_ERR_TIMEOUT);
    return false;
  };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity)) != 0; };
  int seg = at.p0 / at.T, tile = at.p0 - seg * at.T;
  // row tiles of the segment: the second one may hold no row
  auto second = [&](int sg) { return rows_all - (sg - div_by(sg, a.row_tiles) * a.row_tiles.d) * kRows > 128; };

  if (warp < 8) {
    // ================= softmax: row tile r, a thread a row =================
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
          // the tile's queries: 8 lanes a row, four rows a warp at a time
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
          mbar_arrive(bar_q + r);
        }
        if (!wait_warp(bar_s + r, n)) break;
        tmem_after();
        // ---- scores in log2 units; they are rounded before the maximum is taken from them, so that the largest one's
        //      weight is exact however large it is ----
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
            for (int i = 0; i < 16; ++i)
              x[16 * g + i] = __fmul2_rn(__ffma2_rn(x[16 * g + i], make_float2(f, f), make_float2(z, z)), make_float2(rowc, rowc));
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
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        const bool up = mx + nm > kSlack + kRaise;
        if (__any_sync(0xFFFFFFFFu, up)) {
          const float f = up ? exp2_approx((kRaise - mx) - nm) : 1.f;
          if (up) nm = kRaise - mx;
          if (!first) {  // the sums, once the value product of the tile before is done
            if (!wait_warp(bar_o + r, n - 1)) break;
            tmem_after();
#pragma unroll 1
            for (int i = 0; i < (int)kColO; i += 8) {
              uint32_t u[8];
              float o[8];
              tmem_ld8(t_o + i, u);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = __uint_as_float(u[e]) * f;
              tmem_st8(t_o + i, o);
            }
          }
        }
        // ---- weights, into the scores' columns ----
#pragma unroll
        for (int c = 0; c < kTok / 32; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 d = __fadd2_rn(x[16 * c + i], make_float2(nm, nm));
            w[i] = pack_h2(exp2_approx(d.x), exp2_approx(d.y));
          }
          tmem_st16(t_s + 16 * c, w);
        }
        tmem_wait_st();
        tmem_before();
        mbar_arrive(bar_p + r);
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
  } else if (warp < 12) {
    // ================= keys: four warps, the next group on its way meanwhile =================
    const CodeScale cs0;
    const KeyLane<KB> kl(warp & 3, lane);
    KeyRegs<KB> now, next;
    int h = div_by(seg, a.row_tiles);
    // the place kAhead tiles on, whose stored part is fetched into L2
    constexpr int kAhead = 4;
    auto fetch = [&](int p) {
      if (p >= at.p1) return;
      const int fseg = p / at.T;
      prefetch_tile<KB, VB>(a, len, div_by(fseg, a.row_tiles), (p - fseg * at.T) * kTok);
    };
    load_keys<KB>(a, len, h, tile * kTok, 0, kl, now);
    int g = 0, p = at.p0;
#pragma unroll 1
    while (p < at.p1) {
      const int it = p - at.p0, st = it & 1, t = tile * kTok + g * kGroupT, h0 = h, g0 = g;
      if (g == 0) {
        if (warp == 8 && lane == 0) fetch(p + kAhead);
        if (it >= 2 && !wait_warp(k_empty + st, (it >> 1) + 1)) break;
      }
      if (++g == kGroups) {
        g = 0;
        ++p;
        if (++tile == at.T) {
          tile = 0;
          h = div_by(++seg, a.row_tiles);
        }
      }
      if (p < at.p1) load_keys<KB>(a, len, h, tile * kTok + g * kGroupT, g, kl, next);
      store_keys<KB>(cs0, a, len, h0, t, g0, kl, now, sm + L::kOffK + st * L::kK, sm + L::kOffKr + st * L::kKr,
                     unit + ((at.p0 + it) & 3) * 8);
      if (g == 0) {
        fence_proxy_async_smem();
        mbar_arrive(k_full + st);
      }
      now = next;
    }
  } else if (warp < 12 + kGroups) {
    // ================= values: a warp a 32-token group, one value group after the other =================
    const CodeScale cs0;
    ValueRegs<VB> now, next;
    int h = div_by(seg, a.row_tiles);
    const int lt = 32 * (warp - 12) + lane;  // the lane's token of the tile
    load_values<VB>(a, len, h, tile * kTok + lt, 0, now);
    int w = 0, p = at.p0;
#pragma unroll 1
    while (p < at.p1) {
      const int it = p - at.p0, st = it & 1, t = tile * kTok + lt, h0 = h, w0 = w;
      if (w == 0 && it >= 2 && !wait_warp(v_empty + st, (it >> 1) + 1)) break;
      if (++w == 4) {
        w = 0;
        ++p;
        if (++tile == at.T) {
          tile = 0;
          h = div_by(++seg, a.row_tiles);
        }
      }
      if (p < at.p1) load_values<VB>(a, len, h, tile * kTok + lt, w, next);
      store_values<VB>(cs0, a, len, h0, t, w0, now, sm + L::kOffV + st * L::kV + lt * 16);
      if (w == 0) {
        fence_proxy_async_smem();
        mbar_arrive(v_full + st);
      }
      now = next;
    }
  } else if (lane == 0) {
    // ================= products =================
    const uint64_t desc_q = tree_desc(smem_u32(sm + L::kOffQ), 128, 2048);
    const uint64_t desc_k = tree_desc(smem_u32(sm + L::kOffK), 128, 2048);
    const uint64_t desc_kr = tree_desc(smem_u32(sm + L::kOffKr), 128, 2048);
    const uint64_t desc_v = tree_desc(smem_u32(sm + L::kOffV), 128, kVSbo);
    uint32_t n[2] = {0, 0}, parts[2] = {0, 0};  // tiles, and parts of segments, of each row tile
    // the scores of row tile r for the tile in stage st; starts: the part's first
    auto scores = [&](int r, int st, bool starts) {
      if (starts && !wait(bar_q + r, parts[r]++)) return false;
      tmem_after();
      const uint64_t q = desc_q + r * (128 * kD * 2 / 16), k = desc_k + st * (L::kK / 16);
#pragma unroll
      for (int i = 0; i < 8; ++i) umma_f16(tmem + r * kColS, q + 16 * i, k + 16 * i, tree_idesc(kColS, false), i > 0);
      if constexpr (KB == 4) {
        const uint64_t kk = desc_kr + st * (L::kKr / 16);
#pragma unroll
        for (int i = 0; i < 8; ++i) umma_f16(tmem + r * kColS, q + 16 * i, kk + 16 * i, tree_idesc(kTok, false), 1);
      }
      tree_commit(bar_s + r);
      return true;
    };
    bool ok = true, starts = true;
    int last_r = second(seg) ? 1 : 0;
    ok = wait(k_full, 0);
    for (int r = 0; ok && r <= last_r; ++r) ok = scores(r, 0, true);
    if (ok) tree_commit(k_empty);
    for (int p = at.p0; ok && p < at.p1; ++p) {
      const int it = p - at.p0, st = it & 1;
      const bool ends = tile + 1 == at.T, more = p + 1 < at.p1;
      const int nseg = ends ? seg + 1 : seg, next_r = !more ? -1 : second(nseg) ? 1 : 0;
      if (more) ok = wait(k_full + (st ^ 1), (it + 1) >> 1);
      if (ok) ok = wait(v_full + st, it >> 1);
      for (int r = 0; ok && r < 2; ++r) {
        if (r <= last_r) {
          if (!(ok = wait(bar_p + r, n[r]))) break;
          tmem_after();
          const uint64_t v = desc_v + st * (L::kV / 16);
#pragma unroll
          for (int i = 0; i < kTok / 16; ++i)
            umma_f16_ta(tmem + 2 * kColS + r * kColO, tmem + r * kColS + 8 * i, v + 16 * i, tree_idesc(kColO, true), !starts || i > 0);
          tree_commit(bar_o + r);
          if (r == last_r) tree_commit(v_empty + st);
          // the scores of the next tile take the columns that this product reads
          if (!(ok = wait(bar_o + r, n[r]))) break;
          ++n[r];
        }
        if (r <= next_r) {
          if (!(ok = scores(r, st ^ 1, ends))) break;
          if (r == next_r) tree_commit(k_empty + (st ^ 1));
        }
      }
      starts = ends;
      last_r = next_r;
      seg = nseg;
      tile = ends ? 0 : tile + 1;
    }
    if (!ok) {  // let what was issued end before the memory goes
      mbar_wait_bounded(bar_s, n[0] & 1, 10000000ull);
      mbar_wait_bounded(bar_s + 1, n[1] & 1, 10000000ull);
      mbar_wait_bounded(bar_o, n[0] & 1, 10000000ull);
      mbar_wait_bounded(bar_o + 1, n[1] & 1, 10000000ull);
    }
  }
  __syncwarp();
  tmem_before();
  __syncthreads();
  if (warp == 15) {
    tmem_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// ======================================================================================
// Joining the two sides
// ======================================================================================

// A warp a row, a lane four channels.
constexpr int kCombineThreads = 128;
__device__ __forceinline__ void combine_row(const KiviPrefixArgs& a, size_t at, float l0, float4 x, float l1, float4 y) {
  // a side that saw nothing stays out, whatever its row holds; one that is not a number says so in the result
  const float top = fmaxf(fmaxf(l0, l1), -FLT_MAX);
  float w0 = l0 != l0 ? l0 : exp2f(l0 - top), w1 = l1 != l1 ? l1 : exp2f(l1 - top);
  const float sum = w0 + w1;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  w0 *= inv;
  w1 *= inv;
  auto mix = [&](float p, float q) { return (w0 == 0.f ? 0.f : w0 * p) + (w1 == 0.f ? 0.f : w1 * q); };
  const float v[4] = {mix(x.x, y.x), mix(x.y, y.y), mix(x.z, y.z), mix(x.w, y.w)};
  if (a.out_fp32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
        make_uint2(f32_to_bf16(v[0]) | ((uint32_t)f32_to_bf16(v[1]) << 16), f32_to_bf16(v[2]) | ((uint32_t)f32_to_bf16(v[3]) << 16));
}
__global__ void __launch_bounds__(kCombineThreads) kivi_prefix_combine_kernel(const KiviPrefixArgs a, const int rows) {
  const int row = blockIdx.x * (kCombineThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= rows) return;
  const int tok = div_by(row, a.heads), b = div_by(tok, a.tokens);
  if (a.own.n_draft && tok - b * a.own.N >= a.own.n_draft[b]) return;  // padding
  const size_t at = (size_t)row * kD + 4 * lane;
  combine_row(a, at, a.prefix.lse[row], *reinterpret_cast<const float4*>(static_cast<const float*>(a.prefix.out) + at), a.own.lse[row],
              *reinterpret_cast<const float4*>(static_cast<const float*>(a.own.out) + at));
}

// The same behind the kernel above: the parts of a segment lie in the slots block + segment of the blocks that shared
// it. A block takes eight rows of a KV head, a thread four channels of one of them.
constexpr int kJoinThreads = 256, kJoinRows = 8;
__global__ void __launch_bounds__(kJoinThreads) kivi_prefix_join_kernel(const KiviPrefixArgs a) {
  const KiviTreeArgs& t = a.prefix;
  const int lane = threadIdx.x & 31, c = 4 * (threadIdx.x >> 5) + (lane >> 3), h = blockIdx.y;
  const int row = blockIdx.x * kJoinRows + (lane & 7);  // of the KV head
  if (row >= t.N * t.rep.d) return;
  const int tok = div_by(row, t.rep), b = div_by(tok, a.tokens);
  if (a.own.n_draft && tok - b * a.own.N >= a.own.n_draft[b]) return;  // padding
  const size_t out_row = (size_t)tok * t.Hq + h * t.rep.d + row - tok * t.rep.d;
  const TreeLens len = tree_lens(t, 0, kTok);
  const int T = (int)((uint32_t)(len.n + kTok - 1) / kTok), P = T * t.segs.d;
  const int seg = h * t.row_tiles.d + row / kRows, r = row & (kRows - 1);
  float top = -FLT_MAX, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (T > 0) {
    // the first block that holds a position of the segment
    const int begin = seg * T, end = begin + T;
    int k = P <= t.blocks.d ? begin : (int)((long long)begin * t.blocks.d / P);
    while (k > 0 && share_begin(P, k, t.blocks) > begin) --k;
    while (share_begin(P, k + 1, t.blocks) <= begin) ++k;
    for (; k < t.blocks.d && share_begin(P, k, t.blocks) < end; ++k) {
      const float* slot = t.part + (size_t)(k + seg) * kSlotFloats;
      const float m = slot[(size_t)kRows * kD + r], lp = slot[(size_t)kRows * (kD + 1) + r];
      const float4 v = reinterpret_cast<const float4*>(slot)[c * kRows + r];
      if (lp == 0.f) continue;  // the row saw nothing there
      const float up = fmaxf(top, m), f = l == 0.f ? 0.f : exp2_approx(top - up), w = lp != lp ? 1.f : exp2_approx(m - up);
      top = up;
      l = (f == 0.f ? 0.f : l * f) + (w == 0.f ? 0.f : lp * w);
      auto add = [&](float x, float y) { return (f == 0.f ? 0.f : x * f) + (w == 0.f ? 0.f : y * w); };
      o = make_float4(add(o.x, v.x), add(o.y, v.y), add(o.z, v.z), add(o.w, v.w));
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const size_t at = out_row * kD + 4 * c;
  combine_row(a, at, l == 0.f ? -INFINITY : top + __log2f(l), make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv), a.own.lse[out_row],
              *reinterpret_cast<const float4*>(static_cast<const float*>(a.own.out) + at));
}

template <int KB, int VB>
cudaError_t launch_prefix_rows(const KiviTreeArgs& a, cudaStream_t st) {
  auto kernel = kivi_prefix_kernel<KB, VB>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PrefixLayout<KB>::kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<a.blocks.d, kThreads, PrefixLayout<KB>::kSmem, st>>>(a, 1.4426950408889634f / sqrtf((float)kD));
  return cudaGetLastError();
}

// Rows of a KV head from which on the kernel of this file takes the prefix
bool many_rows(int rows) { return rows > 64; }
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
    e = t.k_bits == 2 ? (t.v_bits == 2 ? launch_prefix_rows<2, 2>(t, st) : launch_prefix_rows<2, 4>(t, st))
                      : (t.v_bits == 2 ? launch_prefix_rows<4, 2>(t, st) : launch_prefix_rows<4, 4>(t, st));
  } else {
    e = launch_kivi_tree(t, st);
  }
  if (e != cudaSuccess) return e;
  if ((e = launch_kivi_tree(a.own, st)) != cudaSuccess) return e;
  if (many) {
    kivi_prefix_join_kernel<<<dim3((rows + kJoinRows - 1) / kJoinRows, t.H), kJoinThreads, 0, st>>>(a);
  } else {
    const int all = a.own.B * a.own.N * a.own.Hq, per = kCombineThreads / 32;
    kivi_prefix_combine_kernel<<<(all + per - 1) / per, kCombineThreads, 0, st>>>(a, all);
  }
  return cudaGetLastError();
}

}  // namespace kvq
