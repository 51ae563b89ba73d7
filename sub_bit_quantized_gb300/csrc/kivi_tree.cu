// Attention of a tree of drafted tokens over a KIVI cache.
//
// Request b has n cached tokens and up to N <= 64 drafted ones with their own fp16 keys and
// values. Drafted token i attends every cached token and the drafted tokens j whose bit is set
// in its mask, with one softmax over both (scale 1/sqrt(D)):
//   o_i = sum_t p_it v_t / sum_t p_it,  p_it = exp(q_i k_t / sqrt(D) - m_i).
// The rows of a KV head are the N drafted tokens times its n_q_heads / n_heads query heads.
//
// Tokens (cached, then drafted) form tiles of 128. For a tile and up to kRows query rows:
//   S^T [128 tokens x rows] = K [128 x 128] . q^T      tcgen05, K dequantized to fp16
//   P^T = exp2(S^T c - m)                               a thread owns a token and half the rows
//   O^T [128 channels x rows] += V^T [128 x 128] . P^T  tcgen05, V dequantized to fp16
// so the 128 lanes of every product are full however few rows there are, and no shuffle is
// needed inside the tile: the running maximum m of a row moves only when a score passes it by
// 2^kSlack (a block-wide vote), the sums l stay per thread until the segment ends.
#include <cuda_fp16.h>

#include <cfloat>

#include "kvq_common.cuh"
#include "kvq_internal.h"
#include "../../include/kvq.h"

namespace kvq {
namespace {

constexpr int kTreeThreads = 256;
constexpr int kTreeWarps = kTreeThreads / 32;
constexpr int kTile = 128;    // tokens per tile (MMA M of the scores, K of the value product)
constexpr int kGroupT = 32;   // tokens per key group, channels per value group
constexpr float kSlack = 7.f;   // log2 by which a score may pass its row's running maximum
constexpr float kRaise = 8.f;   // weights are exp2(x - m + kRaise) <= 2^15, held as fp16: one below 2^-32 of the
                                // maximum's is lost instead of one below 2^-24

// V^T is staged in 8 channel x 8 token core matrices: the 16 of a row group (8 channels) are contiguous, row
// groups 2064 bytes apart, so that eight threads with eight row groups store to different banks
constexpr int kVRowGrp = (kTile / 8) * 128 + 16;

template <int KB, int VB, int ROWS>
struct TreeLayout {
  static constexpr int kKRow = kD * KB / 8, kVRow = kD * VB / 8;   // code bytes per token
  static constexpr int kOffQ = 0;                                  // fp16 [ROWS x 128], K-major
  static constexpr int kOffK = kOffQ + ROWS * kD * 2;              // fp16 [128 tokens x 128], K-major; then P
  static constexpr int kOffV = kOffK + kTile * kD * 2;             // fp16 [128 channels x 128 tokens], K-major
  // a tile as it is stored: key codes, scales and zeros [4 groups][128], value codes, scales and zeros [128][4]
  static constexpr int kOffKc = (kOffV + (kD / 8) * kVRowGrp + 127) / 128 * 128;
  static constexpr int kOffKs = kOffKc + kTile * kKRow;
  static constexpr int kOffKz = kOffKs + (kTile / kGroupT) * kD * 2;
  static constexpr int kOffVc = kOffKz + (kTile / kGroupT) * kD * 2;
  static constexpr int kOffVs = kOffVc + kTile * kVRow;
  static constexpr int kOffVz = kOffVs + kTile * (kD / kGroupT) * 2;
  static constexpr int kOffMask = kOffVz + kTile * (kD / kGroupT) * 2;  // uint64 [ROWS]
  static constexpr int kOffC = kOffMask + ROWS * 8;                // float [ROWS]: log2 units per score unit
  static constexpr int kOffM = kOffC + ROWS * 4;                   // float [ROWS]: running maximum (log2) - kRaise
  static constexpr int kOffT = kOffM + ROWS * 4;                   // float [ROWS]: running maximum + kSlack
  static constexpr int kOffF = kOffT + ROWS * 4;                   // float [ROWS]: rescale factor
  static constexpr int kOffRed = kOffF + ROWS * 4;                 // float [4][ROWS]: per lane quadrant
  static constexpr int kOffBar = kOffRed + 4 * ROWS * 4;           // mbarriers, TMEM address, flags
  static constexpr int kSmem = kOffBar + 64;
  static constexpr uint32_t kCols = 2 * ROWS < 32 ? 32 : 2 * ROWS;  // TMEM: S^T, O^T
  static constexpr uint32_t kKBytes = kOffVc - kOffKc, kVBytes = kOffMask - kOffVc;
  static_assert(ROWS * 256 <= kTile * kD * 2, "P fits in the key tile");
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
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}

__device__ __forceinline__ float th2f(uint32_t b) { return __half2float(__ushort_as_half((unsigned short)b)); }
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The work of a call, the same for every block: segment (b, h, row tile) has T_b tiles (its cached
// and drafted tokens), all segments in the order b, h, row tile form one list of P tile positions,
// and block k of G takes positions [k P / G, (k + 1) P / G).
struct TreeLens {
  int nqk, nqv, n, nd;  // quantized keys, quantized values, cached tokens, drafted tokens
  int tiles;
};
__device__ __forceinline__ TreeLens tree_lens(const KiviTreeArgs& a, int b) {
  TreeLens L;
  L.nqk = min(max(a.n_quant_k[b], 0), a.max_tokens) / kGroupT * kGroupT;
  L.nqv = (a.residual > 0) ? min(max(a.n_quant_v[b], 0), L.nqk) : L.nqk;
  L.n = L.nqk + max(0, min(a.n_tok[b] - L.nqk, a.residual));
  L.nd = a.n_draft ? min(max(a.n_draft[b], 0), a.N) : a.N;
  L.tiles = L.nd > 0 ? (int)(((long long)L.n + L.nd + kTile - 1) / kTile) : 0;
  return L;
}
__device__ __forceinline__ long long share_begin(long long P, int k, int G) { return P * k / G; }
// the block whose share holds position p
__device__ __forceinline__ int share_of(long long P, long long p, int G) { return (int)(((p + 1) * G - 1) / P); }

// partial softmax of a segment: rows of o[128], then m, l per row
template <int ROWS>
__host__ __device__ constexpr size_t slot_floats() { return (size_t)ROWS * (kD + 2); }

struct Token {
  const KiviTreeArgs* a;
  TreeLens L;
  size_t bh;  // b * H + h
  int b, h;
};

// channels 8c .. 8c+7 of token t's key / value as fp16 (zero past the last drafted token)
template <int KB>
__device__ __forceinline__ uint4 key8(const Token& k, int t, int c) {
  const KiviTreeArgs& a = *k.a;
  if (t < k.L.nqk) {
    const uint8_t* row = a.k_codes + (k.bh * a.max_tokens + t) * (kD * KB / 8);
    const uint32_t w = (KB == 2) ? __ldg(reinterpret_cast<const uint16_t*>(row) + c) : __ldg(reinterpret_cast<const uint32_t*>(row) + c);
    const size_t g = (k.bh * (a.max_tokens / kGroupT) + t / kGroupT) * kD + 8 * c;
    const uint4 s = __ldg(reinterpret_cast<const uint4*>(a.k_scale + g)), z = __ldg(reinterpret_cast<const uint4*>(a.k_zero + g));
    const uint32_t sw[4] = {s.x, s.y, s.z, s.w}, zw[4] = {z.x, z.y, z.z, z.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c0 = (float)((w >> (KB * 2 * i)) & ((1 << KB) - 1)), c1 = (float)((w >> (KB * (2 * i + 1))) & ((1 << KB) - 1));
      o[i] = pack_h2(th2f(sw[i] & 0xFFFFu) * (c0 - th2f(zw[i] & 0xFFFFu)), th2f(sw[i] >> 16) * (c1 - th2f(zw[i] >> 16)));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (t < k.L.n)
    return __ldg(reinterpret_cast<const uint4*>(a.k_resid + (k.bh * a.residual + (t - k.L.nqk)) * kD + 8 * c));
  if (t < k.L.n + k.L.nd)
    return __ldg(reinterpret_cast<const uint4*>(a.k_draft + (((size_t)k.b * a.N + (t - k.L.n)) * a.H + k.h) * kD + 8 * c));
  return make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ bool half2_finite(uint32_t w) { return (w & 0x7C00u) != 0x7C00u && (w & 0x7C000000u) != 0x7C000000u; }
template <int VB>
__device__ __forceinline__ uint4 value8(const Token& k, int t, int c, int* nonfinite) {
  const KiviTreeArgs& a = *k.a;
  if (t < k.L.nqv) {
    const size_t tok = k.bh * a.max_tokens + t;
    const uint8_t* row = a.v_codes + tok * (kD * VB / 8);
    const uint32_t w = (VB == 2) ? __ldg(reinterpret_cast<const uint16_t*>(row) + c) : __ldg(reinterpret_cast<const uint32_t*>(row) + c);
    const float s = th2f(__ldg(a.v_scale + tok * (kD / kGroupT) + c / 4)), z = th2f(__ldg(a.v_zero + tok * (kD / kGroupT) + c / 4));
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c0 = (float)((w >> (VB * 2 * i)) & ((1 << VB) - 1)), c1 = (float)((w >> (VB * (2 * i + 1))) & ((1 << VB) - 1));
      o[i] = pack_h2(s * (c0 - z), s * (c1 - z));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (t < k.L.n) return __ldg(reinterpret_cast<const uint4*>(a.v_resid + (k.bh * a.residual + t % a.residual) * kD + 8 * c));
  if (t < k.L.n + k.L.nd) {
    // A drafted value is seen only by the rows whose mask has it, but the product multiplies it by
    // every row's weight, 0 for the others: one that is not finite is staged as 0 and added at the
    // end to the rows that see it.
    uint4 u = __ldg(reinterpret_cast<const uint4*>(a.v_draft + (((size_t)k.b * a.N + (t - k.L.n)) * a.H + k.h) * kD + 8 * c));
    if (!(half2_finite(u.x) && half2_finite(u.y) && half2_finite(u.z) && half2_finite(u.w))) {
      *nonfinite = 1;
      uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if ((w[i] & 0x7C00u) == 0x7C00u) w[i] &= 0xFFFF0000u;
        if ((w[i] & 0x7C000000u) == 0x7C000000u) w[i] &= 0xFFFFu;
      }
      u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return u;
  }
  return make_uint4(0u, 0u, 0u, 0u);
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
// Code j of both halves of w as fp16 (exact): masked in place under the exponent of 2^10, where it stands for
// 1024 + c 2^(b j), and scaled back by one FMA. Codes above the ten mantissa bits come from w shifted right.
template <int BITS>
__device__ __forceinline__ __half2 code_h2(uint32_t w, int j) {
  constexpr int kIn = (BITS == 2) ? 5 : 2;  // codes that fit in place
  const int jj = j < kIn ? j : j - kIn;
  const uint32_t m = ((j < kIn ? w : w >> (BITS * kIn)) & ((((1u << BITS) - 1u) << (BITS * jj)) * 0x10001u)) | 0x64006400u;
  const float p = 1.f / (float)(1 << (BITS * jj));
  return __hfma2(as_h2(m), __float2half2_rn(p), __float2half2_rn(-1024.f * p));
}
// s c - s z, one rounding of s z and one of the result
__device__ __forceinline__ uint32_t dequant_h2(__half2 c, __half2 s, __half2 nsz) { return as_u(__hfma2(c, s, nsz)); }
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int KB, int VB, int ROWS>
__global__ void __launch_bounds__(kTreeThreads, 2) kivi_tree_kernel(const KiviTreeArgs a, const float scale_log2) {
  using L = TreeLayout<KB, VB, ROWS>;
  extern __shared__ __align__(128) unsigned char sm[];
  uint64_t* mask = reinterpret_cast<uint64_t*>(sm + L::kOffMask);
  float* rowc = reinterpret_cast<float*>(sm + L::kOffC);
  float* rowm = reinterpret_cast<float*>(sm + L::kOffM);
  float* rowt = reinterpret_cast<float*>(sm + L::kOffT);
  float* rowf = reinterpret_cast<float*>(sm + L::kOffF);
  float* red = reinterpret_cast<float*>(sm + L::kOffRed);
  uint64_t* bar_s = reinterpret_cast<uint64_t*>(sm + L::kOffBar);  // scores done
  uint64_t* bar_o = bar_s + 1;                                      // value product done
  uint64_t* bar_k = bar_s + 2;                                      // the tile's stored keys landed
  uint64_t* bar_v = bar_s + 3;                                      // its stored values
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_s + 4);
  volatile int* failed = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* nonfinite = reinterpret_cast<int*>(tmem_slot + 2);
  long long* scan = reinterpret_cast<long long*>(sm);  // before the first tile: one per thread

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rep = a.Hq / a.H, rows_all = a.N * rep;
  const int n_rt = (rows_all + ROWS - 1) / ROWS;  // row tiles of a KV head
  const int seg_per_b = a.H * n_rt;

  // ---- the block's share: tiles of all requests, and the request its first position lies in ----
  const int chunk = (a.B + kTreeThreads - 1) / kTreeThreads;
  const int chunks = (a.B + chunk - 1) / chunk;  // threads with requests
  long long mine = 0;
  for (int b = tid * chunk; b < min(a.B, (tid + 1) * chunk); ++b) mine += tree_lens(a, b).tiles;
  scan[tid] = mine;
  __syncthreads();
  long long P = 0, before = 0;
  for (int i = 0; i < chunks; ++i) P += scan[i];
  P *= seg_per_b;
  const long long p0 = share_begin(P, blockIdx.x, gridDim.x), p1 = share_begin(P, blockIdx.x + 1, gridDim.x);
  if (p0 >= p1) return;  // uniform
  int c0 = 0;
  while (p0 >= (before + scan[c0]) * seg_per_b) before += scan[c0++];  // ends: p0 < P
  int b = c0 * chunk;
  TreeLens len = tree_lens(a, b);
  while (p0 >= (before + len.tiles) * seg_per_b) {  // ends inside chunk c0
    before += len.tiles;
    len = tree_lens(a, ++b);
  }
  int seg = (int)((p0 - before * seg_per_b) / len.tiles);  // h * n_rt + row tile
  int tile = (int)((p0 - before * seg_per_b) % len.tiles);
  __syncthreads();

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(L::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // the stored keys (values) of a tile whose tokens are all quantized: into the stage by bulk copies
  auto copy_keys = [&](int cb, int ch, int t0) {
    const size_t bh = (size_t)cb * a.H + ch, g = (bh * (a.max_tokens / kGroupT) + t0 / kGroupT) * kD;
    fence_proxy_async_smem();
    mbar_arrive_expect_tx(bar_k, L::kKBytes);
    bulk_g2s(sm + L::kOffKc, a.k_codes + (bh * a.max_tokens + t0) * L::kKRow, kTile * L::kKRow, bar_k);
    bulk_g2s(sm + L::kOffKs, a.k_scale + g, L::kOffKz - L::kOffKs, bar_k);
    bulk_g2s(sm + L::kOffKz, a.k_zero + g, L::kOffVc - L::kOffKz, bar_k);
  };
  auto copy_values = [&](int cb, int ch, int t0) {
    const size_t tok = ((size_t)cb * a.H + ch) * a.max_tokens + t0;
    fence_proxy_async_smem();
    mbar_arrive_expect_tx(bar_v, L::kVBytes);
    bulk_g2s(sm + L::kOffVc, a.v_codes + tok * L::kVRow, kTile * L::kVRow, bar_v);
    bulk_g2s(sm + L::kOffVs, a.v_scale + tok * (kD / kGroupT), L::kOffVz - L::kOffVs, bar_v);
    bulk_g2s(sm + L::kOffVz, a.v_zero + tok * (kD / kGroupT), L::kOffMask - L::kOffVz, bar_v);
  };
  auto stored = [](const TreeLens& l, int tl) { return (tl + 1) * kTile <= l.nqv; };  // nqv <= nqk
  if (tid == 0) {
    mbar_init(bar_s, 1);
    mbar_init(bar_o, 1);
    mbar_init(bar_k, 1);
    mbar_init(bar_v, 1);
    *failed = 0;
    *nonfinite = 0;
    fence_mbar_init();
    if (stored(len, tile)) {
      copy_keys(b, seg / n_rt, tile * kTile);
      copy_values(b, seg / n_rt, tile * kTile);
    }
  }
  tmem_before();
  __syncthreads();
  tmem_after();
  const uint32_t tmem = *tmem_slot;
  const int quad = warp & 3, half = warp >> 2;            // TMEM lane quadrant, half of the rows
  const uint32_t t_lane = tmem + ((uint32_t)(32 * quad) << 16);
  constexpr int kHR = ROWS / 2;                            // rows a thread works on
  const int r0 = half * kHR;
  uint32_t phase = 0;    // of bar_s and bar_o: one completion each per tile
  uint32_t landed = 0;   // tiles that came through the stage: their parity is that of bar_k and bar_v
  float l[kHR];
  bool first = true;    // of the segment's tiles in this block
  int tile_first = 0;   // that tile
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!mbar_wait_bounded(bar, parity)) {
      *failed = 1;
      set_error(a.err, KVQ_ERR_TIMEOUT);
    }
  };

  for (long long p = p0; p < p1; ++p) {
    const int h = seg / n_rt, rt = seg % n_rt;
    const Token tk = {&a, len, (size_t)b * a.H + h, b, h};
    const int row0 = rt * ROWS;
    const int t0 = tile * kTile;
    const bool from_stage = stored(len, tile);
    // ---- the position after this one ----
    const bool last = tile + 1 == len.tiles;
    int nb = b, nseg = seg, ntile = tile + 1;
    TreeLens nlen = len;
    if (last) {
      ntile = 0;
      if (++nseg == seg_per_b) {
        nseg = 0;
        if (p + 1 < p1) {
          do nlen = tree_lens(a, ++nb);
          while (nlen.tiles == 0);  // a position is left, so such a request exists
        }
      }
    }
    const bool copy_next = p + 1 < p1 && stored(nlen, ntile);
    if (first) {
      // ---- the segment's query rows: fp16, each divided by a power of two that puts its largest
      //      magnitude in [2^14, 2^15); the masks and the running state ----
#pragma unroll
      for (int i = 0; i < kHR; ++i) l[i] = 0.f;
      for (int i = tid; i < ROWS * 8; i += kTreeThreads) {  // 8 lanes per row, 16 channels each
        const int r = i >> 3, c = i & 7, row = row0 + r, di = row / rep;
        uint4 u[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (row < rows_all && di < len.nd) {
          const uint4* src = reinterpret_cast<const uint4*>(
              a.q + (((size_t)b * a.N + di) * a.Hq + (size_t)h * rep + row % rep) * kD + 16 * c);
          u[0] = __ldg(src);
          u[1] = __ldg(src + 1);
        }
        const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
        float mx = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
#pragma unroll
        for (int off = 4; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
        const int ex = (int)(__float_as_uint(mx) >> 23);  // biased exponent; 0: zero or subnormal, 255: not finite
        // times 2^(14 - (ex - 127)) in two factors, since the power may pass the fp32 range
        const int sh = (ex == 0 || ex == 255) ? 0 : 141 - ex;
        const float f1 = __uint_as_float((uint32_t)(127 + sh / 2) << 23), f2 = __uint_as_float((uint32_t)(127 + sh - sh / 2) << 23);
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = pack_h2(bf16_lo(w[e]) * f1 * f2, bf16_hi(w[e]) * f1 * f2);
        uint4 x0, x1;
        pair_order<KB>(make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]), x0, x1);
        unsigned char* dst = sm + L::kOffQ + (r >> 3) * 2048 + c * 256 + (r & 7) * 16;
        *reinterpret_cast<uint4*>(dst) = x0;
        *reinterpret_cast<uint4*>(dst + 128) = x1;
        if (c == 0) {
          rowc[r] = scale_log2 / f1 / f2;
          rowm[r] = rowt[r] = -FLT_MAX;
          mask[r] = (row < rows_all && di < len.nd) ? a.mask[(size_t)b * a.N + di] : 0ull;
        }
      }
      if (tid == 0) *nonfinite = 0;
      tile_first = tile;
    }
    // ---- keys of the tile. A lane takes token lane % 8 of an octet and a code word (2 bits: 16 channels, 4
    //      bits: 8); a warp one key group and half of the words, so a lane unpacks four tokens per scale ----
    if (from_stage) {
      wait(bar_k, landed & 1);
      const int g = warp & 3, tok = 32 * g + (lane & 7);
      constexpr int kBlocks = (KB == 2) ? 1 : 2;   // of four words
#pragma unroll
      for (int blk = 0; blk < kBlocks; ++blk) {
        const int w = (warp >> 2) * 4 * kBlocks + 4 * blk + (lane >> 3);
        constexpr int kPairs = (KB == 2) ? 8 : 4;  // channel pairs of a word
        __half2 s[kPairs], nsz[kPairs];
        const uint4* sp = reinterpret_cast<const uint4*>(sm + L::kOffKs + (g * kD + 2 * kPairs * w) * 2);
        const uint4* zp = reinterpret_cast<const uint4*>(sm + L::kOffKz + (g * kD + 2 * kPairs * w) * 2);
        {
          uint4 s0, s1 = make_uint4(0u, 0u, 0u, 0u), z0, z1 = s1;
          if constexpr (KB == 2) {
            pair_order<2>(sp[0], sp[1], s0, s1);
            pair_order<2>(zp[0], zp[1], z0, z1);
          } else {
            uint4 none;
            pair_order<4>(sp[0], sp[0], s0, none);
            pair_order<4>(zp[0], zp[0], z0, none);
          }
          const uint32_t sw[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
          const uint32_t zw[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            s[j] = as_h2(sw[j]);
            nsz[j] = __hneg2(__hmul2(s[j], as_h2(zw[j])));
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = tok + 8 * i;
          const uint32_t u = *reinterpret_cast<const uint32_t*>(sm + L::kOffKc + t * L::kKRow + 4 * w);
          uint32_t o[kPairs];
#pragma unroll
          for (int j = 0; j < kPairs; ++j) o[j] = dequant_h2(code_h2<KB>(u, j), s[j], nsz[j]);
          unsigned char* dst = sm + L::kOffK + (t >> 3) * 2048 + w * (kPairs * 32) + (t & 7) * 16;
          *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
          if constexpr (KB == 2) *reinterpret_cast<uint4*>(dst + 128) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
    } else {
#pragma unroll 1
      for (int i = warp; i < 32; i += kTreeWarps) {
        const int t = 8 * (i >> 1) + (lane & 7), c = 4 * (i & 1) + (lane >> 3);  // 16 channels c
        uint4 x0, x1;
        pair_order<KB>(key8<KB>(tk, t0 + t, 2 * c), key8<KB>(tk, t0 + t, 2 * c + 1), x0, x1);
        unsigned char* dst = sm + L::kOffK + (t >> 3) * 2048 + c * 256 + (t & 7) * 16;
        *reinterpret_cast<uint4*>(dst) = x0;
        *reinterpret_cast<uint4*>(dst + 128) = x1;
      }
    }
    fence_proxy_async_smem();
    tmem_before();
    if (__syncthreads_or(*failed)) break;
    if (tid == 0) {
      tmem_after();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        umma_f16(tmem, tree_desc(smem_u32(sm + L::kOffK) + k * 256, 128, 2048),
                 tree_desc(smem_u32(sm + L::kOffQ) + k * 256, 128, 2048), tree_idesc(ROWS, false), k > 0);
      tree_commit(bar_s);
      if (copy_next) copy_keys(nb, nseg / n_rt, ntile * kTile);  // every thread has read this tile's
    }
    // ---- values of the tile, transposed. A thread takes a token octet and eight channels ----
    {
      const int c = lane & 15, oct = 2 * warp + (lane >> 4), flip = oct & 1;
      unsigned char* dst = sm + L::kOffV + c * kVRowGrp + oct * 128;
      if (from_stage) {
        wait(bar_v, landed & 1);
        uint32_t w[8];  // place i of the octet: token i ^ flip
        __half2 s[4], nsz[4];
        const unsigned char* cw = sm + L::kOffVc + 8 * oct * L::kVRow + ((VB == 2) ? (c >> 1) : c) * 4;
        const uint16_t* sp = reinterpret_cast<const uint16_t*>(sm + L::kOffVs) + 8 * oct * 4 + (c >> 2);
        const uint16_t* zp = reinterpret_cast<const uint16_t*>(sm + L::kOffVz) + 8 * oct * 4 + (c >> 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const uint32_t*>(cw + (i ^ flip) * L::kVRow);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ta = ((2 * i) ^ flip) * 4, tb = ((2 * i + 1) ^ flip) * 4;
          s[i] = as_h2(sp[ta] | ((uint32_t)sp[tb] << 16));
          nsz[i] = __hneg2(__hmul2(s[i], as_h2(zp[ta] | ((uint32_t)zp[tb] << 16))));
        }
        if constexpr (VB == 2) {
          const uint32_t sel = (c & 1) ? 0x7632u : 0x5410u;
          uint32_t x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = __byte_perm(w[2 * i], w[2 * i + 1], sel);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = dequant_h2(code_h2<2>(x[i], e), s[i], nsz[i]);
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
              for (int i = 0; i < 4; ++i) o[i] = dequant_h2(code_h2<4>(x[i], e), s[i], nsz[i]);
              *reinterpret_cast<uint4*>(dst + (4 * hw + e) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
        ++landed;
      } else {
        uint32_t x[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 u = value8<VB>(tk, t0 + 8 * oct + (i ^ flip), c, nonfinite);
          x[i][0] = u.x;
          x[i][1] = u.y;
          x[i][2] = u.z;
          x[i][3] = u.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = __byte_perm(x[2 * i][e >> 1], x[2 * i + 1][e >> 1], (e & 1) ? 0x7632 : 0x5410);
          *reinterpret_cast<uint4*>(dst + e * 16) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
    wait(bar_s, phase);
    tmem_after();
    // ---- weights: this thread's token against rows r0 .. r0 + kHR - 1. x = s c is rounded before the
    //      maximum is taken from it, so that the largest score's weight is exact however large it is ----
    const int tt = 32 * quad + lane, t = t0 + tt;
    float x[kHR];
    {
      uint32_t xr[kHR];
#pragma unroll
      for (int i = 0; i < kHR; i += 8) tmem_ld8(t_lane + r0 + i, xr + i);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < kHR; i += 4) {
        const float4 c4 = *reinterpret_cast<const float4*>(rowc + r0 + i);
        x[i] = __fmul_rn(__uint_as_float(xr[i]), c4.x);
        x[i + 1] = __fmul_rn(__uint_as_float(xr[i + 1]), c4.y);
        x[i + 2] = __fmul_rn(__uint_as_float(xr[i + 2]), c4.z);
        x[i + 3] = __fmul_rn(__uint_as_float(xr[i + 3]), c4.w);
      }
    }
    if (t0 + kTile > len.n) {  // drafted tokens in the tile, or none at all behind the last one
      const int dj = t - len.n;
      if (dj >= 0) {
#pragma unroll
        for (int i = 0; i < kHR; ++i)
          if (dj >= len.nd || !((mask[r0 + i] >> dj) & 1ull)) x[i] = -INFINITY;
      }
    }
    bool over = false;
#pragma unroll
    for (int i = 0; i < kHR; i += 4) {
      const float4 t4 = *reinterpret_cast<const float4*>(rowt + r0 + i);
      over = over || x[i] > t4.x || x[i + 1] > t4.y || x[i + 2] > t4.z || x[i + 3] > t4.w;
    }
    tmem_before();
    const bool raise = __syncthreads_or(over);
    if (tid == 0 && copy_next) copy_values(nb, nseg / n_rt, ntile * kTile);  // every thread has read this tile's
    if (raise) {
      // ---- raise the running maxima of the rows with a score past them ----
#pragma unroll
      for (int i = 0; i < kHR; ++i) {
        float mx = x[i];
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
        if (lane == 0) red[quad * ROWS + r0 + i] = mx;
      }
      __syncthreads();
      for (int r = tid; r < ROWS; r += kTreeThreads) {
        const float mt = fmaxf(fmaxf(red[r], red[ROWS + r]), fmaxf(red[2 * ROWS + r], red[3 * ROWS + r]));
        const bool up = mt > rowt[r];
        rowf[r] = up ? exp2_approx(rowm[r] - (mt - kRaise)) : 1.f;
        if (up) {
          rowm[r] = mt - kRaise;
          rowt[r] = mt + kSlack;
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kHR; ++i) l[i] *= rowf[r0 + i];
      if (!first) {  // O^T: the value product of the tile before is done (waited for below)
        tmem_after();
#pragma unroll
        for (int i = 0; i < kHR; i += 8) {
          uint32_t u[8];
          float o[8];
          tmem_ld8(t_lane + ROWS + r0 + i, u);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = __uint_as_float(u[e]) * rowf[r0 + i + e];
          tmem_st8(t_lane + ROWS + r0 + i, o);
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
        const float p0e = exp2_approx(x[i + e] - m4.x), p1e = exp2_approx(x[i + e + 1] - m4.y);
        const float p2e = exp2_approx(x[i + e + 2] - m4.z), p3e = exp2_approx(x[i + e + 3] - m4.w);
        l[i + e] += p0e;
        l[i + e + 1] += p1e;
        l[i + e + 2] += p2e;
        l[i + e + 3] += p3e;
        o[e / 2] = pack_h2(p0e, p1e);
        o[e / 2 + 1] = pack_h2(p2e, p3e);
      }
      *reinterpret_cast<uint4*>(sm + L::kOffK + ((r0 + i) >> 3) * 2048 + token_place(tt) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    fence_proxy_async_smem();
    tmem_before();
    __syncthreads();
    if (tid == 0) {
      tmem_after();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        umma_f16(tmem + ROWS, tree_desc(smem_u32(sm + L::kOffV) + k * 256, 128, kVRowGrp),
                 tree_desc(smem_u32(sm + L::kOffK) + k * 256, 128, 2048), tree_idesc(ROWS, true), !first || k > 0);
      tree_commit(bar_o);
    }
    wait(bar_o, phase);
    tmem_after();
    phase ^= 1;
    first = false;

    // ---- the segment ends here (or the share does): hand its sums on ----
    if (last || p + 1 == p1) {
      // l: over the tokens (lanes and quadrants)
#pragma unroll
      for (int i = 0; i < kHR; ++i) {
        float s = l[i];
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
        if (lane == 0) red[quad * ROWS + r0 + i] = s;
      }
      __syncthreads();
      const bool earlier = p - tile < p0;  // the segment began in an earlier block
      const bool whole = last && !earlier;
      float* slot = a.part + ((size_t)blockIdx.x * 2 + (earlier ? 0 : 1)) * slot_floats<ROWS>();
      const int ch = 32 * quad + lane;
      const bool fix = *nonfinite != 0;
#pragma unroll 1
      for (int i = 0; i < kHR; i += 8) {
        uint32_t u[8];
        tmem_ld8(t_lane + ROWS + r0 + i, u);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float o = __uint_as_float(u[e]);
          const int r = r0 + i + e, row = row0 + r, di = row / rep;
          if (row >= rows_all || di >= len.nd) continue;  // padding
          const float lt = red[r] + red[ROWS + r] + red[2 * ROWS + r] + red[3 * ROWS + r];
          if (fix) {  // of the drafted tokens in this block's tiles
            const int j1 = min(len.nd, (tile + 1) * kTile - len.n);
            for (int j = max(0, tile_first * kTile - len.n); j < j1; ++j) {
              if (!((mask[r] >> j) & 1ull)) continue;
              const uint16_t v = a.v_draft[(((size_t)b * a.N + j) * a.H + h) * kD + ch];
              if ((v & 0x7C00u) == 0x7C00u) o += th2f(v);
            }
          }
          if (whole) {
            const size_t at = (((size_t)b * a.N + di) * a.Hq + (size_t)h * rep + row % rep) * kD + ch;
            const float val = lt > 0.f || lt != lt ? o / lt : 0.f;
            if (a.out_fp32) reinterpret_cast<float*>(a.out)[at] = val;
            else reinterpret_cast<uint16_t*>(a.out)[at] = f32_to_bf16(val);
          } else {
            slot[(size_t)r * kD + ch] = o;
            if (ch == 0) {
              slot[(size_t)ROWS * kD + r] = rowm[r];
              slot[(size_t)ROWS * kD + ROWS + r] = lt;
            }
          }
        }
      }
      tmem_before();
      __syncthreads();  // the row state is read before the next segment resets it
      first = true;
    }
    b = nb;
    seg = nseg;
    tile = ntile;
    len = nlen;
  }
  // a wait that ran out leaves the loop at the next barrier: let this block's copies land first
  if (tid == 0 && *failed) {
    mbar_wait_bounded(bar_k, landed & 1);
    mbar_wait_bounded(bar_v, landed & 1);
  }
  tmem_before();
  __syncthreads();
  if (warp == 0) {
    tmem_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kCols) : "memory");
  }
}

// Joins the partials of the segments that several blocks shared, in block order: a warp takes a
// row, a lane four channels.
constexpr int kMergeThreads = 128;
template <int ROWS>
__global__ void __launch_bounds__(kMergeThreads) kivi_tree_merge_kernel(const KiviTreeArgs a, const int G) {
  __shared__ long long part[2][kMergeThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rep = a.Hq / a.H, rows_all = a.N * rep, n_rt = (rows_all + ROWS - 1) / ROWS, seg_per_b = a.H * n_rt;
  const int per_seg = ROWS / (kMergeThreads / 32);
  const int sg = blockIdx.x / per_seg;
  const int b = sg / seg_per_b, seg = sg % seg_per_b, h = seg / n_rt, rt = seg % n_rt;
  const int r = (int)(blockIdx.x % per_seg) * (kMergeThreads / 32) + warp, row = rt * ROWS + r, di = row / rep;
  long long all = 0, pre = 0;
  for (int i = tid; i < a.B; i += kMergeThreads) {
    const int t = tree_lens(a, i).tiles;
    all += t;
    if (i < b) pre += t;
  }
  part[0][tid] = all;
  part[1][tid] = pre;
  __syncthreads();
  all = pre = 0;
  for (int i = 0; i < min(a.B, kMergeThreads); ++i) {
    all += part[0][i];
    pre += part[1][i];
  }
  const TreeLens len = tree_lens(a, b);
  if (len.tiles == 0 || row >= rows_all || di >= len.nd) return;
  const long long P = all * seg_per_b, s0 = pre * seg_per_b + (long long)seg * len.tiles, s1 = s0 + len.tiles;
  const int k0 = share_of(P, s0, G), k1 = share_of(P, s1 - 1, G);
  if (k0 == k1) return;  // one block wrote the output
  auto slot = [&](int k) {  // a segment that began in an earlier block is in a block's first slot
    return a.part + ((size_t)k * 2 + (share_begin(P, k, G) > s0 ? 0 : 1)) * slot_floats<ROWS>();
  };
  float M = -FLT_MAX;
  for (int k = k0; k <= k1; ++k)
    if (share_begin(P, k, G) < share_begin(P, k + 1, G)) M = fmaxf(M, slot(k)[(size_t)ROWS * kD + r]);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float lt = 0.f;
  for (int k = k0; k <= k1; ++k) {
    if (share_begin(P, k, G) == share_begin(P, k + 1, G)) continue;  // an empty share
    const float* s = slot(k);
    const float lk = s[(size_t)ROWS * kD + ROWS + r];
    if (lk == 0.f) continue;  // the row saw nothing there
    const float w = exp2f(s[(size_t)ROWS * kD + r] - M);
    const float4 v = *reinterpret_cast<const float4*>(s + (size_t)r * kD + 4 * lane);
    lt = fmaf(w, lk, lt);
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  }
  const bool none = !(lt > 0.f || lt != lt);
  const size_t at = (((size_t)b * a.N + di) * a.Hq + (size_t)h * rep + row % rep) * kD + 4 * lane;
  float val[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) val[e] = none ? 0.f : val[e] / lt;
  if (a.out_fp32) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = make_float4(val[0], val[1], val[2], val[3]);
  } else {
    uint2 w;
    w.x = f32_to_bf16(val[0]) | ((uint32_t)f32_to_bf16(val[1]) << 16);
    w.y = f32_to_bf16(val[2]) | ((uint32_t)f32_to_bf16(val[3]) << 16);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at) = w;
  }
}

// rows of a tile: the smallest that holds a KV head's, 64 at most
int tree_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }
int tree_blocks() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return 2 * sms;
}

template <int KB, int VB, int ROWS>
cudaError_t launch_tree(const KiviTreeArgs& a, cudaStream_t st) {
  using L = TreeLayout<KB, VB, ROWS>;
  cudaError_t e = cudaFuncSetAttribute(kivi_tree_kernel<KB, VB, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  const int G = tree_blocks();
  kivi_tree_kernel<KB, VB, ROWS><<<G, kTreeThreads, L::kSmem, st>>>(a, 1.4426950408889634f / sqrtf((float)kD));
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const long long segs = (long long)a.B * a.H * ((a.N * (a.Hq / a.H) + ROWS - 1) / ROWS);
  kivi_tree_merge_kernel<ROWS><<<(unsigned)(segs * (ROWS / (kMergeThreads / 32))), kMergeThreads, 0, st>>>(a, G);
  return cudaGetLastError();
}
template <int KB, int VB>
cudaError_t launch_tree_rows(const KiviTreeArgs& a, cudaStream_t st) {
  const int r = tree_rows(a.N * (a.Hq / a.H));
  if (r == 16) return launch_tree<KB, VB, 16>(a, st);
  if (r == 32) return launch_tree<KB, VB, 32>(a, st);
  return launch_tree<KB, VB, 64>(a, st);
}

}  // namespace

size_t kivi_tree_ws_bytes(int B, int N, int H, int Hq, int k_bits, int v_bits) {
  const int r = tree_rows(N * (Hq / H));
  return (size_t)tree_blocks() * 2 * r * (kD + 2) * sizeof(float);
}

cudaError_t launch_kivi_tree(const KiviTreeArgs& a, cudaStream_t st) {
  if (a.k_bits == 2 && a.v_bits == 2) return launch_tree_rows<2, 2>(a, st);
  if (a.k_bits == 2) return launch_tree_rows<2, 4>(a, st);
  if (a.v_bits == 2) return launch_tree_rows<4, 2>(a, st);
  return launch_tree_rows<4, 4>(a, st);
}

}  // namespace kvq
