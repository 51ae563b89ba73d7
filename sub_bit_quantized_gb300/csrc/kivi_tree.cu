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

#include <algorithm>

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

// V^T is staged in 8 channel x 8 token core matrices; those of consecutive token octets are 144
// bytes apart so that eight threads with eight octets store to different banks
constexpr int kVOct = 144;
constexpr int kVRowGrp = (kTile / 8) * kVOct;

template <int ROWS>
struct TreeLayout {
  static constexpr int kOffQ = 0;                                  // fp16 [ROWS x 128], K-major
  static constexpr int kOffK = kOffQ + ROWS * kD * 2;              // fp16 [128 tokens x 128], K-major; then P
  static constexpr int kOffV = kOffK + kTile * kD * 2;             // fp16 [128 channels x 128 tokens], K-major
  static constexpr int kOffMask = kOffV + (kD / 8) * kVRowGrp;     // uint64 [ROWS]
  static constexpr int kOffC = kOffMask + ROWS * 8;                // float [ROWS]: log2 units per score unit
  static constexpr int kOffM = kOffC + ROWS * 4;                   // float [ROWS]: running maximum (log2)
  static constexpr int kOffF = kOffM + ROWS * 4;                   // float [ROWS]: rescale factor
  static constexpr int kOffRed = kOffF + ROWS * 4;                 // float [4][ROWS]: per lane quadrant
  static constexpr int kOffBar = kOffRed + 4 * ROWS * 4;           // mbarriers, TMEM address, flags
  static constexpr int kSmem = kOffBar + 64;
  static constexpr uint32_t kCols = 2 * ROWS < 32 ? 32 : 2 * ROWS;  // TMEM: S^T, O^T
  static_assert(ROWS * 256 <= kTile * kD * 2, "P fits in the key tile");
  static_assert(kSmem <= 232448, "shared memory");
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

template <int KB, int VB, int ROWS>
__global__ void __launch_bounds__(kTreeThreads, 2) kivi_tree_kernel(const KiviTreeArgs a, const float scale_log2) {
  using L = TreeLayout<ROWS>;
  extern __shared__ __align__(128) unsigned char sm[];
  uint64_t* mask = reinterpret_cast<uint64_t*>(sm + L::kOffMask);
  float* rowc = reinterpret_cast<float*>(sm + L::kOffC);
  float* rowm = reinterpret_cast<float*>(sm + L::kOffM);
  float* rowf = reinterpret_cast<float*>(sm + L::kOffF);
  float* red = reinterpret_cast<float*>(sm + L::kOffRed);
  uint64_t* bar_s = reinterpret_cast<uint64_t*>(sm + L::kOffBar);  // scores done
  uint64_t* bar_o = bar_s + 1;                                      // value product done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_o + 1);
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
  if (tid == 0) {
    mbar_init(bar_s, 1);
    mbar_init(bar_o, 1);
    *failed = 0;
    *nonfinite = 0;
    fence_mbar_init();
  }
  tmem_before();
  __syncthreads();
  tmem_after();
  const uint32_t tmem = *tmem_slot;
  const int quad = warp & 3, half = warp >> 2;            // TMEM lane quadrant, half of the rows
  const uint32_t t_lane = tmem + ((uint32_t)(32 * quad) << 16);
  constexpr int kHR = ROWS / 2;                            // rows a thread works on
  const int r0 = half * kHR;
  uint32_t phase = 0;   // of both barriers: one completion each per tile
  float l[kHR];
  bool first = true;    // of the segment's tiles in this block
  int tile_first = 0;   // that tile

  for (long long p = p0; p < p1; ++p) {
    const int h = seg / n_rt, rt = seg % n_rt;
    const Token tk = {&a, len, (size_t)b * a.H + h, b, h};
    const int row0 = rt * ROWS;
    if (first) {
      // ---- the segment's query rows: fp16, each divided by a power of two that puts its largest
      //      magnitude in [2^14, 2^15); the masks and the running state ----
#pragma unroll
      for (int i = 0; i < kHR; ++i) l[i] = 0.f;
      for (int i = tid; i < ROWS * 16; i += kTreeThreads) {  // 16 lanes per row
        const int r = i >> 4, c = i & 15, row = row0 + r, di = row / rep;
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows_all && di < len.nd)
          u = __ldg(reinterpret_cast<const uint4*>(a.q + (((size_t)b * a.N + di) * a.Hq + (size_t)h * rep + row % rep) * kD + 8 * c));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        float mx = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
        const int ex = (int)(__float_as_uint(mx) >> 23);  // biased exponent; 0: zero or subnormal, 255: not finite
        // times 2^(14 - (ex - 127)) in two factors, since the power may pass the fp32 range
        const int sh = (ex == 0 || ex == 255) ? 0 : 141 - ex;
        const float f1 = __uint_as_float((uint32_t)(127 + sh / 2) << 23), f2 = __uint_as_float((uint32_t)(127 + sh - sh / 2) << 23);
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack_h2(bf16_lo(w[e]) * f1 * f2, bf16_hi(w[e]) * f1 * f2);
        *reinterpret_cast<uint4*>(sm + L::kOffQ + (r >> 3) * 2048 + c * 128 + (r & 7) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
        if (c == 0) {
          rowc[r] = scale_log2 / f1 / f2;
          rowm[r] = -INFINITY;
          mask[r] = (row < rows_all && di < len.nd) ? a.mask[(size_t)b * a.N + di] : 0ull;
        }
      }
      if (tid == 0) *nonfinite = 0;
      tile_first = tile;
    }
    const int t0 = tile * kTile;
    // ---- keys of the tile: thread (token, 16-byte chunk), eight tokens x four chunks a warp step ----
#pragma unroll 2
    for (int i = warp; i < 64; i += kTreeWarps) {
      const int t = 8 * (i >> 2) + (lane & 7), c = 4 * (i & 3) + (lane >> 3);
      *reinterpret_cast<uint4*>(sm + L::kOffK + (t >> 3) * 2048 + c * 128 + (t & 7) * 16) = key8<KB>(tk, t0 + t, c);
    }
    fence_proxy_async_smem();
    tmem_before();
    __syncthreads();
    if (tid == 0) {
      tmem_after();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        umma_f16(tmem, tree_desc(smem_u32(sm + L::kOffK) + k * 256, 128, 2048),
                 tree_desc(smem_u32(sm + L::kOffQ) + k * 256, 128, 2048), tree_idesc(ROWS, false), k > 0);
      tree_commit(bar_s);
    }
    // ---- values of the tile, transposed: thread (token octet, eight channels) ----
    {
      const int oct = lane & 15, c = 2 * warp + (lane >> 4);
      uint32_t x[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 u = value8<VB>(tk, t0 + 8 * oct + i, c, nonfinite);
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
        *reinterpret_cast<uint4*>(sm + L::kOffV + c * kVRowGrp + oct * kVOct + e * 16) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    if (!mbar_wait_bounded(bar_s, phase)) {
      *failed = 1;
      set_error(a.err, KVQ_ERR_TIMEOUT);
    }
    tmem_after();
    // ---- weights: this thread's token against rows r0 .. r0 + kHR - 1 ----
    const int t = t0 + 32 * quad + lane;
    const bool cached = t < len.n;
    const int dj = t - len.n;  // drafted token
    uint32_t xr[kHR];
#pragma unroll
    for (int i = 0; i < kHR; i += 8) tmem_ld8(t_lane + r0 + i, xr + i);
    tmem_wait_ld();
    float x[kHR];
    bool over = false;
#pragma unroll
    for (int i = 0; i < kHR; ++i) {
      const bool seen = cached || (dj < len.nd && ((mask[r0 + i] >> dj) & 1ull));
      x[i] = seen ? __uint_as_float(xr[i]) * rowc[r0 + i] : -INFINITY;
      over = over || (x[i] > rowm[r0 + i] + kSlack);
    }
    tmem_before();
    if (__syncthreads_or(over)) {
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
        const float mo = rowm[r];
        const float mt = fmaxf(fmaxf(red[r], red[ROWS + r]), fmaxf(red[2 * ROWS + r], red[3 * ROWS + r]));
        const bool up = mt > mo + kSlack;
        rowm[r] = up ? mt : mo;
        rowf[r] = !up ? 1.f : (mo == -INFINITY) ? 0.f : exp2f(mo - mt);
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
      for (int e = 0; e < 8; e += 2) {
        float pe[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const float xe = x[i + e + f];  // NaN stays NaN
          pe[f] = (xe == -INFINITY) ? 0.f : exp2f(xe - rowm[r0 + i + e + f] + kRaise);
          l[i + e + f] += pe[f];
        }
        o[e / 2] = pack_h2(pe[0], pe[1]);
      }
      *reinterpret_cast<uint4*>(sm + L::kOffK + ((r0 + i) >> 3) * 2048 + (32 * quad + lane) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    fence_proxy_async_smem();
    tmem_before();
    __syncthreads();
    if (tid == 0) {
      tmem_after();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        umma_f16(tmem + ROWS, tree_desc(smem_u32(sm + L::kOffV) + k * 2 * kVOct, kVOct, kVRowGrp),
                 tree_desc(smem_u32(sm + L::kOffK) + k * 256, 128, 2048), tree_idesc(ROWS, true), !first || k > 0);
      tree_commit(bar_o);
    }
    if (!mbar_wait_bounded(bar_o, phase)) {
      *failed = 1;
      set_error(a.err, KVQ_ERR_TIMEOUT);
    }
    tmem_after();
    phase ^= 1;
    first = false;

    // ---- the segment ends here (or the share does): hand its sums on ----
    const bool last = tile + 1 == len.tiles;
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
    if (__syncthreads_or(*failed)) break;
    if (last) {
      tile = 0;
      if (++seg == seg_per_b) {
        seg = 0;
        if (p + 1 < p1) {
          do len = tree_lens(a, ++b);
          while (len.tiles == 0);  // a position is left, so such a request exists
        }
      }
    } else {
      ++tile;
    }
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
  float M = -INFINITY;
  for (int k = k0; k <= k1; ++k)
    if (share_begin(P, k, G) < share_begin(P, k + 1, G)) M = fmaxf(M, slot(k)[(size_t)ROWS * kD + r]);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float lt = 0.f;
  for (int k = k0; k <= k1; ++k) {
    if (share_begin(P, k, G) == share_begin(P, k + 1, G)) continue;  // an empty share
    const float* s = slot(k);
    const float lk = s[(size_t)ROWS * kD + ROWS + r];
    if (lk == 0.f) continue;  // the row saw nothing there
    const float w = (M == -INFINITY) ? 1.f : exp2f(s[(size_t)ROWS * kD + r] - M);
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
  using L = TreeLayout<ROWS>;
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
