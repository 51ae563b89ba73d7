// What the attention kernels over a KIVI cache with many query rows share (kivi_tree.cu, kivi_prefix.cu): the lengths
// of a request, query rows and codes as fp16, and the tcgen05 instructions.
#pragma once

#include <cuda_fp16.h>

#include "kvq_common.cuh"
#include "kvq_internal.h"

namespace kvq {

// The end of a kernel that was launched early behind one that it does not depend on: what comes next waits for this
// kernel alone, so it does not end before the other. (All blocks of that one run: otherwise this would not have begun.)
__device__ __forceinline__ void end_behind(const KiviTreeArgs& a) {
  if (a.chained == kChainedBehind && blockIdx.x == 0) wait_behind();
}

constexpr int kGroupT = 32;   // tokens per key group, channels per value group
// A row's weights are exp2(x - m + kRaise), m its running maximum, which moves when a score passes it by kSlack (log2):
// weights stay below 2^15 and are held as fp16, where one below 2^-30 of the maximum's is lost (2^-25 without kRaise).
// Raising costs a pass over the sums; at a slack of 7 the peaked scores of outlier channels raise some row of a tile
// of 64 in most of a segment's first tiles.
constexpr float kSlack = 10.f, kRaise = 5.f;

__device__ __forceinline__ float th2f(uint32_t b) { return __half2float(__ushort_as_half((unsigned short)b)); }
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

struct TreeLens {
  int nqk, nqv, n, nd;  // quantized keys, quantized values, cached tokens, drafted tokens that rows may attend
  int tiles, nr;        // tiles; tokens whose rows attend (nd, or without drafts the queries')
};
__device__ __forceinline__ TreeLens tree_lens(const KiviTreeArgs& a, int b, int tile) {
  TreeLens L;
  L.nqk = min(max(a.n_quant_k[b], 0), a.max_tokens) & -kGroupT;
  L.n = L.nqk + max(0, min(a.n_tok[b] - L.nqk, a.residual));
  // at least n - residual, as in every valid state: the ring holds no more values
  L.nqv = (a.residual > 0) ? min(max(a.n_quant_v[b], max(L.n - a.residual, 0)), L.nqk) : L.nqk;
  L.nr = a.n_draft ? min(max(a.n_draft[b], 0), a.N) : a.N;
  L.nd = a.mask ? L.nr : 0;
  L.tiles = L.nr > 0 ? max((int)((uint32_t)(L.n + L.nd + tile - 1) / tile), 1) : 0;
  return L;
}
// where the share of block k of G begins, without leaving 32 bits (k <= G, G far below 2^15)
__device__ __forceinline__ int share_begin(int P, int k, const IntDiv& G) {
  if (P <= G.d) return min(k, P);
  const int q = div_by(P, G);
  return k * q + div_by(k * (P - q * G.d), G);
}

// The row of a token behind the quantized ones (token t, value: of the ring): residual, drafted, or none. By selection: where
// many are loaded in a row, a branch between two of them would keep the second from starting before the first arrives.
__device__ __forceinline__ const uint16_t* fp16_row(const KiviTreeArgs& a, const TreeLens& L, int b, int h, int t, int place,
                                                    const uint16_t* resid, const uint16_t* draft) {
  const size_t r = ((size_t)b * a.H + h) * a.residual + place, d = ((size_t)b * a.N + (t - L.n)) * a.H + h;
  const uint16_t* from = t < L.n ? resid : draft;
  const size_t at = t < L.n ? r : d;
  return t < L.n + L.nd ? from + at * kD : nullptr;
}
__device__ __forceinline__ const uint16_t* fp16_key(const KiviTreeArgs& a, const TreeLens& L, int b, int h, int t) {
  return fp16_row(a, L, b, h, t, t - L.nqk, a.k_resid, a.k_draft);
}
// place: t % residual for a token that is cached
__device__ __forceinline__ const uint16_t* fp16_value(const KiviTreeArgs& a, const TreeLens& L, int b, int h, int t, int place) {
  return fp16_row(a, L, b, h, t, place, a.v_resid, a.v_draft);
}
// place of token t0 + i (i < 32) when t0's is p: the ring holds at least 32 rows, or none (no token is there then)
__device__ __forceinline__ int ring_place(int p, int i, int R) {
  p += i;
  if (p >= R) p -= R;
  return p;
}
// channels 8c .. 8c+7 of a row, zero without one: a load under a predicate, as branches around several of them would keep
// each from starting before the one ahead has arrived
__device__ __forceinline__ uint4 row8(const uint16_t* p, int c) {
  const uint64_t at = p ? reinterpret_cast<uint64_t>(p + 8 * c) : 0;
  uint4 v;
  asm("{\n\t.reg .pred there;\n\t"
      "setp.ne.u64 there, %4, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@there ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(at));
  return v;
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
  const bool real = row < a.N * a.rep.d && di < len.nr;
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

// 32 consecutive fp32 columns of this thread's TMEM lane (valid after tmem_wait_ld)
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Products of a warp that walks together, of which one lane issues: operands stay in uniform registers. Descriptors in
// two words, the upper one a constant.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t desc_lo(const void* p, uint32_t lbo) {
  return __shfl_sync(0xFFFFFFFFu, ((smem_u32(p) & 0x3FFFFu) >> 4) | (lbo >> 4) << 16, 0);
}
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | 1u << 14; }
template <uint32_t AHI, uint32_t BHI, uint32_t IDESC>
__device__ __forceinline__ void umma_lo(uint32_t leader, uint32_t d_tmem, uint32_t alo, uint32_t blo, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "mov.b64 x, {%1, %5};\n\t"
      "mov.b64 y, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %7, p;\n\t}" ::"r"(d_tmem),
      "r"(alo), "r"(blo), "r"(accumulate), "r"(leader), "n"(AHI), "n"(BHI), "n"(IDESC)
      : "memory");
}
// A in TMEM: a lane a row, a column two elements of K
template <uint32_t BHI, uint32_t IDESC>
__device__ __forceinline__ void umma_lo_ta(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint32_t blo, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %6, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(blo), "r"(accumulate), "r"(leader), "n"(BHI), "n"(IDESC)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}

// the largest of the lanes' values that are numbers
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(x));
  return r;
}

}  // namespace kvq
