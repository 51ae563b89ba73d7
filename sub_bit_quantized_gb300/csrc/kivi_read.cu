// Reading a KIVI cache back: keys and values of cached tokens in fp16, bf16 or fp32.
//
// Token t of request b is X = s (q - z) from the codes when t < n_quant_k (keys) or
// t < n_quant_v (values), else its fp16 residual row; q - z and the product are fp32, the
// output is rounded once.
//
// Bound: HBM, mostly the writes (a 2-bit token and head reads 96 bytes and writes 512 in fp16).
// Sixteen lanes share a token, lane c holding channels 8c .. 8c+7, so a warp stores two whole
// rows at a time; a warp takes 32 consecutive tokens of one head, keys or values.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_common.cuh"
#include "kvq_internal.h"
#include "../../include/kvq.h"

namespace kvq {
namespace {

constexpr int kReadThreads = 256;
constexpr int kReadTok = 32;  // tokens of a warp

__device__ __forceinline__ void half8(const uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// the codes of channels 8c .. 8c+7 of a token row
template <int BITS>
__device__ __forceinline__ uint32_t load_codes8(const uint8_t* row, int c) {
  if constexpr (BITS == 2) return __ldg(reinterpret_cast<const uint16_t*>(row) + c);
  else return __ldg(reinterpret_cast<const uint32_t*>(row) + c);
}
// code i of the eight as a float: masked in under the exponent of 2^23, which is then subtracted (exact)
template <int BITS>
__device__ __forceinline__ float code_f(uint32_t w, int i) {
  return __uint_as_float(((w >> (BITS * i)) & ((1u << BITS) - 1u)) | 0x4B000000u) - 8388608.f;
}

template <int OUT>
__device__ __forceinline__ void store_row8(void* base, int64_t elem, const float (&v)[8]) {
  if constexpr (OUT == KVQ_DT_FP32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + elem);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (OUT == KVQ_DT_BF16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + elem) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// BITS: of the codes read; kKeys: scales per (32-token group, channel), else per (token, 32-channel group)
template <int BITS, bool kKeys, int OUT>
__device__ __forceinline__ void read_rows(const KiviReadArgs& a, int b, int h, int j0, int lane) {
  constexpr int kRow = kD * BITS / 8, kGroup = 32;
  const int c = lane & 15;
  const int R = a.residual;
  const int nqk = min(max(a.n_quant_k[b], 0), a.max_tokens) / kGroup * kGroup;
  const int n = nqk + max(0, min(a.n_tok[b] - nqk, R));
  const int nq = kKeys ? nqk : (R > 0) ? min(max(a.n_quant_v[b], 0), nqk) : nqk;
  const int first = a.tok_begin ? a.tok_begin[b - a.b0] : 0;
  const size_t bh = (size_t)b * a.H + h;
  const uint8_t* codes = (kKeys ? a.k_codes : a.v_codes) + bh * a.max_tokens * kRow;
  const uint16_t* scale = kKeys ? a.k_scale + bh * (a.max_tokens / kGroup) * kD : a.v_scale + bh * a.max_tokens * (kD / kGroup);
  const uint16_t* zero = kKeys ? a.k_zero + bh * (a.max_tokens / kGroup) * kD : a.v_zero + bh * a.max_tokens * (kD / kGroup);
  const uint16_t* resid = (kKeys ? a.k_resid : a.v_resid) + bh * R * kD;
  void* out = kKeys ? a.k_out : a.v_out;
  const int64_t o = (int64_t)(b - a.b0) * a.sb + (int64_t)h * a.sh + 8 * c;
#pragma unroll 4
  for (int i = lane >> 4; i < kReadTok; i += 2) {
    const int j = j0 + i;
    const long long tl = (long long)first + j;
    if (j >= a.n_tok_out || tl < 0 || tl >= n) continue;
    const int t = (int)tl;
    float v[8];
    if (t < nq) {
      const uint32_t w = load_codes8<BITS>(codes + (size_t)t * kRow, c);
      if constexpr (kKeys) {
        float s[8], z[8];
        half8(__ldg(reinterpret_cast<const uint4*>(scale + (size_t)(t / kGroup) * kD + 8 * c)), s);
        half8(__ldg(reinterpret_cast<const uint4*>(zero + (size_t)(t / kGroup) * kD + 8 * c)), z);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = s[e] * (code_f<BITS>(w, e) - z[e]);
      } else {
        const float s = __half2float(__ushort_as_half(__ldg(scale + (size_t)t * (kD / kGroup) + c / 4)));
        const float z = __half2float(__ushort_as_half(__ldg(zero + (size_t)t * (kD / kGroup) + c / 4)));
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = s * (code_f<BITS>(w, e) - z);
      }
    } else {
      const int row = kKeys ? t - nqk : t % R;
      half8(__ldg(reinterpret_cast<const uint4*>(resid + (size_t)row * kD + 8 * c)), v);
    }
    store_row8<OUT>(out, o + (int64_t)j * kD, v);
  }
}

template <int OUT>
__global__ void __launch_bounds__(kReadThreads) kivi_read_kernel(const KiviReadArgs a) {
  const int lane = threadIdx.x & 31;
  const int chunks = (a.n_tok_out - 1) / kReadTok + 1, both = (a.k_out ? 1 : 0) + (a.v_out ? 1 : 0);
  const long long unit = (long long)blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5);
  if (unit >= (long long)a.B * a.H * chunks * both) return;
  const long long row = unit / chunks;  // (b, h, keys or values)
  const int j0 = (int)(unit - row * chunks) * kReadTok;
  const bool keys = a.k_out && (both == 1 || (row & 1) == 0);
  const long long bh = row / both;
  const int b = a.b0 + (int)(bh / a.H), h = (int)(bh % a.H);
  if (keys) {
    if (a.k_bits == 2) read_rows<2, true, OUT>(a, b, h, j0, lane);
    else read_rows<4, true, OUT>(a, b, h, j0, lane);
  } else {
    if (a.v_bits == 2) read_rows<2, false, OUT>(a, b, h, j0, lane);
    else read_rows<4, false, OUT>(a, b, h, j0, lane);
  }
}

}  // namespace

cudaError_t launch_kivi_read(const KiviReadArgs& a, int out_dt, cudaStream_t s) {
  const long long chunks = (a.n_tok_out - 1) / kReadTok + 1;
  const long long units = (long long)a.B * a.H * chunks * ((a.k_out ? 1 : 0) + (a.v_out ? 1 : 0));
  const long long blocks = (units + kReadThreads / 32 - 1) / (kReadThreads / 32);
  const unsigned g = (unsigned)blocks;  // below 2^31 (checked by the host)
  if (out_dt == KVQ_DT_FP32) kivi_read_kernel<KVQ_DT_FP32><<<g, kReadThreads, 0, s>>>(a);
  else if (out_dt == KVQ_DT_FP16) kivi_read_kernel<KVQ_DT_FP16><<<g, kReadThreads, 0, s>>>(a);
  else kivi_read_kernel<KVQ_DT_BF16><<<g, kReadThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
