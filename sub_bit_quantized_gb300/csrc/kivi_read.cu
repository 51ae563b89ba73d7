// Reading a KIVI cache back: keys and values of cached tokens in fp16, bf16 or fp32.
//
// Token t of request b is X = s (q - z) from the codes when t < n_quant_k (keys) or
// t < n_quant_v (values), else its fp16 residual row; q - z and the product are fp32, the
// output is rounded once.
//
// Bound: HBM, mostly the writes (a 2-bit token and head reads 96 bytes and writes 512 in fp16).
// Sixteen lanes share a token, so a warp stores two whole rows at a time; a warp takes the 32
// tokens of a key group of one head, keys or values, eight of a lane's loads in flight at once.
// Measured (calls back to back): 16 requests, 32 heads, 4K tokens at 2 bits into fp16 (1.14 GB) 174 to 180 us, 6.4 TB/s,
// 95 % of the copy rate; 3 requests, 8 heads, 20011 tokens at 4 bits into fp32 (498 MB) 86 to 90 us, 5.7 TB/s,
// 84 %. The first form, without the loads in flight together, took 265 and 102 us. Stores that are
// the first to leave L2 change nothing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_common.cuh"
#include "kvq_internal.h"
#include "../../include/kvq.h"

namespace kvq {
namespace {

// Threads of a block: small blocks leave their places sooner, which pays when a warp writes 16 KB (fp32: 3 requests, 8
// heads, 20011 tokens, 4 bits 87.7 us with 64, 90.1 with 256; 64 requests, 32 heads, 160 tokens 77.5 and 82.6) and does
// not when it writes 8 (fp16: 54.2 and 53.7; 53.1 and 51.6).
constexpr int read_threads(int out) { return out == KVQ_DT_FP32 ? 64 : 256; }
constexpr int kGroup = 32;     // tokens per key group, channels per value group; tokens of a warp

// A lane's eight channels of a token are two quads: channels 8c .. 8c+7 for 16-bit outputs, so that a lane stores
// 16 bytes; channels 4c .. 4c+3 and 64 + 4c .. for fp32, so that 16 lanes store 256 contiguous bytes at a time.
template <int OUT>
__device__ __forceinline__ int quad_ch(int c, int q) { return OUT == KVQ_DT_FP32 ? 64 * q + 4 * c : 8 * c + 4 * q; }

__device__ __forceinline__ void half4(const uint2 u, float2& x, float2& y) {
  x = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
  y = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
}
// the lane's eight fp16 values of a row
template <int OUT>
__device__ __forceinline__ uint4 load_half8(const uint16_t* row, int c) {
  if constexpr (OUT == KVQ_DT_FP32) {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(row + quad_ch<OUT>(c, 0)));
    const uint2 b = __ldg(reinterpret_cast<const uint2*>(row + quad_ch<OUT>(c, 1)));
    return make_uint4(a.x, a.y, b.x, b.y);
  } else {
    return __ldg(reinterpret_cast<const uint4*>(row + 8 * c));
  }
}
__device__ __forceinline__ void half8(const uint4 u, float2 (&v)[4]) {
  half4(make_uint2(u.x, u.y), v[0], v[1]);
  half4(make_uint2(u.z, u.w), v[2], v[3]);
}
// the codes of the lane's eight channels of a token row, in the order of the channels
template <int BITS, int OUT>
__device__ __forceinline__ uint32_t load_codes8(const uint8_t* row, int c) {
  if constexpr (OUT == KVQ_DT_FP32) {
    if constexpr (BITS == 2) return __ldg(row + c) | ((uint32_t)__ldg(row + 16 + c) << 8);
    else return __ldg(reinterpret_cast<const uint16_t*>(row) + c) | ((uint32_t)__ldg(reinterpret_cast<const uint16_t*>(row) + 16 + c) << 16);
  } else {
    if constexpr (BITS == 2) return __ldg(reinterpret_cast<const uint16_t*>(row) + c);
    else return __ldg(reinterpret_cast<const uint32_t*>(row) + c);
  }
}
// The eight codes minus z, times s: each code is masked in place under the exponent of 2^23, where it stands for
// 2^23 + c 2^(b i); the 2^23 comes off exactly, one FMA gives c - z and one product s (c - z).
template <int BITS>
__device__ __forceinline__ void dequant8(uint32_t w, const float2 (&s)[4], const float2 (&nz)[4], float2 (&v)[4]) {
  const float2 big = make_float2(-8388608.f, -8388608.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    constexpr int kIn = (BITS == 2) ? 8 : 4;  // codes below the exponent
    const int i0 = 2 * i, i1 = 2 * i + 1;
    const uint32_t u0 = i0 < kIn ? w : w >> (BITS * kIn), u1 = i1 < kIn ? w : w >> (BITS * kIn);
    const uint32_t m0 = ((1u << BITS) - 1u) << (BITS * (i0 % kIn)), m1 = ((1u << BITS) - 1u) << (BITS * (i1 % kIn));
    float2 f = make_float2(__uint_as_float((u0 & m0) | 0x4B000000u), __uint_as_float((u1 & m1) | 0x4B000000u));
    f = __fadd2_rn(f, big);
    f = __ffma2_rn(f, make_float2(1.f / (float)(1 << (BITS * (i0 % kIn))), 1.f / (float)(1 << (BITS * (i1 % kIn)))), nz[i]);
    v[i] = __fmul2_rn(f, s[i]);
  }
}

template <int OUT>
__device__ __forceinline__ void store_row8(void* row, int c, const float2 (&v)[4]) {
  if constexpr (OUT == KVQ_DT_FP32) {
    float* p = static_cast<float*>(row);
    *reinterpret_cast<float4*>(p + quad_ch<OUT>(c, 0)) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    *reinterpret_cast<float4*>(p + quad_ch<OUT>(c, 1)) = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (OUT == KVQ_DT_BF16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[i].x, v[i].y);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        const __half2 h = __floats2half2_rn(v[i].x, v[i].y);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + 8 * c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The warp's 32 tokens t0 .. t0 + 31 (t0 a multiple of 32, may lie before or behind what is asked for) of one head.
// BITS: of the codes; kKeys: scales per (32-token group, channel), else per (token, 32-channel group).
template <int BITS, bool kKeys, int OUT>
__device__ __forceinline__ void read_rows(const KiviReadArgs& a, int b, int h, int u, int lane) {
  constexpr int kRow = kD * BITS / 8;
  constexpr int kElem = (OUT == KVQ_DT_FP32) ? 4 : 2;
  const int c = lane & 15, odd = lane >> 4;
  const int R = a.residual;
  const int nqk = min(max(a.n_quant_k[b], 0), a.max_tokens) / kGroup * kGroup;
  const int n = nqk + max(0, min(a.n_tok[b] - nqk, R));
  const int nq = kKeys ? nqk : (R > 0) ? min(max(a.n_quant_v[b], 0), nqk) : nqk;
  const int first = a.tok_begin ? a.tok_begin[b - a.b0] : 0;
  // tokens [lo, hi) are asked for and there
  const int lo = max(first, 0), hi = (int)min((long long)first + a.n_tok_out, (long long)n);
  if ((long long)lo + kGroup * (long long)u >= (long long)hi + kGroup) return;
  const int t0 = (lo / kGroup + u) * kGroup;
  if (t0 >= hi) return;
  const int i0 = max(lo - t0, 0), i1 = min(hi - t0, kGroup);  // of the 32
  const size_t bh = (size_t)b * a.H + h;
  // token t goes to row t - first
  unsigned char* out = static_cast<unsigned char*>(kKeys ? a.k_out : a.v_out) +
                       ((int64_t)(b - a.b0) * a.sb + (int64_t)h * a.sh + ((int64_t)t0 - first) * kD) * kElem;
  const uint8_t* codes = (kKeys ? a.k_codes : a.v_codes) + (bh * a.max_tokens + t0) * kRow;
  // the two scales of a token's quads (values: both channels groups of the lane)
  const uint16_t* sp = a.v_scale + (bh * a.max_tokens + t0) * (kD / kGroup);
  const uint16_t* zp = a.v_zero + (bh * a.max_tokens + t0) * (kD / kGroup);
  const int g0 = quad_ch<OUT>(c, 0) / kGroup, g1 = quad_ch<OUT>(c, 1) / kGroup;
  auto value_scales = [&](uint16_t s0, uint16_t s1, uint16_t z0, uint16_t z1, float2 (&s)[4], float2 (&nz)[4]) {
    const float a0 = __half2float(__ushort_as_half(s0)), a1 = __half2float(__ushort_as_half(s1));
    const float b0 = -__half2float(__ushort_as_half(z0)), b1 = -__half2float(__ushort_as_half(z1));
    s[0] = s[1] = make_float2(a0, a0);
    s[2] = s[3] = make_float2(a1, a1);
    nz[0] = nz[1] = make_float2(b0, b0);
    nz[2] = nz[3] = make_float2(b1, b1);
  };
  if (t0 + kGroup <= nq) {
    float2 ks[4], knz[4];
    if constexpr (kKeys) {
      const size_t g = (bh * (a.max_tokens / kGroup) + t0 / kGroup) * kD;
      half8(load_half8<OUT>(a.k_scale + g, c), ks);
      half8(load_half8<OUT>(a.k_zero + g, c), knz);
#pragma unroll
      for (int i = 0; i < 4; ++i) knz[i] = make_float2(-knz[i].x, -knz[i].y);
    }
#pragma unroll
    for (int k0 = 0; k0 < 16; k0 += 8) {
      uint32_t w[8];
      uint16_t s0[8], s1[8], z0[8], z1[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = 2 * (k0 + k) + odd;
        w[k] = load_codes8<BITS, OUT>(codes + i * kRow, c);
        if constexpr (!kKeys) {
          s0[k] = __ldg(sp + i * (kD / kGroup) + g0);
          z0[k] = __ldg(zp + i * (kD / kGroup) + g0);
          s1[k] = OUT == KVQ_DT_FP32 ? __ldg(sp + i * (kD / kGroup) + g1) : s0[k];
          z1[k] = OUT == KVQ_DT_FP32 ? __ldg(zp + i * (kD / kGroup) + g1) : z0[k];
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = 2 * (k0 + k) + odd;
        float2 v[4];
        if constexpr (kKeys) {
          dequant8<BITS>(w[k], ks, knz, v);
        } else {
          float2 s[4], nz[4];
          value_scales(s0[k], s1[k], z0[k], z1[k], s, nz);
          dequant8<BITS>(w[k], s, nz, v);
        }
        if (i >= i0 && i < i1) store_row8<OUT>(out + i * kD * kElem, c, v);
      }
    }
    return;
  }
  // tokens behind the quantized ones; a group's value rows wrap around the ring at most once (R >= 32)
  const uint16_t* resid = (kKeys ? a.k_resid : a.v_resid) + bh * R * kD;
  const int r0 = kKeys ? t0 - nqk : t0 % R;
  auto ring = [&](int i) { return kKeys || r0 + i < R ? r0 + i : r0 + i - R; };
  if (t0 >= nq) {
#pragma unroll
    for (int k0 = 0; k0 < 16; k0 += 8) {
      uint4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = 2 * (k0 + k) + odd;
        if (i >= i0 && i < i1) x[k] = load_half8<OUT>(resid + (size_t)ring(i) * kD, c);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = 2 * (k0 + k) + odd;
        if (i < i0 || i >= i1) continue;
        if constexpr (OUT == KVQ_DT_FP16) {
          *reinterpret_cast<uint4*>(out + i * kD * kElem + 16 * c) = x[k];
        } else {
          float2 v[4];
          half8(x[k], v);
          store_row8<OUT>(out + i * kD * kElem, c, v);
        }
      }
    }
    return;
  }
  if constexpr (kKeys) return;  // not reached: the keys' count is a multiple of the group
  // the group in which the quantized values end
#pragma unroll 1
  for (int k0 = 0; k0 < 16; k0 += 8) {
    uint4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = 2 * (k0 + k) + odd, t = t0 + i;
      x[k] = make_uint4(0u, 0u, 0u, 0u);
      if (i < i0 || i >= i1) continue;
      if (t >= nq) {
        x[k] = load_half8<OUT>(resid + (size_t)ring(i) * kD, c);
      } else {
        x[k].x = load_codes8<BITS, OUT>(codes + i * kRow, c);
        x[k].y = __ldg(sp + i * (kD / kGroup) + g0) | ((uint32_t)__ldg(sp + i * (kD / kGroup) + g1) << 16);
        x[k].z = __ldg(zp + i * (kD / kGroup) + g0) | ((uint32_t)__ldg(zp + i * (kD / kGroup) + g1) << 16);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = 2 * (k0 + k) + odd, t = t0 + i;
      if (i < i0 || i >= i1) continue;
      float2 v[4];
      if (t >= nq) {
        half8(x[k], v);
      } else {
        float2 s[4], nz[4];
        value_scales(x[k].y & 0xFFFFu, x[k].y >> 16, x[k].z & 0xFFFFu, x[k].z >> 16, s, nz);
        dequant8<BITS>(x[k].x, s, nz, v);
      }
      store_row8<OUT>(out + i * kD * kElem, c, v);
    }
  }
}

template <int OUT>
__global__ void __launch_bounds__(read_threads(OUT)) kivi_read_kernel(const KiviReadArgs a) {
  const int lane = threadIdx.x & 31;
  const int two = a.k_out && a.v_out;
  const unsigned unit = blockIdx.x * (read_threads(OUT) / 32) + (threadIdx.x >> 5);
  if (unit >= (unsigned)(a.B * a.H * a.chunks.d) << two) return;  // below 2^31 (checked by the host)
  const int row = div_by((int)unit, a.chunks), u = (int)unit - row * a.chunks.d;  // row: (b, h, keys or values)
  const bool keys = a.k_out && !(two && (row & 1));
  const int bh = row >> two, x = div_by(bh, a.heads);
  const int b = a.b0 + x, h = bh - x * a.H;
  if (keys) {
    if (a.k_bits == 2) read_rows<2, true, OUT>(a, b, h, u, lane);
    else read_rows<4, true, OUT>(a, b, h, u, lane);
  } else {
    if (a.v_bits == 2) read_rows<2, false, OUT>(a, b, h, u, lane);
    else read_rows<4, false, OUT>(a, b, h, u, lane);
  }
}

template <int OUT>
void launch(const KiviReadArgs& a, unsigned units, cudaStream_t s) {
  constexpr int kThreads = read_threads(OUT);
  kivi_read_kernel<OUT><<<(units + kThreads / 32 - 1) / (kThreads / 32), kThreads, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_kivi_read(const KiviReadArgs& args, int out_dt, cudaStream_t s) {
  KiviReadArgs a = args;
  a.chunks = int_div(a.n_tok_out / kGroup + 2);  // the asked tokens may begin and end inside a group
  a.heads = int_div(a.H);
  const unsigned units = (unsigned)(a.B * a.H * a.chunks.d) << (a.k_out && a.v_out);  // below 2^31 (checked by the host)
  if (out_dt == KVQ_DT_FP32) launch<KVQ_DT_FP32>(a, units, s);
  else if (out_dt == KVQ_DT_FP16) launch<KVQ_DT_FP16>(a, units, s);
  else launch<KVQ_DT_BF16>(a, units, s);
  return cudaGetLastError();
}

}  // namespace kvq
