// Norms of queries and keys for each head with the position rotation in the same pass.
//
// A row is the D = 128 channels of one head of one token. y = x rsqrt(mean(x^2) + eps) w, then
// (rotary tables given) the rotate-half pairs (i, i + 64) turn by the angle of the token's
// position: y_i' = y_i cos - y_{i+64} sin, y_{i+64}' = y_{i+64} cos + y_i sin. Value rows are
// only converted to the type the cache stores. All arithmetic is fp32, each output is rounded
// once.
//
// Bound: HBM (each row is read once and written once; about 6 operations a channel). Eight
// lanes share a row, lane l holding channels 8l .. 8l+7 and their partners 64 + 8l .., so both
// halves of every pair are in one lane, the loads and stores are 16 bytes and the mean takes
// three shuffles; a warp works on four rows of one token at a time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_common.cuh"
#include "kvq_internal.h"
#include "../../include/kvq.h"

namespace kvq {
namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ float2 bf2(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ float2 hf2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// eight consecutive channels as fp32
template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t elem, float (&v)[8]) {
  if constexpr (DT == KVQ_DT_FP32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + elem);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + elem);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = (DT == KVQ_DT_BF16) ? bf2(w[i]) : hf2(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

__device__ __forceinline__ void store8(void* base, int64_t elem, int dt, const float (&v)[8]) {
  if (dt == KVQ_DT_FP32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + elem);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (dt == KVQ_DT_BF16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + elem) = make_uint4(w[0], w[1], w[2], w[3]);
}

// sum over the eight lanes of a row
__device__ __forceinline__ float sum8(unsigned mask, float x) {
#pragma unroll
  for (int off = 4; off >= 1; off >>= 1) x += __shfl_xor_sync(mask, x, off);
  return x;
}

template <int DT>
__global__ void __launch_bounds__(kRowThreads) qk_rows_kernel(const QkRowsArgs a) {
  const int lane = threadIdx.x & 31, l8 = lane & 7;
  const int rows = a.q.heads + a.k.heads + a.v.heads, quads = (rows + 3) / 4;
  const int64_t unit = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (unit >= (int64_t)a.B * a.N * quads) return;  // warp-uniform
  const int64_t token = unit / quads;
  const int b = (int)(token / a.N), j = (int)(token - (int64_t)b * a.N);
  int h = (int)(unit - token * quads) * 4 + (lane >> 3);
  const int pos = a.pos ? a.pos[token] : 0;
  if (pos < 0) return;  // padding: neither read nor written
  if (a.cos && pos >= a.max_ctx) {
    if (lane == 0) set_error(a.err, KVQ_ERR_CAPACITY);
    return;
  }
  const bool there = h < rows;
  const bool is_q = h < a.q.heads, is_v = h >= a.q.heads + a.k.heads;
  if (!is_q) h -= a.q.heads;
  if (is_v) h -= a.k.heads;
  const QkRows& t = is_q ? a.q : is_v ? a.v : a.k;
  const void* w = is_q ? a.wq : a.wk;
  float lo[8] = {}, hi[8] = {};
  if (there) {
    const int64_t e = (int64_t)b * t.sb + (int64_t)j * t.st + (int64_t)h * t.sh + 8 * l8;
    load8<DT>(t.in, e, lo);
    load8<DT>(t.in, e + 64, hi);
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(lo[i], lo[i], fmaf(hi[i], hi[i], ss));
  ss = sum8(0xFFFFFFFFu, ss);
  float r = rsqrtf(fmaf(ss, 1.f / kD, a.eps));
  if (!is_v && !(ss < 1e37f)) {
    // squares of large bf16 or fp32 values pass the fp32 range: the row times 2^-72 instead (eps is far
    // below the mean's rounding). All eight lanes of a row come here, the warp's others may not.
    constexpr float kDown = 2.117582368135750837e-22f;  // 2^-72
    float s2 = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] *= kDown;
      hi[i] *= kDown;
      s2 = fmaf(lo[i], lo[i], fmaf(hi[i], hi[i], s2));
    }
    r = rsqrtf(sum8(0xFFu << (lane & 24), s2) * (1.f / kD));
  }
  if (!there) return;
  if (!is_v) {
    float wl[8], wh[8];
    load8<DT>(w, 8 * l8, wl);
    load8<DT>(w, 64 + 8 * l8, wh);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = lo[i] * r * wl[i];
      hi[i] = hi[i] * r * wh[i];
    }
    if (a.cos) {
      float c[8], s[8];
      load8<KVQ_DT_FP32>(a.cos, (int64_t)pos * (kD / 2) + 8 * l8, c);
      load8<KVQ_DT_FP32>(a.sin, (int64_t)pos * (kD / 2) + 8 * l8, s);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = lo[i], y = hi[i];
        lo[i] = x * c[i] - y * s[i];
        hi[i] = y * c[i] + x * s[i];
      }
    }
  }
  const int64_t o = (int64_t)b * t.ob + (int64_t)j * t.ot + (int64_t)h * t.oh + 8 * l8;
  store8(t.out, o, t.out_dt, lo);
  store8(t.out, o + 64, t.out_dt, hi);
}

}  // namespace

cudaError_t launch_qk_rows(const QkRowsArgs& a, int in_dt, cudaStream_t s) {
  const int rows = a.q.heads + a.k.heads + a.v.heads;
  const int64_t units = (int64_t)a.B * a.N * ((rows + 3) / 4);
  const int64_t blocks = (units + kRowThreads / 32 - 1) / (kRowThreads / 32);
  if (blocks == 0) return cudaSuccess;
  const unsigned g = (unsigned)blocks;  // below 2^31 (checked by the host)
  if (in_dt == KVQ_DT_FP32) qk_rows_kernel<KVQ_DT_FP32><<<g, kRowThreads, 0, s>>>(a);
  else if (in_dt == KVQ_DT_FP16) qk_rows_kernel<KVQ_DT_FP16><<<g, kRowThreads, 0, s>>>(a);
  else qk_rows_kernel<KVQ_DT_BF16><<<g, kRowThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
