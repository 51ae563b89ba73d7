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
// three shuffles; a warp works on four rows of one token at a time, three such quads at once in
// large calls. Measured (launches back to back in a graph, cos and sin in L2 from the one before): 16381 tokens of
// 32 + 8 + 8 heads, bf16 in, bf16 and fp16 out (411 MB): 67.8 us, 6.1 TB/s, 90 % of the copy rate (a plain copy of as
// many bytes takes 61.3); without the rotation 62.6: what is left is the table's rows, which come from L2. As calls of
// their own with the table from DRAM 70 to 74. One token of 48 rows 2.3 us, all latency. On the way, as
// calls of their own: the first form 91 us, two quads with their loads in flight together 79, two with rows that are
// the first to leave L2 72, three 70.5, four 74; blocks of 256 threads cost 3 us more than blocks of 64, which leave
// their places sooner.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_common.cuh"
#include "kvq_internal.h"
#include "../../include/kvq.h"

namespace kvq {
namespace {

constexpr int kRowThreads = 64;

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

// kStream: the first to leave L2 again
template <bool kStream>
__device__ __forceinline__ void put16(void* p, uint4 u) {
  if constexpr (kStream) __stcs(static_cast<uint4*>(p), u);
  else *static_cast<uint4*>(p) = u;
}
template <bool kStream>
__device__ __forceinline__ void store8(void* base, int64_t elem, int dt, const float (&v)[8]) {
  if (dt == KVQ_DT_FP32) {
    float* p = static_cast<float*>(base) + elem;
#pragma unroll
    for (int i = 0; i < 8; i += 4)
      put16<kStream>(p + i, make_uint4(__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3])));
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
  put16<kStream>(static_cast<uint16_t*>(base) + elem, make_uint4(w[0], w[1], w[2], w[3]));
}

// sum over the eight lanes of a row
__device__ __forceinline__ float sum8(unsigned mask, float x) {
#pragma unroll
  for (int off = 4; off >= 1; off >>= 1) x += __shfl_xor_sync(mask, x, off);
  return x;
}

// eight consecutive channels as stored
template <int DT>
struct Raw8 {
  uint4 u[DT == KVQ_DT_FP32 ? 2 : 1];
};
template <int DT, bool kStream>
__device__ __forceinline__ Raw8<DT> load_raw8(const void* base, int64_t elem) {
  Raw8<DT> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(base) + elem * (DT == KVQ_DT_FP32 ? 4 : 2));
  r.u[0] = kStream ? __ldcs(p) : p[0];
  if constexpr (DT == KVQ_DT_FP32) r.u[1] = kStream ? __ldcs(p + 1) : p[1];
  return r;
}
template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == KVQ_DT_FP32) {
      const uint4 u = r.u[i >> 1];
      v[2 * i] = __uint_as_float((i & 1) ? u.z : u.x);
      v[2 * i + 1] = __uint_as_float((i & 1) ? u.w : u.y);
    } else {
      const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
      const float2 f = (DT == KVQ_DT_BF16) ? bf2(w[i]) : hf2(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

// A warp takes kPer row quads of one token (the first quads of the query, key and value rows, in that order, are
// part 0), all their loads in flight before the first is used; the token's cos and sin serve them all.
template <int DT, int kPer>
__global__ void __launch_bounds__(kRowThreads) qk_rows_kernel(const QkRowsArgs a, const unsigned units) {
  const int lane = threadIdx.x & 31, l8 = lane & 7;
  const int rows = a.q.heads + a.k.heads + a.v.heads;
  const unsigned unit = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;  // warp-uniform
  const int token = div_by((int)unit, a.parts), part = (int)unit - token * a.parts.d;
  const int b = div_by(token, a.tokens), j = token - b * a.N;
  const int pos = a.pos ? a.pos[token] : 0;
  if (pos < 0) return;  // padding: neither read nor written
  if (a.cos && pos >= a.max_ctx) {
    if (lane == 0) set_error(a.err, KVQ_ERR_CAPACITY);
    return;
  }
  Raw8<DT> rl[kPer], rh[kPer];
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    int h = (part * kPer + p) * 4 + (lane >> 3);
    if (h >= rows) {
      rl[p] = rh[p] = {};
      continue;
    }
    const QkRows& t = h < a.q.heads ? a.q : h < a.q.heads + a.k.heads ? a.k : a.v;
    if (h >= a.q.heads) h -= h < a.q.heads + a.k.heads ? a.q.heads : a.q.heads + a.k.heads;
    const int64_t e = (int64_t)b * t.sb + (int64_t)j * t.st + (int64_t)h * t.sh + 8 * l8;
    rl[p] = load_raw8<DT, (kPer > 1)>(t.in, e);
    rh[p] = load_raw8<DT, (kPer > 1)>(t.in, e + 64);
  }
  float c[8] = {}, s[8] = {};
  if (a.cos) {
    load8<KVQ_DT_FP32>(a.cos, (int64_t)pos * (kD / 2) + 8 * l8, c);
    load8<KVQ_DT_FP32>(a.sin, (int64_t)pos * (kD / 2) + 8 * l8, s);
  }
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    int h = (part * kPer + p) * 4 + (lane >> 3);
    const bool there = h < rows;
    const bool is_q = h < a.q.heads, is_v = h >= a.q.heads + a.k.heads;
    if (!is_q) h -= is_v ? a.q.heads + a.k.heads : a.q.heads;
    const QkRows& t = is_q ? a.q : is_v ? a.v : a.k;
    float lo[8], hi[8];
    widen8<DT>(rl[p], lo);
    widen8<DT>(rh[p], hi);
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
    if (!there) continue;
    if (!is_v) {
      const void* w = is_q ? a.wq : a.wk;
      float wl[8], wh[8];
      load8<DT>(w, 8 * l8, wl);
      load8<DT>(w, 64 + 8 * l8, wh);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo[i] = lo[i] * r * wl[i];
        hi[i] = hi[i] * r * wh[i];
      }
      if (a.cos) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = lo[i], y = hi[i];
          lo[i] = x * c[i] - y * s[i];
          hi[i] = y * c[i] + x * s[i];
        }
      }
    }
    const int64_t o = (int64_t)b * t.ob + (int64_t)j * t.ot + (int64_t)h * t.oh + 8 * l8;
    store8<(kPer > 1)>(t.out, o, t.out_dt, lo);
    store8<(kPer > 1)>(t.out, o + 64, t.out_dt, hi);
  }
}

template <int DT, int kPer>
cudaError_t launch_rows(const QkRowsArgs& args, int quads, cudaStream_t s) {
  QkRowsArgs a = args;
  a.parts = int_div((quads + kPer - 1) / kPer);
  a.tokens = int_div(a.N);
  const unsigned units = (unsigned)(a.B * a.N * a.parts.d);  // below 2^31 (checked by the host)
  qk_rows_kernel<DT, kPer><<<(units + kRowThreads / 32 - 1) / (kRowThreads / 32), kRowThreads, 0, s>>>(a, units);
  return cudaGetLastError();
}
template <int DT>
cudaError_t launch_rows_of(const QkRowsArgs& a, cudaStream_t s) {
  const int quads = (a.q.heads + a.k.heads + a.v.heads + 3) / 4;
  // Three quads a warp, read and written past the table's rows in L2, once every SM has thirty; one quad below, where
  // more warps shorten the chain. 48 heads, bf16, back to back in a graph, three / one: 1 token 2.9 / 2.3 us, 64 tokens
  // 3.1 / 2.6, 272 3.6 / 3.2, 500 4.2 / 4.4, 1000 5.9 / 6.5, 4000 18.2 / 22.2, 16381 67.8 / 93.2.
  if ((int64_t)a.B * a.N * quads >= 30 * device_sms()) return launch_rows<DT, 3>(a, quads, s);
  return launch_rows<DT, 1>(a, quads, s);
}

}  // namespace

cudaError_t launch_qk_rows(const QkRowsArgs& a, int in_dt, cudaStream_t s) {
  if ((int64_t)a.B * a.N == 0) return cudaSuccess;
  if (in_dt == KVQ_DT_FP32) return launch_rows_of<KVQ_DT_FP32>(a, s);
  if (in_dt == KVQ_DT_FP16) return launch_rows_of<KVQ_DT_FP16>(a, s);
  return launch_rows_of<KVQ_DT_BF16>(a, s);
}

}  // namespace kvq
