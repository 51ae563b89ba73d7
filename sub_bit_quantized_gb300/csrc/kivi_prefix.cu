// Attention of a batch whose requests share a prefix that is cached once.
//
// Row r (request, drafted token, query head) attends the prefix's tokens and its request's own: with
// (o0, L0) the normalised output and the log2 of the sum of 2^score over the prefix, (o1, L1) over the
// request's cache and drafts,
//   o = (2^(L0 - M) o0 + 2^(L1 - M) o1) / (2^(L0 - M) + 2^(L1 - M)),  M = max(L0, L1).
// Over the prefix the rows of all requests are rows of one matrix per KV head, as if they were the
// tokens of one request; over its own tokens a request is a tree without the prefix. Both parts write
// fp32 outputs and L into the workspace.
#include <cfloat>

#include "kvq_common.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

// A warp a row, a lane four channels.
constexpr int kCombineThreads = 128;
__global__ void __launch_bounds__(kCombineThreads) kivi_prefix_combine_kernel(const KiviPrefixArgs a, const int rows) {
  const int row = blockIdx.x * (kCombineThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= rows) return;
  const int tok = div_by(row, a.heads), b = div_by(tok, a.tokens);
  if (a.own.n_draft && tok - b * a.own.N >= a.own.n_draft[b]) return;  // padding
  const size_t at = (size_t)row * kD + 4 * lane;
  const float l0 = a.prefix.lse[row], l1 = a.own.lse[row];
  const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.prefix.out) + at);
  const float4 y = *reinterpret_cast<const float4*>(static_cast<const float*>(a.own.out) + at);
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

}  // namespace

cudaError_t launch_kivi_prefix(const KiviPrefixArgs& args, cudaStream_t st) {
  cudaError_t e;
  if ((e = launch_kivi_tree(args.prefix, st)) != cudaSuccess) return e;
  if ((e = launch_kivi_tree(args.own, st)) != cudaSuccess) return e;
  KiviPrefixArgs a = args;
  a.heads = int_div(a.own.Hq);
  a.tokens = int_div(a.own.N);
  const int rows = a.own.B * a.own.N * a.own.Hq, per = kCombineThreads / 32;
  kivi_prefix_combine_kernel<<<(rows + per - 1) / per, kCombineThreads, 0, st>>>(a, rows);
  return cudaGetLastError();
}

}  // namespace kvq
