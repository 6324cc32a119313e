// quant_mla.cu -- multi-head latent attention over the quantised latent cache.
//
//     logit[t, h, s] = scale * (q_nope[t, h] . c[s] + q_rope[t, h] . r[s])
//     out[t, h]      = sum_s softmax_s(logit[t, h, :]) c[s],   lse[t, h] = ln sum_s exp(logit[t, h, s])
//
// over the selected positions s = topk[t, j] of the query's sequence, or over every position up to its own.
// One warp takes a (query, head) row: one pass over its keys with the running maximum and sum, lane i
// holding 16 latent and 2 rotary values.
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"
#include "quant_rows.cuh"

namespace dsa {
namespace {

using namespace quant;

constexpr int kWarps = 4;

template <bool FP4>
__global__ void __launch_bounds__(kWarps * 32) quant_mla_kernel(const dsa_quant_mla_args a, unsigned* status) {
  constexpr int kRow = FP4 ? kRow4 : kRow8;
  const int lane = threadIdx.x & 31;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const long long row_id = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row_id >= static_cast<long long>(a.total_q) * a.H) return;
  const int t = static_cast<int>(row_id / a.H), h = static_cast<int>(row_id % a.H);
  long long n = 0;  // keys to look at
  int b = 0, len = 0;
  if (t < __ldg(a.cu_q_lens + a.B)) {
    b = sequence_of(a.cu_q_lens, a.B, t);
    len = __ldg(a.seq_lens + b);
    n = a.topk ? a.topk_width : static_cast<long long>(len) - __ldg(a.cu_q_lens + b + 1) + t + 1;
    if (!a.topk) {
      const long long room = static_cast<long long>(a.max_pages_per_seq) * a.page_size;
      if (n > room) {
        if (lane == 0) atomicOr(status, kStatusUncovered);
        n = room;
      }
    }
  }
  const __nv_bfloat16* qn = static_cast<const __nv_bfloat16*>(a.q_nope) + t * a.qn_stride_t + h * a.qn_stride_h + 16 * lane;
  const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q_rope) + t * a.qr_stride_t + h * a.qr_stride_h + 2 * lane;
  float q[18], o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) q[i] = __bfloat162float(qn[i]), o[i] = 0.f;
  q[16] = __bfloat162float(qr[0]), q[17] = __bfloat162float(qr[1]);
  const uint8_t* cache = static_cast<const uint8_t*>(a.cache);
  const float f = a.scale * 1.4426950408889634f;
  float m = -INFINITY, l = 0.f;
  for (long long j = 0; j < n; ++j) {
    const long long s = a.topk ? __ldg(a.topk + static_cast<long long>(t) * a.topk_width + j) : j;
    if (s < 0 || s >= len) continue;
    const long long lp = s / a.page_size;
    const int page = lp < a.max_pages_per_seq ? __ldg(a.block_tables + static_cast<long long>(b) * a.max_pages_per_seq + lp) : -1;
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) atomicOr(status, kStatusBadPage);
      continue;
    }
    const uint8_t* row = cache + (static_cast<long long>(page) * a.page_size + s % a.page_size) * kRow;
    uint2 c01, c23;
    float scale;
    if (FP4) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(row) + lane);
      const int byte = __ldg(row + kScale4 + lane);
      scale = pow2f(static_cast<int>(__ballot_sync(0xffffffffu, byte >> 7) & 0xFFu) - 128);
      const uint2 lv = levels_at(levels_base(byte & 7), byte & 127);
      c01 = codes4_to_e4m3(w.x, lv);
      c23 = codes4_to_e4m3(w.y, lv);
    } else {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(row) + lane);
      c01 = make_uint2(w.x, w.y);
      c23 = make_uint2(w.z, w.w);
      scale = __ldg(reinterpret_cast<const float*>(row + kScale8));
    }
    float v[16];
    const uint32_t cw[4] = {c01.x, c01.y, c23.x, c23.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 p = from_e4m3x2((cw[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
      v[2 * i] = p.x, v[2 * i + 1] = p.y;
    }
    const uint32_t r = __ldg(reinterpret_cast<const uint32_t*>(row + (FP4 ? kRope4 : kRope8)) + lane);
    float dot = q[16] * __uint_as_float(r << 16) + q[17] * __uint_as_float(r & 0xFFFF0000u);
#pragma unroll
    for (int i = 0; i < 16; ++i) dot = fmaf(q[i], v[i], dot);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, k);
    const float x = dot * scale * f, mn = fmaxf(m, x);
    const float old = exp2f(m - mn), p = exp2f(x - mn);
    m = mn;
    l = l * old + p;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = o[i] * old + p * scale * v[i];
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row_id * kRank + 16 * lane);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    out[i] = make_uint4(pack_bf16(o[8 * i] * inv, o[8 * i + 1] * inv), pack_bf16(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                        pack_bf16(o[8 * i + 4] * inv, o[8 * i + 5] * inv), pack_bf16(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
  if (lane == 0 && a.lse) a.lse[row_id] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

dsa_status validate(const dsa_quant_mla_args* a) {
  if (!a) return DSA_ERR_INVALID_ARGUMENT;
  if (a->B < 0 || a->total_q < 0 || a->H <= 0 || a->topk_width < 0 || a->page_size <= 0 || a->num_pages < 0 ||
      a->max_pages_per_seq < 0 || !(a->scale > 0.f))
    return DSA_ERR_INVALID_ARGUMENT;
  if (a->kv_rank != quant::kRank || a->rope_dim != quant::kRope || quant::row_bytes(a->format) == 0 || a->H > 128)
    return DSA_ERR_UNSUPPORTED;
  if (static_cast<long long>(a->total_q) * a->H >= 0x7FFFFF80LL || static_cast<long long>(a->num_pages) * a->page_size >= 0x7FFFFF80LL)
    return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_quant_mla_workspace_size(const dsa_quant_mla_args* a, size_t* bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARGUMENT;
  const dsa_status st = validate(a);
  if (st != DSA_OK) return st;
  *bytes = 16;
  return DSA_OK;
}

dsa_status dsa_quant_mla(const dsa_quant_mla_args* a, dsa_stream_t stream) {
  const dsa_status st = validate(a);
  if (st != DSA_OK) return st;
  if (a->total_q == 0) return DSA_OK;
  if (!a->q_nope || !a->q_rope || !a->out || !a->cu_q_lens || (!a->seq_lens && a->B > 0) || (!a->cache && a->num_pages > 0) ||
      (!a->block_tables && a->B > 0 && a->max_pages_per_seq > 0) || (a->topk_width > 0 && !a->topk))
    return DSA_ERR_INVALID_ARGUMENT;
  const bool many_t = a->total_q > 1, many_h = a->H > 1;
  if ((many_t && (a->qn_stride_t < 0 || a->qr_stride_t < 0 || a->qn_stride_t % 8 != 0 || a->qr_stride_t % 8 != 0)) ||
      (many_h && (a->qn_stride_h < 0 || a->qr_stride_h < 0 || a->qn_stride_h % 8 != 0 || a->qr_stride_h % 8 != 0)))
    return DSA_ERR_INVALID_ARGUMENT;
  auto al = [](const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  if (!al(a->q_nope, 16) || !al(a->q_rope, 16) || !al(a->cache, 16) || !al(a->out, 16) || !al(a->lse, 4) ||
      !al(a->block_tables, 4) || !al(a->cu_q_lens, 4) || !al(a->seq_lens, 4) || !al(a->topk, 4))
    return DSA_ERR_INVALID_ARGUMENT;
  size_t need = 0;
  dsa_quant_mla_workspace_size(a, &need);
  if (!a->workspace || a->workspace_bytes < need || !al(a->workspace, 16)) return DSA_ERR_WORKSPACE;
  unsigned* status = device_status_ptr();
  if (!status) return DSA_ERR_CUDA;
  const long long rows = static_cast<long long>(a->total_q) * a->H;
  const unsigned blocks = static_cast<unsigned>((rows + kWarps - 1) / kWarps);
  auto* kern = a->format == DSA_FP4_E2M1 ? quant_mla_kernel<true> : quant_mla_kernel<false>;
  const cudaError_t e = launch_pdl(kern, dim3(blocks), dim3(kWarps * 32), 0, reinterpret_cast<cudaStream_t>(stream), *a, status);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
