// prefix_mla.cu -- latent attention for a batch whose sequences share their first tokens.
//
//     logit[t, h, s] = scale * (q_nope[t, h] . c_kv[s] + q_rope[t, h] . k_rope[s]),  s <= p(t)
//     out[t, h]      = sum_s softmax_s(logit[t, h, :]) c_kv[s],   lse[t, h] = ln sum_s exp(logit[t, h, s])
//
// One warp per (query, head) row walks the row's keys once with a running maximum and sum;
// a lane holds 16 latent and 2 rotary values of the query and 16 of the output, all in fp32.
#include <cuda_bf16.h>

#include <algorithm>

#include "dsa_indexer.h"
#include "internal.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kRank = 512, kRope = 64;

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__global__ void __launch_bounds__(256) prefix_mla_rows_kernel(const dsa_prefix_mla_args a, unsigned* status) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(a.total_q) * a.H) return;
  const int t = static_cast<int>(row / a.H), h = static_cast<int>(row - static_cast<long long>(t) * a.H);
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.cu_q_lens + mid) <= t) lo = mid; else hi = mid;
  }
  const int q0 = __ldg(a.cu_q_lens + lo), q1 = __ldg(a.cu_q_lens + lo + 1);
  int sees = t < q1 ? __ldg(a.seq_lens + lo) - (q1 - q0) + (t - q0) + 1 : 0;
  const long long room = static_cast<long long>(a.max_pages_per_seq) * a.page_size;
  if (sees > a.prefix_len && sees > room) {
    if (lane == 0) atomicOr(status, kStatusUncovered);
    sees = static_cast<int>(max(room, static_cast<long long>(a.prefix_len)));
  }
  float q[18];
  const __nv_bfloat16* qn = static_cast<const __nv_bfloat16*>(a.q_nope) + t * a.qn_stride_t + h * a.qn_stride_h;
  const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q_rope) + t * a.qr_stride_t + h * a.qr_stride_h;
  unpack8(reinterpret_cast<const uint4*>(qn)[lane], q);
  unpack8(reinterpret_cast<const uint4*>(qn)[32 + lane], q + 8);
  q[16] = __bfloat162float(qr[2 * lane]);
  q[17] = __bfloat162float(qr[2 * lane + 1]);
  float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  const float sl2 = a.scale * 1.4426950408889634f;
  for (int s = 0; s < sees; ++s) {
    const int j = s / a.page_size;
    const int pg = s < a.prefix_len ? __ldg(a.prefix_pages + j)
                                    : __ldg(a.block_tables + static_cast<long long>(lo) * a.max_pages_per_seq + j);
    if (pg < 0 || pg >= a.num_pages) {
      if (lane == 0) atomicOr(status, kStatusBadPage);
      continue;
    }
    const long long slot = static_cast<long long>(pg) * a.page_size + (s - j * a.page_size);
    float k[18];
    const uint4* cr = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.cache_c) + slot * kRank);
    unpack8(cr[lane], k);
    unpack8(cr[32 + lane], k + 8);
    const __nv_bfloat162 r2 =
        reinterpret_cast<const __nv_bfloat162*>(static_cast<const __nv_bfloat16*>(a.cache_r) + slot * kRope)[lane];
    k[16] = __low2float(r2);
    k[17] = __high2float(r2);
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < 18; ++i) x = fmaf(q[i], k[i], x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x *= sl2;
    const float mn = fmaxf(m, x), c = exp2f(m - mn), p = exp2f(x - mn);
    m = mn;
    l = l * c + p;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = fmaf(p, k[i], o[i] * c);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * i] * inv, o[2 * i + 1] * inv);
    u[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * kRank);
  dst[lane] = make_uint4(u[0], u[1], u[2], u[3]);
  dst[32 + lane] = make_uint4(u[4], u[5], u[6], u[7]);
  if (a.lse && lane == 0) a.lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

dsa_status validate(const dsa_prefix_mla_args* a) {
  if (!a) return DSA_ERR_INVALID_ARGUMENT;
  if (a->B < 0 || a->total_q < 0 || a->H <= 0 || a->kv_rank <= 0 || a->rope_dim <= 0 || a->page_size <= 0 ||
      a->num_pages < 0 || a->max_pages_per_seq < 0 || a->prefix_len < 0 || a->num_prefix_pages < 0 ||
      !(a->scale > 0.f) || !(a->scale < INFINITY))
    return DSA_ERR_INVALID_ARGUMENT;
  if (static_cast<long long>(a->num_prefix_pages) * a->page_size < a->prefix_len) return DSA_ERR_INVALID_ARGUMENT;
  if (a->kv_rank != kRank || a->rope_dim != kRope) return DSA_ERR_UNSUPPORTED;
  if (a->H > 128) return DSA_ERR_UNSUPPORTED;
  if (a->page_size != 16 && a->page_size != 32 && a->page_size != 64 && a->page_size != 128)
    return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_prefix_mla_workspace_size(const dsa_prefix_mla_args* a, size_t* bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARGUMENT;
  const dsa_status st = validate(a);
  if (st != DSA_OK) return st;
  *bytes = 0;
  return DSA_OK;
}

dsa_status dsa_prefix_mla(const dsa_prefix_mla_args* a, dsa_stream_t stream) {
  const dsa_status st = validate(a);
  if (st != DSA_OK) return st;
  if (a->total_q == 0) return DSA_OK;
  if (!a->q_nope || !a->q_rope || !a->out) return DSA_ERR_INVALID_ARGUMENT;
  if (a->B < 1 || !a->cache_c || !a->cache_r || !a->cu_q_lens || !a->seq_lens ||
      (a->max_pages_per_seq > 0 && !a->block_tables) || (a->prefix_len > 0 && !a->prefix_pages))
    return DSA_ERR_INVALID_ARGUMENT;
  auto al = [](const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  if (!al(a->q_nope, 16) || !al(a->q_rope, 16) || !al(a->cache_c, 16) || !al(a->cache_r, 16) || !al(a->out, 16) ||
      !al(a->lse, 4) || !al(a->prefix_pages, 4) || !al(a->block_tables, 4) || !al(a->cu_q_lens, 4) ||
      !al(a->seq_lens, 4))
    return DSA_ERR_INVALID_ARGUMENT;
  if (a->qn_stride_t % 8 || a->qn_stride_h % 8 || a->qr_stride_t % 8 || a->qr_stride_h % 8)
    return DSA_ERR_INVALID_ARGUMENT;
  size_t need = 0;
  dsa_prefix_mla_workspace_size(a, &need);
  if (need > 0 && (!a->workspace || a->workspace_bytes < need || !al(a->workspace, 16))) return DSA_ERR_WORKSPACE;
  unsigned* status = device_status_ptr();
  if (!status) return DSA_ERR_CUDA;
  const long long rows = static_cast<long long>(a->total_q) * a->H;
  if ((rows + 7) / 8 > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  const cudaError_t e = launch_pdl(prefix_mla_rows_kernel, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0,
                                   reinterpret_cast<cudaStream_t>(stream), *a, status);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
