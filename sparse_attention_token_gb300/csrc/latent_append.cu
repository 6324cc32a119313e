// latent_append.cu -- the step's latent rows (norm, RoPE) through slot_mapping into the paged cache.
//
//     cache_c[slot] = bf16(w * c * rsqrt(mean(c^2) + eps)),   cache_r[slot] = bf16(RoPE(r, position))
//
// One warp takes TOK tokens and issues all their loads before it uses any.  A lane holds two
// 16-byte chunks of a token's 512 latent values (the mean is one warp reduction in fp32); the
// rotary rows of four tokens take one 16-byte load of the warp, 8 lanes a token, and the half
// that a pair needs from the other half of the row comes by a shuffle of four lanes.  Memory
// bound: 1152 bytes read and 1152 written per token, plus 256 of cosines and sines.  65537 tokens
// take 29.4 us (5.6 TB/s of the 6.8 that a copy reaches; without norm and RoPE 23.7 us, 6.3 TB/s),
// 64 take 1.7 us.  Loading the cosines ahead of the norm took 32.1 us: the warps hold more
// registers and fewer run at once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dsa_indexer.h"
#include "internal.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kRank = 512, kRope = 64;
constexpr int kWarps = 4;

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

template <int TOK>
__global__ void __launch_bounds__(kWarps * 32) latent_append_kernel(const dsa_mla_cache_append_args a,
                                                                    unsigned* status) {
  const int lane = threadIdx.x & 31;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const long long t0 = (static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * TOK;
  const long long n_slots = static_cast<long long>(a.num_pages) * a.page_size;
  const __nv_bfloat16* c_in = static_cast<const __nv_bfloat16*>(a.c_kv);
  const __nv_bfloat16* r_in = static_cast<const __nv_bfloat16*>(a.k_rope);
  long long slot[TOK];
  uint4 raw[TOK][2];
#pragma unroll
  for (int k = 0; k < TOK; ++k) {
    const long long t = t0 + k;
    slot[k] = t < a.n ? a.slot_mapping[t] : -1;
    raw[k][0] = raw[k][1] = make_uint4(0u, 0u, 0u, 0u);
    if (t < a.n) {
      const uint4* row = reinterpret_cast<const uint4*>(c_in + t * a.c_stride);
      raw[k][0] = __ldg(row + lane);
      raw[k][1] = __ldg(row + 32 + lane);
    }
  }
  // rotary part: lanes 8k .. 8k + 7 hold token k's 64 values
  const int rk = lane >> 3, ch = lane & 7;
  const long long rt = t0 + rk;
  const bool r_live = rk < TOK && rt < a.n;
  uint4 rraw = make_uint4(0u, 0u, 0u, 0u);
  long long rpos = -1;
  if (r_live) {
    rraw = __ldg(reinterpret_cast<const uint4*>(r_in + rt * a.r_stride) + ch);
    rpos = a.positions ? __ldg(a.positions + rt) : rt;
  }
  const bool turn = a.rope_cos != nullptr;
  const bool pos_ok = !turn || (rpos >= 0 && rpos < a.rope_rows);
  // a token is written when its slot and its position are inside; lane k's view for all lanes
  const unsigned pos_mask = __ballot_sync(0xffffffffu, pos_ok);
  bool bad = false;
#pragma unroll
  for (int k = 0; k < TOK; ++k) {
    if (slot[k] < 0) continue;
    if (slot[k] >= n_slots || !((pos_mask >> (8 * k)) & 1u)) {
      bad = true;
      slot[k] = -1;
    }
  }
  if (bad && lane == 0) atomicOr(status, kStatusBadPage);
  long long rslot = -1;
#pragma unroll
  for (int k = 0; k < TOK; ++k)
    if (rk == k) rslot = slot[k];

  float w[2][8];
  if (a.norm_weight) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4* wp = reinterpret_cast<const float4*>(a.norm_weight + i * 256 + lane * 8);
      const float4 u = __ldg(wp), v = __ldg(wp + 1);
      w[i][0] = u.x, w[i][1] = u.y, w[i][2] = u.z, w[i][3] = u.w;
      w[i][4] = v.x, w[i][5] = v.y, w[i][6] = v.z, w[i][7] = v.w;
    }
  }
  uint4* out_c = reinterpret_cast<uint4*>(a.cache_c);
#pragma unroll
  for (int k = 0; k < TOK; ++k) {
    if (slot[k] < 0) continue;  // the same in the whole warp
    uint4* dst = out_c + slot[k] * (kRank / 8);
    if (a.norm_weight) {
      float x[2][8];
      unpack8(raw[k][0], x[0]);
      unpack8(raw[k][1], x[1]);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(x[i >> 3][i & 7], x[i >> 3][i & 7], ss);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = rsqrtf(ss * (1.f / kRank) + a.norm_eps);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i >> 3][i & 7] *= inv * w[i >> 3][i & 7];
      dst[lane] = pack8(x[0]);
      dst[32 + lane] = pack8(x[1]);
    } else {
      dst[lane] = raw[k][0];
      dst[32 + lane] = raw[k][1];
    }
  }
  // RoPE: the lane's eight values are elements 8 ch .. 8 ch + 7 of its token's row
  uint4 res = rraw;
  if (turn) {
    uint4 other;  // the chunk that holds the other members of the pairs (i, i + 32)
    other.x = __shfl_xor_sync(0xffffffffu, rraw.x, 4);
    other.y = __shfl_xor_sync(0xffffffffu, rraw.y, 4);
    other.z = __shfl_xor_sync(0xffffffffu, rraw.z, 4);
    other.w = __shfl_xor_sync(0xffffffffu, rraw.w, 4);
    if (rslot >= 0) {
      float x[8], y[8], z[8];
      unpack8(rraw, x);
      const float* cosr = a.rope_cos + rpos * (kRope / 2);
      const float* sinr = a.rope_sin + rpos * (kRope / 2);
      if (a.rope_interleaved) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(cosr) + ch);
        const float4 s = __ldg(reinterpret_cast<const float4*>(sinr) + ch);
        const float cc[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[2 * i] = x[2 * i] * cc[i] - x[2 * i + 1] * sv[i];
          z[2 * i + 1] = x[2 * i] * sv[i] + x[2 * i + 1] * cc[i];
        }
      } else {
        unpack8(other, y);
        const int c4 = (ch & 3) * 2;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const float4 c = __ldg(reinterpret_cast<const float4*>(cosr) + c4 + hh);
          const float4 s = __ldg(reinterpret_cast<const float4*>(sinr) + c4 + hh);
          const float cc[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = 4 * hh + i;
            // first half: a cos - b sin; second half: a sin + b cos (a from the first half)
            z[e] = ch < 4 ? x[e] * cc[i] - y[e] * sv[i] : y[e] * sv[i] + x[e] * cc[i];
          }
        }
      }
      res = pack8(z);
    }
  }
  if (rslot >= 0) reinterpret_cast<uint4*>(a.cache_r)[rslot * (kRope / 8) + ch] = res;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_mla_cache_append(const dsa_mla_cache_append_args* a, dsa_stream_t stream) {
  if (!a) return DSA_ERR_INVALID_ARGUMENT;
  if (a->n < 0 || a->page_size <= 0 || a->num_pages < 0 || a->kv_rank <= 0 || a->rope_dim < 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (a->kv_rank != kRank || a->rope_dim != kRope) return DSA_ERR_UNSUPPORTED;
  if (a->n == 0) return DSA_OK;
  if (!a->c_kv || !a->k_rope || !a->slot_mapping || !a->cache_c || !a->cache_r) return DSA_ERR_INVALID_ARGUMENT;
  if ((a->rope_cos == nullptr) != (a->rope_sin == nullptr)) return DSA_ERR_INVALID_ARGUMENT;
  if (a->rope_cos && (a->rope_rows < 1 || (!a->positions && a->rope_rows < a->n))) return DSA_ERR_INVALID_ARGUMENT;
  if (a->norm_weight && !(a->norm_eps >= 0.f)) return DSA_ERR_INVALID_ARGUMENT;
  // (one token's strides lead nowhere)
  if (a->n > 1 && (a->c_stride < 0 || a->r_stride < 0 || a->c_stride % 8 != 0 || a->r_stride % 8 != 0))
    return DSA_ERR_INVALID_ARGUMENT;
  auto al = [](const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  if (!al(a->c_kv, 16) || !al(a->k_rope, 16) || !al(a->cache_c, 16) || !al(a->cache_r, 16) ||
      !al(a->norm_weight, 16) || !al(a->rope_cos, 16) || !al(a->rope_sin, 16) || !al(a->slot_mapping, 8) ||
      !al(a->positions, 4))
    return DSA_ERR_INVALID_ARGUMENT;
  unsigned* status = device_status_ptr();
  if (!status) return DSA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // Tokens a warp: more of them keep more loads in flight, as long as some 4096 warps remain.
  // Of 1, 2, 4: 64 tokens 1.7, 2.0, 2.4 us; 2048 2.3, 2.3, 2.5; 8192 5.1, 4.1, 4.5; 65537 34.0, 30.9, 29.4.
  const int tok = a->n >= 16384 ? 4 : (a->n >= 8192 ? 2 : 1);
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(a->n) + kWarps * tok - 1) / (kWarps * tok));
  auto* kern = tok == 4 ? latent_append_kernel<4> : (tok == 2 ? latent_append_kernel<2> : latent_append_kernel<1>);
  const cudaError_t e = launch_pdl(kern, dim3(blocks), dim3(kWarps * 32), 0, s, *a, status);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
