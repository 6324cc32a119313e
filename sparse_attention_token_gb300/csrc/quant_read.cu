// quant_read.cu -- rows of the quantised latent cache back to bf16, gathered from the pages of requests.
//
//     c_kv[t] = 2^E * codes,  k_rope[t] = 2^E * (the row's rotary part),  t = cu_lens[b] + i, position starts[b] + i
//
// Every value is exact in bf16 (the scale is a power of two, a code's value an e4m3 number).
// A warp takes a row; lane i decodes the values 8 i .. 8 i + 7 and 256 + 8 i .. 256 + 8 i + 7, so that loads
// and stores are dense.  Bound by HBM: 203135 rows in 8 bits, 367 MB of rows and values, in 62.7 us, 86 % of the copy bandwidth;
// as many in 4 bits, 319 MB, in 60.4 (78 %); one request of some 1000 rows takes 2.8 us, which is latency (launch, offsets,
// table, row, store).
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"
#include "quant_rows.cuh"

namespace dsa {
namespace {

using namespace quant;

constexpr int kWarps = 4;

__device__ __forceinline__ uint4 values8(uint2 codes, float scale) {
  const float2 a = from_e4m3x2(codes.x & 0xFFFFu), b = from_e4m3x2(codes.x >> 16);
  const float2 c = from_e4m3x2(codes.y & 0xFFFFu), d = from_e4m3x2(codes.y >> 16);
  return make_uint4(pack_bf16(a.x * scale, a.y * scale), pack_bf16(b.x * scale, b.y * scale),
                    pack_bf16(c.x * scale, c.y * scale), pack_bf16(d.x * scale, d.y * scale));
}

template <bool FP4>
__global__ void __launch_bounds__(kWarps * 32) quant_read_kernel(const dsa_mla_quant_read_args a, unsigned* status) {
  constexpr int kRow = FP4 ? kRow4 : kRow8;
  const int lane = threadIdx.x & 31;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int t = static_cast<int>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= a.total || t >= __ldg(a.cu_lens + a.B)) return;
  const int b = sequence_of(a.cu_lens, a.B, t), first = __ldg(a.cu_lens + b);
  if (t < first) return;
  const long long pos = static_cast<long long>(t) - first + (a.starts ? __ldg(a.starts + b) : 0);
  const long long lp = pos / a.page_size;
  const int page = pos >= 0 && lp < a.max_pages_per_seq
                       ? __ldg(a.block_tables + static_cast<long long>(b) * a.max_pages_per_seq + lp) : -1;
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0) atomicOr(status, kStatusBadPage);
    return;
  }
  const uint8_t* row = static_cast<const uint8_t*>(a.cache) + (static_cast<long long>(page) * a.page_size + pos % a.page_size) * kRow;
  uint2 lo, hi;
  float scale;
  if (FP4) {
    const uint32_t* words = reinterpret_cast<const uint32_t*>(row);
    const uint32_t w0 = __ldg(words + lane), w1 = __ldg(words + 32 + lane);
    const int byte = __ldg(row + kScale4 + lane);
    scale = pow2f(static_cast<int>(__ballot_sync(0xffffffffu, byte >> 7) & 0xFFu) - 128);
    const int s0 = __shfl_sync(0xffffffffu, byte, lane >> 1) & 127, s1 = __shfl_sync(0xffffffffu, byte, 16 + (lane >> 1)) & 127;
    lo = codes4_to_e4m3(w0, levels_at(levels_base(s0 & 7), s0));
    hi = codes4_to_e4m3(w1, levels_at(levels_base(s1 & 7), s1));
  } else {
    lo = __ldg(reinterpret_cast<const uint2*>(row) + lane);
    hi = __ldg(reinterpret_cast<const uint2*>(row) + 32 + lane);
    scale = __ldg(reinterpret_cast<const float*>(row + kScale8));
  }
  uint4* out_c = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.c_kv) + t * a.c_stride);
  out_c[lane] = values8(lo, scale);
  out_c[32 + lane] = values8(hi, scale);
  const uint32_t r = __ldg(reinterpret_cast<const uint32_t*>(row + (FP4 ? kRope4 : kRope8)) + lane);
  reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.k_rope) + t * a.r_stride)[lane] =
      pack_bf16(__uint_as_float(r << 16) * scale, __uint_as_float(r & 0xFFFF0000u) * scale);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_mla_quant_read(const dsa_mla_quant_read_args* a, dsa_stream_t stream) {
  if (!a) return DSA_ERR_INVALID_ARGUMENT;
  if (a->B < 0 || a->total < 0 || a->page_size <= 0 || a->num_pages < 0 || a->max_pages_per_seq < 0 || a->kv_rank <= 0 ||
      a->rope_dim < 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (a->kv_rank != quant::kRank || a->rope_dim != quant::kRope || quant::row_bytes(a->format) == 0)
    return DSA_ERR_UNSUPPORTED;
  if (a->total == 0 || a->B == 0) return DSA_OK;
  if ((!a->cache && a->num_pages > 0) || !a->cu_lens || !a->c_kv || !a->k_rope || (!a->block_tables && a->max_pages_per_seq > 0))
    return DSA_ERR_INVALID_ARGUMENT;
  // (rows that lie over one another would be written by two warps)
  if (a->total > 1 && (a->c_stride < quant::kRank || a->r_stride < quant::kRope || a->c_stride % 8 != 0 || a->r_stride % 8 != 0))
    return DSA_ERR_INVALID_ARGUMENT;
  auto al = [](const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  if (!al(a->cache, 16) || !al(a->c_kv, 16) || !al(a->k_rope, 16) || !al(a->block_tables, 4) || !al(a->cu_lens, 4) ||
      !al(a->starts, 4))
    return DSA_ERR_INVALID_ARGUMENT;
  unsigned* status = device_status_ptr();
  if (!status) return DSA_ERR_CUDA;
  const unsigned blocks = (static_cast<unsigned>(a->total) + kWarps - 1) / kWarps;
  auto* kern = a->format == DSA_FP4_E2M1 ? quant_read_kernel<true> : quant_read_kernel<false>;
  const cudaError_t e = launch_pdl(kern, dim3(blocks), dim3(kWarps * 32), 0, reinterpret_cast<cudaStream_t>(stream), *a, status);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
