// page_plan.cu -- block tables, slot mapping, positions and query offsets from request lengths.
//
// With c_b = seq_b - q_b tokens cached before the step, F shared prefix pages and page size P:
//     held_b = max(ceil(c_b / P), F),  have_b = max(ceil(seq_b / P), F),  new_b = have_b - held_b
//     first_b = sum_{i<b} new_i,  cu_b = sum_{i<b} q_i
//     table[b, j] = prefix[j] (j < F), unchanged (j < held_b), free[first_b + j - held_b] (j < have_b), -1
//     token cu_b + i: position p = c_b + i, slot = table[b, p / P] * P + p % P
//
// One launch and no pass between CTAs: a CTA owns up to 256 requests (grid.x), sums the
// lengths of all requests before them itself (two integers a request, L2 hits), scans its
// own, and writes one slice (grid.y) of their table entries and of their tokens.  A slot
// takes its page from the formula above and not from the table, so no CTA waits for another.
// Latency bound: three trips to L2 one after another (lengths, table or free list, stores).  64
// requests with one new token each and tables of 1024 take 3.4 us, 16 with 56162 new tokens 4.1 us,
// 1024 with tables of 4352 (4.5 M entries, 9 MB that change) 8.3 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "dsa_indexer.h"
#include "internal.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kPlanThreads = 256;  // one request per thread in the scan

struct Request {
  int seq, q, held, have;
};

// Lengths of request b, clamped to what the table can hold.
__device__ __forceinline__ Request request(const dsa_page_plan_args& a, int b, bool* bad) {
  const long long room = static_cast<long long>(a.max_pages_per_seq) * a.page_size;
  const int seq0 = __ldg(a.seq_lens + b), q0 = __ldg(a.q_lens + b);
  Request r;
  r.seq = static_cast<int>(min(static_cast<long long>(max(seq0, 0)), room));
  r.q = min(max(q0, 0), r.seq);
  *bad = r.seq != seq0 || r.q != q0;
  const int c = r.seq - r.q;
  const int f = r.seq > 0 ? min(a.num_prefix_pages, a.max_pages_per_seq) : 0;
  // ceil without the sum c + P - 1, which passes 32 bits at the largest lengths
  r.held = max(c / a.page_size + (c % a.page_size != 0), f);
  r.have = max(r.seq / a.page_size + (r.seq % a.page_size != 0), f);
  return r;
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const dsa_page_plan_args a, unsigned* status) {
  __shared__ long long wsum_q[8], wsum_n[8];
  __shared__ long long s_cu[kPlanThreads + 1];
  __shared__ long long s_first[kPlanThreads];
  __shared__ int s_held[kPlanThreads], s_have[kPlanThreads], s_cached[kPlanThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int b0 = blockIdx.x * kPlanThreads;
  const int nb = min(kPlanThreads, a.B - b0);

  // what the requests before b0 take
  long long pq = 0, pn = 0;
  bool bad;
#pragma unroll 4
  for (int b = tid; b < b0; b += kPlanThreads) {
    const Request r = request(a, b, &bad);
    pq += r.q;
    pn += r.have - r.held;
  }
  pq = warp_sum(pq);
  pn = warp_sum(pn);
  if (lane == 0) {
    wsum_q[warp] = pq;
    wsum_n[warp] = pn;
  }
  Request r{0, 0, 0, 0};
  bad = false;
  if (tid < nb) r = request(a, b0 + tid, &bad);
  if (bad && blockIdx.y == 0) atomicOr(status, kStatusUncovered);
  __syncthreads();
  long long base_q = 0, base_n = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    base_q += wsum_q[w];
    base_n += wsum_n[w];
  }
  __syncthreads();
  // inclusive scan over the CTA's requests
  long long sq = r.q, sn = r.have - r.held;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long uq = __shfl_up_sync(0xffffffffu, sq, o), un = __shfl_up_sync(0xffffffffu, sn, o);
    if (lane >= o) {
      sq += uq;
      sn += un;
    }
  }
  if (lane == 31) {
    wsum_q[warp] = sq;
    wsum_n[warp] = sn;
  }
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    sq += wsum_q[w];
    sn += wsum_n[w];
  }
  sq += base_q;
  sn += base_n;
  if (tid == 0) s_cu[0] = base_q;
  s_cu[tid + 1] = sq;
  s_first[tid] = sn - (r.have - r.held);
  s_held[tid] = r.held;
  s_have[tid] = r.have;
  s_cached[tid] = r.seq - r.q;
  if (blockIdx.y == 0 && tid < nb) {
    a.cu_q_lens[b0 + tid + 1] = static_cast<int32_t>(min(sq, static_cast<long long>(a.total_q)));
    if (b0 + tid == 0) a.cu_q_lens[0] = 0;
    if (b0 + tid == a.B - 1) {
      a.used[0] = static_cast<int32_t>(min(sn, 0x7FFFFFFFLL));
      if (sn > a.num_free) atomicOr(status, kStatusUncovered);
      if (sq > a.total_q) atomicOr(status, kStatusUncovered);
    }
  }
  __syncthreads();

  // page at entry j of the CTA's request i, j < have
  auto page_at = [&](int i, int j) -> int {
    if (j < a.num_prefix_pages) return __ldg(a.prefix_pages + j);
    if (j < s_held[i]) return a.block_tables[static_cast<long long>(b0 + i) * a.max_pages_per_seq + j];
    const long long f = s_first[i] + (j - s_held[i]);
    return f < a.num_free ? __ldg(a.free_pages + f) : -1;
  };

  // table entries: four at a time when rows are 16-byte aligned; entries that stay are not touched
  const int W = a.max_pages_per_seq;
  const int vec = (W % 4 == 0 && (reinterpret_cast<uintptr_t>(a.block_tables) & 15u) == 0) ? 4 : 1;
  const int per_row = W / vec;
  const long long step = static_cast<long long>(gridDim.y) * kPlanThreads;
  // (i, j) advance by step without a division an entry
  const int step_i = per_row > 0 ? static_cast<int>(step / per_row) : 0;
  const int step_j = per_row > 0 ? static_cast<int>(step - static_cast<long long>(step_i) * per_row) : 0;
  const int start = blockIdx.y * kPlanThreads + tid;
  int i = per_row > 0 ? start / per_row : nb, j = per_row > 0 ? start - i * per_row : 0;
  for (; i < nb; i += step_i, j += step_j) {
    if (j >= per_row) {
      j -= per_row;
      if (++i >= nb) break;
    }
    const int j0 = j * vec;
    int32_t* row = a.block_tables + static_cast<long long>(b0 + i) * W;
    const int held = s_held[i], have = s_have[i];
    const int f = have > 0 ? min(a.num_prefix_pages, W) : 0;  // have = 0: an empty request
    if (vec == 4 && j0 >= have) {
      *reinterpret_cast<int4*>(row + j0) = make_int4(-1, -1, -1, -1);
      continue;
    }
    for (int e = j0; e < j0 + vec; ++e) {
      if (e >= f && e < held) continue;
      row[e] = e < have ? page_at(i, e) : -1;
    }
  }

  // tokens
  const long long t_end = min(s_cu[nb], static_cast<long long>(a.total_q));
  for (long long t = s_cu[0] + static_cast<long long>(blockIdx.y) * kPlanThreads + tid; t < t_end; t += step) {
    int lo = 0, hi = nb;  // the request: the last i with cu[i] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_cu[mid] <= t) lo = mid; else hi = mid;
    }
    const int p = s_cached[lo] + static_cast<int>(t - s_cu[lo]);
    const int j = p / a.page_size;
    const int pg = page_at(lo, j);
    if (pg < 0) atomicOr(status, kStatusBadPage);
    a.positions[t] = p;
    a.slot_mapping[t] = pg < 0 ? -1 : static_cast<long long>(pg) * a.page_size + (p - j * a.page_size);
  }
  // padding after the last token
  if (blockIdx.x == gridDim.x - 1) {
    for (long long t = s_cu[nb] + static_cast<long long>(blockIdx.y) * kPlanThreads + tid; t < a.total_q; t += step) {
      a.positions[t] = -1;
      a.slot_mapping[t] = -1;
    }
  }
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_page_plan(const dsa_page_plan_args* a, dsa_stream_t stream) {
  if (!a) return DSA_ERR_INVALID_ARGUMENT;
  if (a->B < 0 || a->total_q < 0 || a->page_size <= 0 || a->max_pages_per_seq < 0 || a->num_prefix_pages < 0 ||
      a->num_free < 0 || a->num_prefix_pages > a->max_pages_per_seq)
    return DSA_ERR_INVALID_ARGUMENT;
  if (!a->cu_q_lens || !a->used || (a->num_prefix_pages > 0 && !a->prefix_pages) || (a->num_free > 0 && !a->free_pages) ||
      (a->total_q > 0 && (!a->slot_mapping || !a->positions)))
    return DSA_ERR_INVALID_ARGUMENT;
  if (a->B > 0 && (!a->q_lens || !a->seq_lens || (a->max_pages_per_seq > 0 && !a->block_tables)))
    return DSA_ERR_INVALID_ARGUMENT;
  auto al = [](const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  if (!al(a->q_lens, 4) || !al(a->seq_lens, 4) || !al(a->prefix_pages, 4) || !al(a->free_pages, 4) ||
      !al(a->block_tables, 4) || !al(a->cu_q_lens, 4) || !al(a->slot_mapping, 8) || !al(a->positions, 4) ||
      !al(a->used, 4))
    return DSA_ERR_INVALID_ARGUMENT;
  unsigned* status = device_status_ptr();
  if (!status) return DSA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a->B == 0) {  // no request: offsets and count of zero, padding only
    if (cudaMemsetAsync(a->cu_q_lens, 0, 4, s) != cudaSuccess || cudaMemsetAsync(a->used, 0, 4, s) != cudaSuccess)
      return DSA_ERR_CUDA;
    if (a->total_q > 0 &&
        (cudaMemsetAsync(a->slot_mapping, 0xFF, sizeof(int64_t) * a->total_q, s) != cudaSuccess ||
         cudaMemsetAsync(a->positions, 0xFF, sizeof(int32_t) * a->total_q, s) != cudaSuccess))
      return DSA_ERR_CUDA;
    return DSA_OK;
  }
  const int nx = (a->B + kPlanThreads - 1) / kPlanThreads;
  // Slices: about one unit (four table entries or one token) a thread, at most four CTAs an SM.
  // Of 2048, 1024, 512, 256 units a CTA the first of the cases above took 6.2, 4.6, 3.7, 3.3 us, the
  // last 9.7, 8.3, 8.3, 8.3 us; with eight CTAs an SM the last took 10.5 us.
  const long long units = static_cast<long long>(a->B) * ((a->max_pages_per_seq + 3) / 4) + a->total_q;
  const long long want = (units + 255) / 256;
  const int ny = static_cast<int>(std::max(1LL, std::min(want, 608LL) / nx));
  const cudaError_t e = launch_pdl(page_plan_kernel, dim3(nx, ny), dim3(kPlanThreads), 0, s, *a, status);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
