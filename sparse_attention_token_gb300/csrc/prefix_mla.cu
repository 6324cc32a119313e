// prefix_mla.cu -- latent attention for a batch whose sequences share their first tokens.
//
//     logit[t, h, s] = scale * (q_nope[t, h] . c_kv[s] + q_rope[t, h] . k_rope[s]),  s <= p(t)
//     out[t, h]      = sum_s softmax_s(logit[t, h, :]) c_kv[s],   lse[t, h] = ln sum_s exp(logit[t, h, s])
//
// Three launches.
//
// plan (one CTA): the (query, head) rows are cut into tiles of up to 64 rows, and every tile's
// keys into blocks of 64.  A request of 64 rows or more fills tiles of its own, which walk the
// prefix and then the request's keys.  Smaller requests (few heads, one query) share: tiles
// packed across requests walk the prefix, further tiles, one request each, walk its own keys,
// and the two are joined.  The blocks of all tiles stand in one line, cut into equal parts,
// one per SM: a part may start and end inside a tile, so one long prefix fills every SM.
//
// attend (one CTA per SM): for each piece of a tile in its part
//   warp 4      keys: one TMA box per page piece and 128-byte column, one lane a box, into a ring
//               of two tiles of 64 keys (9 columns of 64 bf16, 128-byte swizzle);
//   warps 5..7  the piece's query rows (16-byte cp.async, any strides);
//   warp 8      TMEM; lane 0 issues  S [rows x 64 keys] = Q . K^T  (M = 128 lanes, 64 used) and
//               O^T [512 x rows] += V^T . P^T (4 x M = 128, the key tile read MN-major), the next
//               block's S ahead of this block's P . V;
//   warps 0..3  softmax with a reference maximum that moves only when a block's maximum passes it
//               by 8 (a factor 256), P as bf16, rescaling of O^T, and the piece's result.
// A tile done in one piece is normalised and written; the others leave (O, m, l) in fp32.
//
// join: out = sum_j 2^(m_j - M) O_j / sum_j 2^(m_j - M) l_j over a row's pieces, in their order.
//
// Every wait is bounded; after one gives up, every role stops, copies and MMAs in flight are
// drained (bounded) and TMEM is freed.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "dsa_indexer.h"
#include "internal.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kRank = 512, kRope = 64, kAtoms = 9;        // 576 = 9 columns of 64 bf16
constexpr int kRows = 64;                                 // rows per tile
constexpr int kKeys = 64;                                 // keys per block
constexpr int kThreads = 288;                             // warps 0-3 softmax, 4 keys, 5-7 queries, 8 MMA
constexpr uint32_t kAtomBytes = 64 * 128;                 // one column of 64 rows or keys
constexpr uint32_t kTileBytes = kAtoms * kAtomBytes;      // 73728
constexpr uint32_t kOffQ = 0, kOffTile = kTileBytes, kOffP = kOffTile + 2 * kTileBytes;
constexpr uint32_t kOffMisc = kOffP + kRows * 128;        // P: 64 rows x 64 keys bf16
constexpr size_t kSmem = kOffMisc + 1024;
constexpr uint32_t kOCol0 = 2 * kKeys;                    // O^T behind the two S buffers
constexpr float kLn2 = 0.6931471805599453f;

struct Tile {
  int row0, nrows;   // rows t * H + h
  int b;             // request, -1: rows of several requests (prefix only)
  int n_pre;         // blocks of the prefix; the rest are the request's own
  int limit;         // the most keys any of its rows sees
  int pad[3];
};

struct Args {
  int B, total_q, H, page_size, num_pages, max_pages, prefix_len, num_prefix_pages;
  int packed;              // small requests: prefix tiles packed across requests
  int max_tiles, G;        // tiles there is room for; CTAs (parts)
  int past_row;            // a row coordinate past the cache: copies from there are zeros
  float scale_log2;        // scale * log2(e)
  const __nv_bfloat16 *qn, *qr;
  long long qn_t, qn_h, qr_t, qr_h;
  const int32_t *prefix_pages, *block_tables, *cu, *lens;
  __nv_bfloat16* out;
  float* lse;
  Tile* tiles;
  long long* u0;           // [max_tiles + 1] first block of each tile in the line of all blocks
  int* head;               // [0] tiles, [1] packed prefix tiles, [2 + b] first own tile of request b
  float *part_o, *part_ml; // pieces: [slot][64][512], [slot][64][2]
  unsigned* status;
};

struct Bars {
  uint64_t qfull, qempty, tfull[2], tempty[2], sfull[2], sempty[2], pfull, ofree, done;
};

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Request of query t: the last b with cu[b] <= t.
__device__ __forceinline__ int request_of(const Args& a, int t) {
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.cu + mid) <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Keys that query t of request b sees, cut to what the table covers (and counted as bad then).
__device__ __forceinline__ int sees(const Args& a, int b, int t, bool* bad) {
  const int q0 = __ldg(a.cu + b), q1 = __ldg(a.cu + b + 1);
  if (t < q0 || t >= q1) return 0;
  long long n = static_cast<long long>(__ldg(a.lens + b)) - (q1 - q0) + (t - q0) + 1;
  const long long room = max(static_cast<long long>(a.max_pages) * a.page_size, static_cast<long long>(a.prefix_len));
  if (n > room) {
    *bad = true;
    n = room;
  }
  return static_cast<int>(max(n, 0LL));
}

// ------------------------------------------------------------------ plan
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ long long block_scan(long long v, long long* wsum, long long* total) {  // exclusive
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();
  if (lane == 31) wsum[warp] = s;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll 8
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const long long x = wsum[w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return before + s - v;
}

__global__ void __launch_bounds__(kPlanThreads) prefix_mla_plan_kernel(const Args a) {
  __shared__ long long wsum[32];
  const int tid = threadIdx.x;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  // rows beyond the last request (padding) count as one more request that sees nothing
  const int n_pre_tiles = a.packed ? (a.total_q * a.H + kRows - 1) / kRows : 0;
  int base = n_pre_tiles;
  const int nreq = a.packed ? a.B : a.B + 1;
  for (int b0 = 0; b0 < nreq; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < nreq) {
      const int q0 = min(max(__ldg(a.cu + b), 0), a.total_q);
      const int q1 = b < a.B ? min(max(__ldg(a.cu + b + 1), q0), a.total_q) : a.total_q;
      n = (static_cast<int>(q1 - q0) * a.H + kRows - 1) / kRows;
    }
    long long total;
    const long long at = block_scan(n, wsum, &total);
    if (b < nreq) a.head[2 + b] = base + static_cast<int>(at);
    base += static_cast<int>(total);
    __syncthreads();
  }
  const int n_tiles = min(base, a.max_tiles);
  if (tid == 0) {
    a.head[0] = n_tiles;
    a.head[1] = n_pre_tiles;
    a.head[2 + nreq] = base;
  }
  __syncthreads();
  const int kO = a.prefix_len / kKeys;  // first block with own keys
  long long u = 0;
  bool bad = false;
  for (int i0 = 0; i0 < n_tiles; i0 += kPlanThreads) {
    const int i = i0 + tid;
    long long units = 0;
    if (i < n_tiles) {
      Tile t{};
      int own = 0;
      if (i < n_pre_tiles) {
        t.row0 = i * kRows;
        t.nrows = min(kRows, a.total_q * a.H - t.row0);
        t.b = -1;
        const int tq0 = t.row0 / a.H, tq1 = (t.row0 + t.nrows - 1) / a.H;
        int b = request_of(a, tq0);
        for (int q = tq0; q <= tq1; ++q) {
          while (b + 1 < a.B && __ldg(a.cu + b + 1) <= q) ++b;
          t.limit = max(t.limit, sees(a, b, q, &bad));
        }
      } else {
        int lo = 0, hi = nreq;  // the last b with head[2 + b] <= i
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (a.head[2 + mid] <= i) lo = mid; else hi = mid;
        }
        const int q0 = min(max(__ldg(a.cu + lo), 0), a.total_q);
        const int q1 = lo < a.B ? min(max(__ldg(a.cu + lo + 1), q0), a.total_q) : a.total_q;
        t.row0 = q0 * a.H + (i - a.head[2 + lo]) * kRows;
        t.nrows = min(kRows, q1 * a.H - t.row0);
        t.b = min(lo, a.B - 1);
        t.limit = lo < a.B ? sees(a, lo, (t.row0 + t.nrows - 1) / a.H, &bad) : 0;
        own = t.limit > a.prefix_len ? (t.limit + kKeys - 1) / kKeys - kO : 0;
      }
      t.n_pre = (a.packed && i >= n_pre_tiles) ? 0 : (min(t.limit, a.prefix_len) + kKeys - 1) / kKeys;
      units = t.n_pre + own;
      a.tiles[i] = t;
    }
    long long total;
    const long long at = block_scan(units, wsum, &total);
    if (i < n_tiles) a.u0[i] = u + at;
    u += total;
    __syncthreads();
  }
  if (tid == 0) a.u0[n_tiles] = u;
  if (bad) atomicOr(a.status, kStatusUncovered);
}

// The line of U blocks in G = min(CTAs, U) parts, none of them empty: part c is
// [c U / G, (c + 1) U / G).
__device__ __forceinline__ int parts(const Args& a, long long U) {
  return static_cast<int>(min(static_cast<long long>(a.G), U));
}
__device__ __forceinline__ long long part_begin(long long U, int G, int c) { return U * c / G; }
__device__ __forceinline__ int part_of(long long U, int G, long long u) {
  return static_cast<int>(((u + 1) * G - 1) / U);
}
// Where a piece of tile i in part c leaves its result: pieces that begin inside a tile are the
// first of their part, those that only end inside one the last, so two slots a part hold them;
// whole tiles come behind (they leave one only where rows are joined over two tiles).
__device__ __forceinline__ long long piece_slot(int G, int c, int i, bool at_start, bool whole) {
  return whole ? 2LL * G + i : 2LL * c + (at_start ? 1 : 0);
}

// Last tile i with u0[i] <= u, all lanes of a warp probing: a factor 32 a step.
__device__ __forceinline__ int find_tile(const long long* u0, int n, long long u) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // u0[lo] <= u, u < u0[hi] (u0[n] = U)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int p = min(lo + lane * step, hi - 1);
    const unsigned m = __ballot_sync(0xffffffffu, __ldcg(u0 + p) <= u);
    const int last = 31 - __clz(m);  // lane 0 always holds
    const int nlo = min(lo + last * step, hi - 1);
    hi = last == 31 ? hi : min(lo + (last + 1) * step, hi);
    lo = nlo;
  }
  return lo;
}

// ------------------------------------------------------------------ attend
__global__ void __launch_bounds__(kThreads, 1) prefix_mla_kernel(const __grid_constant__ CUtensorMap tmap_c,
                                                                  const __grid_constant__ CUtensorMap tmap_r,
                                                                  const Args a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((ptx::smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusSmemAlign);
    return;
  }
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffMisc);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + kOffMisc + 128);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 132);
  volatile int* first_tile = reinterpret_cast<volatile int*>(smem + kOffMisc + 136);
  volatile unsigned* kmask = reinterpret_cast<volatile unsigned*>(smem + kOffMisc + 144);  // [2] 16-key pieces there
  float* corr = reinterpret_cast<float*>(smem + kOffMisc + 256);                          // [64]

  if (threadIdx.x == 0) {
    ptx::mbar_init(&bars->qfull, 96);
    ptx::mbar_init(&bars->qempty, 1);
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&bars->tfull[s], 1);
      ptx::mbar_init(&bars->tempty[s], 1);
      ptx::mbar_init(&bars->sfull[s], 1);
      ptx::mbar_init(&bars->sempty[s], 2);   // the two row warps
    }
    ptx::mbar_init(&bars->pfull, 4);
    ptx::mbar_init(&bars->ofree, 1);
    ptx::mbar_init(&bars->done, 1);
    *abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 8) {
    ptx::tmem_alloc(tmem_holder, 512);
    ptx::tmem_relinquish();
  }
  if (warp == 4 && lane == 0) {
    ptx::prefetch_tmap(&tmap_c);
    ptx::prefetch_tmap(&tmap_r);
  }
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int n_tiles = __ldcg(a.head);
  const long long U = __ldcg(a.u0 + n_tiles);
  const int c = blockIdx.x, G = parts(a, U);
  const long long u_lo = c < G ? part_begin(U, G, c) : 0, u_hi = c < G ? part_begin(U, G, c + 1) : 0;
  if (warp == 0 && u_lo < u_hi) {
    const int i = find_tile(a.u0, n_tiles, u_lo);
    if (lane == 0) *first_tile = i;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int i_first = u_lo < u_hi ? *first_tile : 0;
  const int kO = a.prefix_len / kKeys;

  // The part's pieces: tile i, its blocks [k0, k1).  Every role walks the same list.
  struct Piece {
    int i, k0, k1;
    long long u;   // first block of the piece in the line
  };
  auto next_piece = [&](Piece& p, long long u, Tile& t) -> bool {
    if (u >= u_hi) return false;
    long long b0 = __ldcg(a.u0 + p.i), b1 = __ldcg(a.u0 + p.i + 1);
    while (b1 <= u) {  // tiles without blocks, and the one just done
      ++p.i;
      b0 = b1;
      b1 = __ldcg(a.u0 + p.i + 1);
    }
    p.u = u;
    p.k0 = static_cast<int>(u - b0);
    p.k1 = static_cast<int>(min(b1, u_hi) - b0);
    const int4 w = __ldcg(reinterpret_cast<const int4*>(a.tiles + p.i));
    t.row0 = w.x;
    t.nrows = w.y;
    t.b = w.z;
    t.n_pre = w.w;
    t.limit = __ldcg(reinterpret_cast<const int*>(a.tiles + p.i) + 4);
    return true;
  };

  if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t sbase = ptx::smem_u32(smem);
      const uint32_t id1 = ptx::idesc_f32acc(128, kKeys, true);        // S: 128 lanes (64 rows) x 64 keys
      bool ok = true;
      uint32_t n1 = 0, n2 = 0;  // blocks whose S / P . V was issued, over all pieces
      uint32_t seg = 0;
      Piece p{i_first, 0, 0, 0};
      Tile t;
      uint64_t t0 = ptx::globaltimer();
      for (long long u = u_lo; ok && next_piece(p, u, t); u = p.u + (p.k1 - p.k0), ++seg) {
        const uint32_t id2 = ptx::idesc_f32acc_bf16_amn(128, (t.nrows + 15) / 16 * 16);  // O^T: 128 latent x rows
        if (!ptx::mbar_wait(&bars->qfull, seg & 1, abort, a.status, kStatusTimeout)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t s_begin = n1, s_end = n1 + (p.k1 - p.k0);
        // Issue whichever product has its inputs first: the next block's S or this block's P . V.
        t0 = ptx::globaltimer();
        for (uint32_t spin = 0; ok && n2 < s_end; ++spin) {
          bool progress = false;
          if (n1 < s_end && n1 <= n2 + 1 && ptx::mbar_try_wait(&bars->tfull[n1 & 1], (n1 >> 1) & 1) &&
              ptx::mbar_try_wait(&bars->sempty[n1 & 1], ((n1 >> 1) & 1) ^ 1)) {
            ptx::tc_fence_after();
            const int tb = n1 & 1;
            const uint32_t d = tmem_base + tb * kKeys;
            const uint64_t ad0 = ptx::sw128_kmajor_desc(sbase + kOffQ);
            const uint64_t bd0 = ptx::sw128_kmajor_desc(sbase + kOffTile + tb * kTileBytes);
#pragma unroll
            for (int j = 0; j < kAtoms * 4; ++j) {
              const uint64_t off = ((j >> 2) * kAtomBytes + (j & 3) * 32) >> 4;
              ptx::mma_bf16(d, ad0 + off, bd0 + off, id1, j > 0 ? 1u : 0u);
            }
            ptx::mma_commit(&bars->sfull[tb]);
            if (n1 + 1 == s_end) ptx::mma_commit(&bars->qempty);
            ++n1;
            progress = true;
          }
          if (n2 < n1 && ptx::mbar_try_wait(&bars->pfull, n2 & 1)) {
            ptx::tc_fence_after();
            const int tb = n2 & 1;
            const uint64_t ad0 = ptx::sw128_mnmajor_desc(sbase + kOffTile + tb * kTileBytes, kAtomBytes);
            const uint64_t bd0 = ptx::sw128_kmajor_desc(sbase + kOffP);
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {  // latent 128 cc .. + 127: columns 2 cc and 2 cc + 1
#pragma unroll
              for (int s = 0; s < 4; ++s)     // 16 keys per MMA: two 8-key groups of 1024 bytes
                ptx::mma_bf16(tmem_base + kOCol0 + cc * kRows, ad0 + ((2 * cc * kAtomBytes + s * 2048) >> 4),
                              bd0 + 2 * s, id2, (n2 > s_begin || s > 0) ? 1u : 0u);
            }
            ptx::mma_commit(&bars->tempty[tb]);
            ptx::mma_commit(&bars->ofree);
            ++n2;
            progress = true;
          }
          if (progress) {
            t0 = ptx::globaltimer();
          } else if ((spin & 15u) == 15u) {
            if (*abort) ok = false;
            else if (ptx::globaltimer() - t0 > 2000000000ull) {
              *abort = 1;
              atomicOr(a.status, kStatusTimeout);
              ok = false;
            }
          }
        }
      }
      ptx::mma_commit(&bars->done);
      ptx::mbar_wait_drain(&bars->done, 0, a.status, kStatusTimeout, 200000000ull);
    }
    __syncwarp();
  } else if (warp == 4) {
    // ------------------------------------------------------------ keys
    const int box = min(a.page_size, kKeys), per = kKeys / box;  // boxes per column
    uint32_t n = 0;
    bool ok = true;
    Piece p{i_first, 0, 0, 0};
    Tile t;
    uint32_t issued = 0;
    for (long long u = u_lo; ok && next_piece(p, u, t); u = p.u + (p.k1 - p.k0)) {
      const int32_t* own = a.block_tables + static_cast<long long>(max(t.b, 0)) * a.max_pages;
      for (int k = p.k0; k < p.k1; ++k, ++n) {
        const bool pre = k < t.n_pre;
        const int s0 = (pre ? k : k - t.n_pre + kO) * kKeys;  // first position of the block
        // lane j < per: the page of keys [s0 + j box, + box)
        const int lo = pre ? 0 : a.prefix_len, hi = pre ? min(t.limit, a.prefix_len) : t.limit;
        const int sj = s0 + (lane & (per - 1)) * box;
        const int pj = sj / a.page_size;
        const bool want = sj < hi && sj + box > lo;  // some row of the tile may see a key here
        int pg = -1;
        if (want) pg = pre ? (pj < a.num_prefix_pages ? __ldg(a.prefix_pages + pj) : -1)
                           : (pj < a.max_pages ? __ldg(own + pj) : -1);
        const bool there = want && pg >= 0 && pg < a.num_pages;
        if (want && !there) atomicOr(a.status, kStatusBadPage);
        // a page that is not there: a row past the cache, which the copy fills with zeros
        const int row = there ? pg * a.page_size + (sj & (a.page_size - 1)) : a.past_row;
        const unsigned m = __ballot_sync(0xffffffffu, there) & ((1u << per) - 1u);
        const int st = n & 1;
        int good = 1;
        if (lane == 0) good = ptx::mbar_wait(&bars->tempty[st], ((n >> 1) & 1) ^ 1, abort, a.status, kStatusTimeout);
        good = __shfl_sync(0xffffffffu, good, 0);
        if (!good) {
          ok = false;
          break;
        }
        if (lane == 0) {
          kmask[st] = m;
          ptx::mbar_arrive_expect_tx(&bars->tfull[st], kTileBytes);
        }
        __syncwarp();
        uint8_t* tile = smem + kOffTile + st * kTileBytes;
        for (int e0 = 0; e0 < kAtoms * per; e0 += 32) {
          const int e = e0 + lane;
          const int j = e & (per - 1), at = e / per;
          const int r = __shfl_sync(0xffffffffu, row, j);
          if (at < kAtoms) {
            uint8_t* dst = tile + at * kAtomBytes + j * box * 128;
            if (at < 8) ptx::tma_load_2d(dst, &tmap_c, &bars->tfull[st], at * 64, r);
            else ptx::tma_load_2d(dst, &tmap_r, &bars->tfull[st], 0, r);
          }
        }
        ++issued;
      }
    }
    // every copy lands before the CTA can exit, whatever happened
    if (lane == 0) {
      for (uint32_t q = issued > 2 ? issued - 2 : 0; q < issued; ++q)
        ptx::mbar_wait_drain(&bars->tfull[q & 1], (q >> 1) & 1, a.status, kStatusTimeout, 200000000ull);
    }
    __syncwarp();
  } else if (warp > 4) {
    // ------------------------------------------------------------ queries (96 threads)
    const int gt = threadIdx.x - 160;
    uint32_t seg = 0;
    Piece p{i_first, 0, 0, 0};
    Tile t;
    for (long long u = u_lo; next_piece(p, u, t); u = p.u + (p.k1 - p.k0), ++seg) {
      const bool good = ptx::mbar_wait(&bars->qempty, (seg & 1) ^ 1, abort, a.status, kStatusTimeout);
      if (!good) break;
      for (int e = gt; e < kRows * 72; e += 96) {
        const int r = e / 72, ch = e - r * 72;
        const int at = ch >> 3, c16 = ch & 7;
        const bool live = r < t.nrows;
        const int row = t.row0 + (live ? r : 0);
        const int tq = row / a.H, h = row - tq * a.H;
        const __nv_bfloat16* src = at < 8 ? a.qn + tq * a.qn_t + h * a.qn_h + at * 64 + c16 * 8
                                          : a.qr + tq * a.qr_t + h * a.qr_h + c16 * 8;
        ptx::cp_async_16(smem + kOffQ + at * kAtomBytes + r * 128 + ((c16 ^ (r & 7)) << 4), src, live ? 16u : 0u);
      }
      cp_async_wait_all();
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(&bars->qfull);
    }
  } else {
    // ------------------------------------------------------------ softmax, rescale, output (warps 0..3)
    const int h = threadIdx.x;                  // row of the tile (warps 0, 1) / latent lane within a chunk
    const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
    const bool row_lane = warp < 2;
    bool ok = true;
    uint32_t n = 0;
    Piece p{i_first, 0, 0, 0};
    Tile t;
    for (long long u = u_lo; next_piece(p, u, t); u = p.u + (p.k1 - p.k0)) {
      float m = -INFINITY, l = 0.f;
      int lim = 0;  // keys this row sees
      if (row_lane && h < t.nrows) {
        const int tq = (t.row0 + h) / a.H;
        bool bad = false;
        lim = min(sees(a, t.b >= 0 ? t.b : request_of(a, tq), tq, &bad), t.limit);
      }
      const int nr32 = (t.nrows + 31) / 32 * 32;
      if (threadIdx.x < 64) corr[threadIdx.x] = 1.f;
      for (int k = p.k0; k < p.k1; ++k, ++n) {
        const int tb = n & 1;
        const bool pre = k < t.n_pre;
        const int s0 = (pre ? k : k - t.n_pre + kO) * kKeys;
        const int klo = pre ? 0 : a.prefix_len, khi = pre ? min(t.limit, a.prefix_len) : t.limit;
        float cr = 1.f;
        if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars->sfull[tb], (n >> 1) & 1, abort, a.status,
                                                            kStatusTimeout)) != 0;
        // the copies have landed (S was computed from them); the wait orders kmask as well
        if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars->tfull[tb], (n >> 1) & 1, abort, a.status,
                                                            kStatusTimeout)) != 0;
        if (ok && (s0 < klo || s0 + kKeys > khi)) {
          // rows of the key tile that no row of this tile sees may hold anything: their weights
          // are 0, and the values become 0 so that the product is
          for (int e = threadIdx.x; e < kKeys * 64; e += 128) {
            const int key = e >> 6, ch = e & 63;
            if (s0 + key < klo || s0 + key >= khi)
              *reinterpret_cast<uint4*>(smem + kOffTile + tb * kTileBytes + (ch >> 3) * kAtomBytes + key * 128 +
                                        ((ch & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
          ptx::fence_proxy_async_smem();
        }
        if (row_lane) {
          if (ok) {
            ptx::tc_fence_after();
            uint32_t x0[32], x1[32];
            ptx::tmem_ld_32x32b_x32(tmem_base + lane_addr + tb * kKeys, x0);
            ptx::tmem_ld_32x32b_x32(tmem_base + lane_addr + tb * kKeys + 32, x1);
            ptx::tmem_ld_wait_regs(x0);
            ptx::tmem_ld_wait_regs(x1);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bars->sempty[tb]);
            float x[64];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              x[i] = __uint_as_float(x0[i]) * a.scale_log2;
              x[32 + i] = __uint_as_float(x1[i]) * a.scale_log2;
            }
            const int box = min(a.page_size, kKeys), per = kKeys / box;
            const unsigned km = kmask[tb];
            const int end = min(khi, lim);
            if (s0 < klo || s0 + kKeys > end || km != (1u << per) - 1u) {
#pragma unroll
              for (int i = 0; i < 64; ++i) {
                const int s = s0 + i;
                const bool v = s >= klo && s < end && ((km >> (i / box)) & 1u);
                x[i] = v ? x[i] : -INFINITY;
              }
            }
            float mb = -INFINITY;
#pragma unroll
            for (int i = 0; i < 64; ++i) mb = fmaxf(mb, x[i]);
            // The reference maximum moves only when the block's maximum exceeds it by more
            // than 8 (a factor 256 in probability): p stays below 256 and the output, which
            // divides by the sum taken against the same reference, is unchanged.
            float mn = m;
            if (m == -INFINITY) mn = mb;
            else if (mb > m + 8.f) mn = mb;
            cr = (m == -INFINITY || mn == m) ? 1.f : exp2f(m - mn);
            float ls = 0.f;
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float p0 = mn == -INFINITY ? 0.f : exp2f(x[2 * i] - mn);
              const float p1 = mn == -INFINITY ? 0.f : exp2f(x[2 * i + 1] - mn);
              ls += p0 + p1;
              const __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
              pk[i] = *reinterpret_cast<const uint32_t*>(&pb);
            }
            l = l * cr + ls;
            m = mn;
            // P is free once the previous block's P . V has completed
            if (n > 0)
              ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars->ofree, (n - 1) & 1, abort, a.status,
                                                          kStatusTimeout)) != 0;
            if (ok) {
              uint8_t* prow = smem + kOffP + h * 128;
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *reinterpret_cast<uint4*>(prow + ((q ^ (h & 7)) << 4)) =
                    make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
              corr[h] = cr;
            }
            ptx::fence_proxy_async_smem();
          }
        } else if (n > 0 && ok) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars->ofree, (n - 1) & 1, abort, a.status, kStatusTimeout)) != 0;
        }
        // P and the correction factors are written; does any row need its output rescaled?
        uint32_t any;
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.f32 q, %1, 0f3F800000;\n\t"
                     "bar.red.or.pred p, 2, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(any) : "f"(cr) : "memory");
        if (any && k > p.k0 && ok && !*abort) {
          ptx::tc_fence_after();
          for (int cc = 0; cc < 4; ++cc) {
            const uint32_t col = tmem_base + lane_addr + kOCol0 + cc * kRows;
            for (int h0 = 0; h0 < nr32; h0 += 32) {
              uint32_t r[32];
              ptx::tmem_ld_32x32b_x32(col + h0, r);
              ptx::tmem_ld_wait_regs(r);
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * corr[h0 + i]);
              ptx::tmem_st_32x32b_x32(col + h0, r);
            }
          }
          ptx::tmem_st_wait();
        }
        ptx::tc_fence_before();
        if (any) ptx::named_bar_sync(2, 128);  // corr is read by everyone before the next block rewrites it
        if (lane == 0) ptx::mbar_arrive(&bars->pfull);
      }
      // the piece's result
      const bool at_start = p.k0 == 0;
      const bool whole = at_start && p.u + (p.k1 - p.k0) == __ldcg(a.u0 + p.i + 1);
      const bool direct = whole && !a.packed;
      if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars->ofree, (n - 1) & 1, abort, a.status,
                                                          kStatusTimeout)) != 0;
      ptx::named_bar_sync(2, 128);  // corr was read for the last time
      const long long slot = piece_slot(a.G, c, p.i, at_start, whole) * kRows;
      if (row_lane && h < t.nrows) {
        corr[h] = l > 0.f ? 1.f / l : 0.f;
        if (direct) {
          if (a.lse) a.lse[t.row0 + h] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
        } else {
          *reinterpret_cast<float2*>(a.part_ml + (slot + h) * 2) = make_float2(m, l);
        }
      }
      ptx::named_bar_sync(2, 128);
      if (ok) {
        ptx::tc_fence_after();
        for (int cc = 0; cc < 4; ++cc) {
          const int lat = cc * 128 + warp * 32 + lane;
          for (int h0 = 0; h0 < nr32; h0 += 32) {
            uint32_t r[32];
            ptx::tmem_ld_32x32b_x32(tmem_base + lane_addr + kOCol0 + cc * kRows + h0, r);
            ptx::tmem_ld_wait_regs(r);
            if (direct) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (h0 + i < t.nrows)
                  a.out[(t.row0 + h0 + i) * static_cast<long long>(kRank) + lat] =
                      __float2bfloat16_rn(__uint_as_float(r[i]) * corr[h0 + i]);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (h0 + i < t.nrows) a.part_o[(slot + h0 + i) * kRank + lat] = __uint_as_float(r[i]);
            }
          }
        }
        ptx::tc_fence_before();
      }
      ptx::named_bar_sync(2, 128);  // corr and O^T are read before the next piece writes them
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, 512);
  }
}

// ------------------------------------------------------------------ join
// A CTA takes rows_per rows of a group of 64 (a packed prefix tile, or a tile); a thread four
// latent values.
__global__ void __launch_bounds__(128) prefix_mla_join_kernel(const Args a, int rows_per) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int per = kRows / rows_per;
  const int g = blockIdx.x / per, r0 = (blockIdx.x - g * per) * rows_per;
  const int n_tiles = __ldcg(a.head);
  const int n_groups = a.packed ? __ldcg(a.head + 1) : n_tiles;
  if (g >= n_groups) return;
  const long long U = __ldcg(a.u0 + n_tiles);
  const int G = parts(a, U);
  const Tile t = a.tiles[g];
  const long long g0 = __ldcg(a.u0 + g), g1 = __ldcg(a.u0 + g + 1);
  const int gc0 = g1 > g0 ? part_of(U, G, g0) : 0, gc1 = g1 > g0 ? part_of(U, G, g1 - 1) : -1;
  if (!a.packed && g1 > g0 && gc0 == gc1) return;  // done in one piece: already written
  for (int r = r0; r < min(r0 + rows_per, t.nrows); ++r) {
    const int row = t.row0 + r;
    // up to two tiles hold this row's pieces
    int ti[2] = {g, -1}, rr[2] = {r, 0}, c0[2] = {gc0, 0}, c1[2] = {gc1, -1};
    if (a.packed) {
      const int tq = row / a.H;
      const int b = request_of(a, tq);
      const int q0 = __ldg(a.cu + b);
      if (tq < __ldg(a.cu + b + 1)) {
        const int local = row - q0 * a.H;
        ti[1] = __ldcg(a.head + 2 + b) + local / kRows;
        rr[1] = local % kRows;
        if (ti[1] < n_tiles) {
          const long long b0 = __ldcg(a.u0 + ti[1]), b1 = __ldcg(a.u0 + ti[1] + 1);
          if (b1 > b0) {
            c0[1] = part_of(U, G, b0);
            c1[1] = part_of(U, G, b1 - 1);
          }
        }
      }
    }
    float M = -INFINITY;
#pragma unroll
    for (int q = 0; q < 2; ++q)
      for (int c = c0[q]; c <= c1[q]; ++c) {
        const long long s = piece_slot(a.G, c, ti[q], c == c0[q], c0[q] == c1[q]);
        M = fmaxf(M, __ldcg(a.part_ml + (s * kRows + rr[q]) * 2));
      }
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (M != -INFINITY) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll 4
        for (int c = c0[q]; c <= c1[q]; ++c) {
          const long long s = piece_slot(a.G, c, ti[q], c == c0[q], c0[q] == c1[q]) * kRows + rr[q];
          const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml + s * 2));
          const float4 o = __ldcg(reinterpret_cast<const float4*>(a.part_o + s * kRank) + threadIdx.x);
          const float w = exp2f(ml.x - M);  // 0 for a piece in which the row saw nothing
          L = fmaf(w, ml.y, L);
          acc.x = fmaf(w, o.x, acc.x);
          acc.y = fmaf(w, o.y, acc.y);
          acc.z = fmaf(w, o.z, acc.z);
          acc.w = fmaf(w, o.w, acc.w);
        }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    reinterpret_cast<uint2*>(a.out + static_cast<long long>(row) * kRank)[threadIdx.x] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    if (a.lse && threadIdx.x == 0) a.lse[row] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
  }
}

bool key_map(CUtensorMap* m, const void* base, long long rows, int cols, int box_rows) {
  static PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
  if (!enc) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
  int dev = 0;
  static int cached[64] = {};
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (cached[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
    cached[dev] = n;
  }
  return cached[dev];
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


struct Layout {
  int packed, max_tiles, G;
  size_t off_tiles, off_u0, off_head, off_ml, off_o, total;
};

Layout layout(const dsa_prefix_mla_args* a) {
  Layout p{};
  const long long rows = static_cast<long long>(a->total_q) * a->H;
  // Requests of few rows share prefix tiles: with H a multiple of 64, or 256 rows a request on
  // average, a request's own tiles are (nearly) full and the join would be extra traffic.
  p.packed = a->prefix_len > 0 && a->B > 1 && a->H % kRows != 0 && rows < 256LL * a->B ? 1 : 0;
  p.max_tiles = static_cast<int>((p.packed ? 2 : 1) * (rows / kRows + 1) + a->B + 1);
  p.G = sm_count();
  const size_t slots = 2 * static_cast<size_t>(p.G) + (p.packed ? p.max_tiles : 0);
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  p.off_tiles = 0;
  p.off_u0 = up(p.off_tiles + sizeof(Tile) * p.max_tiles);
  p.off_head = up(p.off_u0 + 8 * (static_cast<size_t>(p.max_tiles) + 1));
  p.off_ml = up(p.off_head + 4 * (static_cast<size_t>(a->B) + 4));
  p.off_o = up(p.off_ml + slots * kRows * 8);
  p.total = up(p.off_o + slots * kRows * kRank * 4);
  return p;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_prefix_mla_workspace_size(const dsa_prefix_mla_args* a, size_t* bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARGUMENT;
  const dsa_status st = validate(a);
  if (st != DSA_OK) return st;
  *bytes = a->total_q == 0 ? 0 : layout(a).total;
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
  if (static_cast<long long>(a->total_q) * a->H > 0x7FFFFFFFLL - kRows ||
      static_cast<long long>(a->num_pages) * a->page_size > 0x7FFFFFFFLL - kKeys)
    return DSA_ERR_UNSUPPORTED;
  const Layout p = layout(a);
  if (!a->workspace || a->workspace_bytes < p.total || !al(a->workspace, 16)) return DSA_ERR_WORKSPACE;
  unsigned* status = device_status_ptr();
  if (!status) return DSA_ERR_CUDA;
  CUtensorMap tc, tr;
  const long long slots = std::max(1LL, static_cast<long long>(a->num_pages) * a->page_size);
  const int box = std::min(a->page_size, kKeys);
  if (!key_map(&tc, a->cache_c, slots, kRank, box) || !key_map(&tr, a->cache_r, slots, kRope, box)) return DSA_ERR_CUDA;
  Args k{};
  k.B = a->B;
  k.total_q = a->total_q;
  k.H = a->H;
  k.page_size = a->page_size;
  k.num_pages = a->num_pages;
  k.max_pages = a->max_pages_per_seq;
  k.prefix_len = a->prefix_len;
  k.num_prefix_pages = a->num_prefix_pages;
  k.packed = p.packed;
  k.max_tiles = p.max_tiles;
  k.G = p.G;
  k.past_row = static_cast<int>(slots);
  k.scale_log2 = a->scale * 1.4426950408889634f;
  k.qn = static_cast<const __nv_bfloat16*>(a->q_nope);
  k.qr = static_cast<const __nv_bfloat16*>(a->q_rope);
  k.qn_t = a->qn_stride_t;
  k.qn_h = a->qn_stride_h;
  k.qr_t = a->qr_stride_t;
  k.qr_h = a->qr_stride_h;
  k.prefix_pages = a->prefix_pages;
  k.block_tables = a->block_tables;
  k.cu = a->cu_q_lens;
  k.lens = a->seq_lens;
  k.out = static_cast<__nv_bfloat16*>(a->out);
  k.lse = a->lse;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  k.tiles = reinterpret_cast<Tile*>(ws + p.off_tiles);
  k.u0 = reinterpret_cast<long long*>(ws + p.off_u0);
  k.head = reinterpret_cast<int*>(ws + p.off_head);
  k.part_ml = reinterpret_cast<float*>(ws + p.off_ml);
  k.part_o = reinterpret_cast<float*>(ws + p.off_o);
  k.status = status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaFuncSetAttribute(prefix_mla_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmem));
  if (e != cudaSuccess) return DSA_ERR_CUDA;
  e = launch_pdl(prefix_mla_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, k);
  if (e != cudaSuccess) return DSA_ERR_CUDA;
  e = launch_pdl(prefix_mla_kernel, dim3(p.G), dim3(kThreads), kSmem, s, tc, tr, k);
  if (e != cudaSuccess) return DSA_ERR_CUDA;
  // few rows: one CTA each, for latency; many: eight a CTA, most of which find nothing to join
  const long long rows = static_cast<long long>(a->total_q) * a->H;
  const int rows_per = rows <= 16384 ? 1 : 8;
  const long long groups = p.packed ? (rows + kRows - 1) / kRows : p.max_tiles;
  e = launch_pdl(prefix_mla_join_kernel, dim3(static_cast<unsigned>(groups * (kRows / rows_per))), dim3(128), 0, s, k,
                 rows_per);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
