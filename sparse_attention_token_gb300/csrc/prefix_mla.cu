// prefix_mla.cu -- latent attention for a batch whose sequences share their first tokens.
//
//     logit[t, h, s] = scale * (q_nope[t, h] . c_kv[s] + q_rope[t, h] . k_rope[s]),  s <= p(t)
//     out[t, h]      = sum_s softmax_s(logit[t, h, :]) c_kv[s],   lse[t, h] = ln sum_s exp(logit[t, h, s])
//
// Three launches.
//
// plan (one CTA): the (query, head) rows are cut into tiles of up to 128 rows, and every tile's
// keys into blocks of 128.  Requests of many rows fill tiles of their own, which walk the prefix
// and then the request's keys.  Where such tiles would stand too empty (few heads, one query; also
// a few long prompts among many of these) the batch shares: tiles packed across requests walk the
// prefix, further tiles, one request each, walk its own keys, and the two are joined.  The blocks of all tiles stand in one line, cut into equal parts, one per pair of SMs:
// a part may start and end inside a tile, so one long prefix fills every SM.
//
// attend (a cluster of two CTAs on two SMs per part, each holding 64 rows of a tile): the 512
// latent sums of 64 rows fill half a TMEM, and the pair's 2-SM MMAs (M = 128) run at the full
// rate of both, which one SM's MMAs on 64 rows cannot.  For each block of a piece of a tile:
//   S [128 rows x 128 keys] = Q . K^T       each CTA stages its rows of Q and 64 of the keys
//   O [128 rows x 512]     += P . V         each CTA stages its rows of P and, of all 128 keys,
//                                           its half of the latent columns (MN-major)
//   warps 0..7  softmax.  A thread holds one row and a quarter: 32 of the block's keys, 128 of the
//               row's latent sums (the quarters meet in shared memory).  The reference maximum
//               moves only when a block's maximum passes it by 8 (a factor 256);
//   warp 8      keys of S, three groups of 3 columns of 64 bf16, and warp 9 keys of P . V, two
//               groups of 2 columns: each group refilled as soon as its MMAs are done; TMA, one
//               lane per page piece and column;
//   warp 10     the query rows of every piece but the first (16-byte cp.async, any strides);
//   warp 11     TMEM; in the even CTA one lane issues the MMAs.
// 12 warps leave 168 registers a thread; with a warp for every group they were 128, which the
// softmax warps spilled.
// A tile done in one piece is normalised and written; the others leave (O, m, l) in fp32.
//
// What bounds it: the refill of the key buffers, with the tensor pipe close behind.  A block's
// products are 36 MMAs of N = 128 (35 cycles each) and 16 of N = 256 (64 each), 2284 cycles; it
// takes 2700 to 3050.  A buffer's MMAs, the commit to both CTAs, the next copy and its arrival at the
// issuer take some 3000 (870 from a V group's first MMA to the next copy, 2000 to 2250 from there).
// Keys are staged twice, once for S and once for P . V (the MMAs of a pair read the same offsets in
// both CTAs, so one copy cannot be split by keys and by columns), which fills shared memory with one
// block; nine K and four V groups cost the two copying warps and the issuer more than they save.
// 1781 x 64 rows behind 6000 keys take 0.98 to 1.03 ms, 1.53 to 1.60 PFLOP/s (0.87 to 0.95 ms, 1.65 to
// 1.80 PFLOP/s, launch after launch in a graph), the tensor pipe active 83 % of its cycles under the profiler.
//
// join: out = sum_j 2^(m_j - M) O_j / sum_j 2^(m_j - M) l_j over a row's pieces, in their order.
//
// Every wait is bounded; after one gives up, every role of both CTAs stops, the MMAs and copies in
// flight are drained (bounded) and TMEM is freed.
#include <cuda_bf16.h>

#include <algorithm>

#include "dsa_indexer.h"
#include "internal.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kRank = 512, kRope = 64, kAtoms = 9;        // 576 = 9 columns of 64 bf16
constexpr int kRows = 128;                                // rows per tile, 64 in each CTA of a pair
constexpr int kKeys = 128;                                // keys per block
constexpr int kThreads = 384;                             // 8 softmax warps, K, V, queries, MMA
constexpr uint32_t kAtomBytes = 64 * 128;                 // a column of 64 rows or keys
constexpr uint32_t kKGroup = 3 * kAtomBytes, kVGroup = 2 * 128 * 128;
constexpr uint32_t kOffQ = 0, kOffK = kAtoms * kAtomBytes, kOffV = kOffK + kAtoms * kAtomBytes;
constexpr uint32_t kOffP = kOffV + 2 * kVGroup, kOffMisc = kOffP + 2 * kAtomBytes;
constexpr size_t kSmem = kOffMisc + 3 * 1024;
constexpr uint32_t kOCol0 = 128;                          // O behind the two S buffers of 64 columns
constexpr int kMaxKeys = 0x7FFFFFFF - kKeys;              // that a query sees: the last block's border fits 32 bits
constexpr int kSetup = 3;                                 // what a tile costs beside its blocks, in blocks
constexpr float kLn2 = 0.6931471805599453f;

struct Tile {
  int row0, nrows;   // rows t * H + h
  int b;             // request, -1: rows of several requests (prefix only)
  int n_pre;         // blocks of the prefix; the rest are the request's own
  int limit;         // the most keys any of its rows sees
  int c0, c1;        // the parts that its blocks lie in (c1 < c0: none)
  int pad;
};
// A part, and the tile it begins in (tile < 0: no such part): all that its first piece needs.
struct Part {
  int tile, c0, c1, row0, nrows, b, n_pre, limit;
  long long begin, end, tile_begin, tile_end;
};
// A query of a packed batch: its request's first own tile, its first row among the request's
// rows, the keys it sees.
struct Query {
  int tile, row, sees, pad;
};

struct Args {
  int B, total_q, H, page_size, page_log2, num_pages, max_pages, prefix_len, num_prefix_pages;
  int may_pack;            // the plan may pack the prefix tiles across requests
  int max_tiles, G;        // tiles there is room for; CTA pairs
  int row_blocks;          // of 128 of the batch's rows
  int room;                // keys that the tables cover, at most kMaxKeys
  int narrow;              // the line is shorter than 2^31 places, whatever the lengths
  int past_row;            // a row coordinate past the cache: copies from there are zeros
  float scale_log2;        // scale * log2(e)
  const __nv_bfloat16 *qn, *qr;
  long long qn_t, qn_h, qr_t, qr_h;
  const int32_t *prefix_pages, *block_tables, *cu, *lens;
  __nv_bfloat16* out;
  float* lse;
  Tile* tiles;
  long long* u0;           // [max_tiles + 1] where each tile begins in the line of all blocks
  int* head;               // [0] tiles, [1] whether some have no blocks, [2] packed, [3 + b] own tiles before request b
  Part* parts;             // [G]
  Query* queries;          // [total_q], packed batches only
  float *part_o, *part_ml; // pieces: [slot][128 columns of 4][128 rows][4], [slot][128 rows][2]
  unsigned* status;
  // failure-path test hook: a role waits, at probe_at, for what never comes
  int probe_site;
  uint32_t probe_at;
  long long probe_cycles;
};

// Roles whose waits the test hook can let run out (the issuer's at a block, the queries' at a piece, the
// others' at their start); + kProbeOdd: in the pairs' odd CTAs.
enum : int { kProbeMma = 1, kProbeKeys = 2, kProbeValues = 3, kProbeQueries = 4, kProbeSoftmax = 5, kProbeOdd = 8 };
struct Probe {
  int site;
  uint32_t at;
  unsigned long long limit_ns;
};
Probe& armed_probe() {
  static thread_local Probe p{0, 0, 0};
  return p;
}

// Barriers of a CTA.  L: the even CTA's, waited for by the issuer; the others are waited for in
// each CTA and completed by the issuer's commits in both.
struct Bars {
  uint64_t qfull, qempty;        // qfull L: each CTA, its query rows
  uint64_t kfull[3], kempty[3];  // L: each CTA's copies
  uint64_t vfull[2], vempty[2];  // L
  uint64_t vown[2];              // this CTA's copies of a block with rows to clear
  uint64_t sfull[2], sempty[2];  // sempty L: 8 softmax warps of each CTA
  uint64_t pfull, ofree, done;   // pfull L; done: the issuer's last commit, in both
  uint64_t never;                // test hook: nothing arrives
  uint32_t kissued, vissued;     // this CTA's arrivals at kfull / vfull, all groups together; for the drain
};
static_assert(sizeof(Bars) <= 256, "the words behind the barriers begin at 256");

// Keys that query t of request b sees, cut to what the table covers (and counted as bad then).
__device__ __forceinline__ int sees(const Args& a, int b, int t, bool* bad) {
  const int q0 = __ldg(a.cu + b), q1 = __ldg(a.cu + b + 1);
  if (t < q0 || t >= q1) return 0;
  long long n = static_cast<long long>(__ldg(a.lens + b)) - (q1 - q0) + (t - q0) + 1;
  if (n > a.room) {
    *bad = true;
    n = a.room;
  }
  return static_cast<int>(max(n, 0LL));
}

// Whether a tile's rows are joined over two tiles, its own being one of a packed batch: tiles of
// several requests, and those that begin with own keys (may_pack: there is a prefix).
__device__ __forceinline__ bool joined(const Args& a, const Tile& t) {
  return a.may_pack && (t.b < 0 || t.n_pre == 0);
}

// The line of all tiles, U long: a tile's blocks stand behind kSetup places for what it costs to
// begin and end one (its queries, its first copies, its result: about 5 us).  Without them the
// parts with many short tiles end last: of 0, 1, 2, 3, 4, 6 places 64 requests x 64 heads behind
// 8192 keys took 109, 98, 90, 84, 84, 87 us, 128 x 16 heads behind 32768 180, 176, 173, 167, 168,
// 173 us.  The line is cut into G = min(CTA pairs, U) parts, part c
// being [c U / G, (c + 1) U / G); a part may hold no block.
__device__ __forceinline__ int parts(const Args& a, long long U) {
  return static_cast<int>(min(static_cast<long long>(a.G), U));
}
__device__ __forceinline__ long long part_begin(long long U, int G, int c) {
  if (U * G < (1LL << 32)) return static_cast<uint32_t>(U * c) / static_cast<uint32_t>(G);
  return U * c / G;
}
__device__ __forceinline__ int part_of(long long U, int G, long long u) {
  if (U * G < (1LL << 32)) return static_cast<uint32_t>((u + 1) * G - 1) / static_cast<uint32_t>(U);
  return static_cast<int>(((u + 1) * G - 1) / U);
}
// Where a piece in part c leaves row `row` of the batch, row r of its tile: the slot, of 128 rows,
// and the row there.  Pieces that begin inside a tile are the first of their part, those that only
// end inside one the last, so two slots a part hold them.  Whole tiles leave a result only where
// rows are joined over two tiles; theirs stand behind, by the rows of the batch, for the tiles of
// the prefix and then for the requests' own, so that they take as much as there are rows (a slot a
// tile took 1.2 GB for 4096 requests of 8 rows, now 0.2).
struct Place {
  int slot, row;
};
__device__ __forceinline__ Place place(const Args& a, int c, bool at_start, bool whole, bool own, int row, int r) {
  if (!whole) return {2 * c + (at_start ? 1 : 0), r};
  return {2 * a.G + (own ? a.row_blocks : 0) + (row >> 7), row & (kRows - 1)};
}

// ------------------------------------------------------------------ plan
constexpr int kPlanThreads = 1024;

// Exclusive scan over the CTA: within the warps, then every warp scans the warps' sums.
template <typename V>
__device__ __forceinline__ V block_scan(V v, V* wsum, V* total) {
  static_assert(kPlanThreads == 32 * 32, "one sum per lane");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](V s) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const V u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    return s;
  };
  const V s = scan(v);
  __syncthreads();
  if (lane == 31) wsum[warp] = s;
  __syncthreads();
  const V w = scan(wsum[lane]);
  *total = __shfl_sync(0xffffffffu, w, 31);
  const V before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return (warp > 0 ? before : V(0)) + s - v;
}

// One CTA; what a batch of up to 1024 requests, queries and tiles needs stays in shared memory and
// registers (a round trip through L2 between two steps costs about 0.4 us).
__global__ void __launch_bounds__(kPlanThreads) prefix_mla_plan_kernel(const Args a) {
  __shared__ long long wsum[32];
  __shared__ unsigned wsum_n[32];
  __shared__ int s_head[kPlanThreads + 1], s_sees[kPlanThreads];
  __shared__ long long s_b0[kPlanThreads];
  const int tid = threadIdx.x;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int q_end = min(max(__ldg(a.cu + a.B), 0), a.total_q);
  // every request's own tiles
  unsigned own_tiles = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    unsigned n = 0, total;
    if (b < a.B) {
      const int q0 = min(max(__ldg(a.cu + b), 0), a.total_q), q1 = min(max(__ldg(a.cu + b + 1), q0), a.total_q);
      n = ((q1 - q0) * a.H + kRows - 1) / kRows;
    }
    const int at = static_cast<int>(own_tiles + block_scan(n, wsum_n, &total));
    own_tiles += total;
    if (b < a.B) a.head[3 + b] = at;
    if (b < min(a.B, kPlanThreads)) s_head[b] = at;
  }
  // Requests share prefix tiles where their own tiles would stand too empty: by more than 15 % of the
  // rows there are (none are with H a multiple of 128).  Behind 8192 keys, shared and own tiles took:
  // 64 rows a request (half empty) 75 and 111 us, 128 (none) 67 and 60, 256 (none) 113 and 100, 320
  // (20 %) 143 and 153, 448 (14 %) 197 and 191, 576 (11 %) 245 and 230; 16 rows a request behind 32768
  // keys 150 and 732 us.
  const bool packed = a.may_pack && 100LL * kRows * own_tiles > 115LL * q_end * a.H;
  // rows beyond the last request (padding) count as one more request that sees nothing
  const int n_pad = packed ? 0 : ((a.total_q - q_end) * a.H + kRows - 1) / kRows;
  const int n_pre_tiles = packed ? a.row_blocks : 0;
  const int nreq = packed ? a.B : a.B + 1;
  const int n_tiles = static_cast<int>(min(n_pre_tiles + n_pad + own_tiles, static_cast<unsigned>(a.max_tiles)));
  if (tid == 0) {
    a.head[2] = packed;
    a.head[3 + a.B] = static_cast<int>(own_tiles);
    if (a.B < kPlanThreads) s_head[a.B] = static_cast<int>(own_tiles);
  }
  __syncthreads();
  auto head = [&](int b) { return n_pre_tiles + (b < kPlanThreads ? s_head[b] : a.head[3 + b]); };
  bool bad = false;
  if (packed) {
    for (int q = tid; q < a.total_q; q += kPlanThreads) {
      const int b = sequence_of(a.cu, a.B, q);
      Query r;
      r.sees = sees(a, b, q, &bad);
      const int q0 = __ldg(a.cu + b);
      const bool mine = q >= q0 && q < __ldg(a.cu + b + 1);
      r.tile = mine ? head(b) : n_tiles;  // n_tiles: no own keys (padding)
      r.row = mine ? (q - q0) * a.H : 0;
      r.pad = 0;
      *reinterpret_cast<int4*>(a.queries + q) = *reinterpret_cast<const int4*>(&r);
      if (q < kPlanThreads) s_sees[q] = r.sees;
    }
    __syncthreads();
  }
  const int kO = a.prefix_len / kKeys;  // first block with own keys
  long long u = 0, my_b0 = 0, my_units = 0;
  int empty = 0;
  Tile t{};
  for (int i0 = 0; i0 < n_tiles; i0 += kPlanThreads) {
    const int i = i0 + tid;
    long long units = 0;
    if (i < n_tiles) {
      t = Tile{};
      int own = 0;
      if (i < n_pre_tiles) {
        t.row0 = i * kRows;
        t.nrows = min(kRows, a.total_q * a.H - t.row0);
        t.b = -1;
        for (int q = t.row0 / a.H; q <= (t.row0 + t.nrows - 1) / a.H; ++q)
          t.limit = max(t.limit, q < kPlanThreads ? s_sees[q] : a.queries[q].sees);
      } else {
        int lo = 0, hi = nreq;  // the last b with head(b) <= i
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (head(mid) <= i) lo = mid; else hi = mid;
        }
        const int q0 = min(max(__ldg(a.cu + lo), 0), a.total_q);
        const int q1 = lo < a.B ? min(max(__ldg(a.cu + lo + 1), q0), a.total_q) : a.total_q;
        const int k = i - head(lo), rows = (q1 - q0) * a.H;  // (offsets that do not rise make any k)
        const bool in = k >= 0 && k < (rows + kRows - 1) / kRows;
        t.row0 = q0 * a.H + (in ? k * kRows : 0);
        t.nrows = in ? min(kRows, rows - k * kRows) : 0;
        t.b = min(lo, a.B - 1);
        const int last = (t.row0 + t.nrows - 1) / a.H;
        if (lo < a.B && in)
          t.limit = !packed ? sees(a, lo, last, &bad) : (last < kPlanThreads ? s_sees[last] : a.queries[last].sees);
        own = t.limit > a.prefix_len ? (t.limit + kKeys - 1) / kKeys - kO : 0;
      }
      t.n_pre = (packed && i >= n_pre_tiles) ? 0 : (min(t.limit, a.prefix_len) + kKeys - 1) / kKeys;
      units = t.n_pre + own > 0 ? t.n_pre + own + kSetup : 0;
      empty += units == 0;
    }
    long long total, at;
    if (a.narrow) {
      unsigned sum;
      at = block_scan(static_cast<unsigned>(units), wsum_n, &sum);
      total = sum;
    } else {
      at = block_scan(units, wsum, &total);
    }
    if (i < n_tiles) {
      if (n_tiles > kPlanThreads) a.tiles[i] = t;
      a.u0[i] = u + at;
    }
    my_b0 = u + at;
    my_units = units;
    u += total;
  }
  if (tid == 0) a.u0[n_tiles] = u;
  empty = __syncthreads_count(empty > 0);
  if (tid == 0) {
    a.head[0] = n_tiles;
    a.head[1] = empty;  // whether there are any
  }
  if (bad) atomicOr(a.status, kStatusUncovered);
  // the parts that each tile's blocks lie in
  const int G = parts(a, u);
  for (int i = tid; i < n_tiles; i += kPlanThreads) {
    if (n_tiles > kPlanThreads) {
      t = a.tiles[i];
      my_b0 = a.u0[i];
      my_units = a.u0[i + 1] - my_b0;
    } else {
      s_b0[i] = my_b0;
    }
    t.c0 = 0;
    t.c1 = -1;
    if (my_units > 0) {
      t.c0 = part_of(u, G, my_b0 + kSetup);
      t.c1 = part_of(u, G, my_b0 + my_units - 1);
    }
    int4* p = reinterpret_cast<int4*>(a.tiles + i);
    p[0] = make_int4(t.row0, t.nrows, t.b, t.n_pre);
    p[1] = make_int4(t.limit, t.c0, t.c1, 0);
  }
  __syncthreads();
  // the tile that each part begins in: the last with b0 <= begin (the ones before it that share
  // its place have no blocks)
  for (int c = tid; c < a.G; c += kPlanThreads) {
    if (c >= G) {
      a.parts[c].tile = -1;
      continue;
    }
    const long long begin = part_begin(u, G, c);
    auto b0 = [&](int i) { return n_tiles > kPlanThreads ? a.u0[i] : s_b0[i]; };
    int lo = 0, hi = n_tiles;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (b0(mid) <= begin) lo = mid; else hi = mid;
    }
    const int4* w = reinterpret_cast<const int4*>(a.tiles + lo);
    const int4 w0 = w[0], w1 = w[1];
    a.parts[c] = Part{lo, w1.y, w1.z, w0.x, w0.y, w0.z, w0.w, w1.x, begin, part_begin(u, G, c + 1), b0(lo),
                      lo + 1 < n_tiles ? b0(lo + 1) : u};
  }
}

// ------------------------------------------------------------------ attend
// The part's pieces: tile i, its blocks [k0, k1).  Every role walks the same list.
struct Piece {
  int i, k0, k1;
  bool whole;          // all the tile's blocks
  long long b0, b1;    // the tile's places in the line
  long long next;      // where the next piece begins
};
__device__ __forceinline__ bool next_piece(const Args& a, Piece& p, long long u_hi, Tile& t) {
  while (p.next < u_hi) {
    const long long first = p.b0 + kSetup, from = p.next, to = min(p.b1, u_hi);
    if (to > from) {
      p.k0 = static_cast<int>(max(from - first, 0LL));
      p.k1 = static_cast<int>(max(to - first, 0LL));
      p.whole = p.k0 == 0 && to == p.b1;
      p.next = to;
      if (p.k1 > p.k0) return true;
      if (to == u_hi) return false;  // the part ends before the tile's first block
    }
    ++p.i;  // done, or without blocks
    p.b0 = p.b1;
    p.b1 = __ldcg(a.u0 + p.i + 1);
    const int4 w = __ldcg(reinterpret_cast<const int4*>(a.tiles + p.i));
    t.limit = __ldcg(reinterpret_cast<const int*>(a.tiles + p.i) + 4);
    t.row0 = w.x;
    t.nrows = w.y;
    t.b = w.z;
    t.n_pre = w.w;
  }
  return false;
}

// Block k of a tile: its first position, and the positions [lo, hi) of it that the tile sees.
struct Block {
  int s0, lo, hi;
  bool pre;
};
__device__ __forceinline__ Block block_at(const Args& a, const Tile& t, int k) {
  Block b;
  b.pre = k < t.n_pre;
  b.s0 = (b.pre ? k : k - t.n_pre + a.prefix_len / kKeys) * kKeys;
  b.lo = b.pre ? 0 : a.prefix_len;
  b.hi = b.pre ? min(t.limit, a.prefix_len) : t.limit;
  return b;
}
// Cache row of position s (a multiple of the box) of a block, for a copy of `box` rows from
// there: past_row (zeros) when the tile sees none of them, or the page is not there (*bad).
__device__ __forceinline__ int cache_row(const Args& a, const Tile& t, const Block& b, int s, int box, bool* bad) {
  if (s >= b.hi || s + box <= b.lo) return a.past_row;
  const int j = s >> a.page_log2;
  int pg = -1;
  if (b.pre) {
    if (j < a.num_prefix_pages) pg = __ldg(a.prefix_pages + j);
  } else if (j < a.max_pages) {
    pg = __ldg(a.block_tables + static_cast<long long>(t.b) * a.max_pages + j);
  }
  if (pg < 0 || pg >= a.num_pages) {
    *bad = true;
    return a.past_row;
  }
  return pg * a.page_size + (s & (a.page_size - 1));
}

// This CTA's rows r0, r0 + step, .. of the tile's queries (16-byte cp.async, zeros past its rows);
// eight lanes a row (ch: which), 128 bytes at a time, swizzled.
__device__ __forceinline__ void load_q(const Args& a, uint8_t* smem, const Tile& t, int rank, int r0, int step,
                                       int ch) {
  for (int r = r0; r < 64; r += step) {
    const bool live = rank * 64 + r < t.nrows;
    const int row = t.row0 + (live ? rank * 64 + r : 0);
    const int tq = row / a.H, h = row - tq * a.H;
    const __nv_bfloat16* qn = a.qn + tq * a.qn_t + h * a.qn_h + ch * 8;
    const __nv_bfloat16* qr = a.qr + tq * a.qr_t + h * a.qr_h + ch * 8;
    uint8_t* dst = smem + kOffQ + r * 128 + ((ch ^ (r & 7)) << 4);
#pragma unroll
    for (int at = 0; at < kAtoms; ++at)
      ptx::cp_async_16(dst + at * kAtomBytes, at < 8 ? qn + at * 64 : qr, live ? 16u : 0u);
  }
}

// kProbe: with the test hook's waits (asked for in every call, they took up to 0.6 us of it; asked for by
// the copying warps before every group, 8 us of the 74 that 64 x 64 heads behind 8192 keys take).
template <bool kProbe>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefix_mla_kernel(const __grid_constant__ CUtensorMap tmap_c, const __grid_constant__ CUtensorMap tmap_r,
                      const Args a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the same in both CTAs, so both return together
  if ((ptx::smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusSmemAlign);
    return;
  }
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffMisc);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + kOffMisc + 256);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 260);
  float* xmax = reinterpret_cast<float*>(smem + kOffMisc + 512);  // [2][4][64] by block parity, quarter, row
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  // A wait that gives up ends the roles of its CTA, and each of them then those of the other CTA.
  auto give_up = [&]() {
    *abort = 1;
    ptx::st_shared_cluster(ptx::mapa_shared(ptx::smem_u32(const_cast<int*>(abort)), ptx::cluster_ctarank() ^ 1u), 1u);
  };
  auto spin = [&](uint64_t* bar, uint32_t parity, long long cycles = ptx::kWaitCycles) {
    return ptx::mbar_spin(bar, parity, abort, a.status, kStatusTimeout, cycles);
  };
  auto probed = [&](int site) { return kProbe && a.probe_site == site + (rank != 0 ? kProbeOdd : 0); };
  auto stop_at = [&](int site) { return probed(site) ? a.probe_at : ~0u; };
  auto run_out = [&]() { return __all_sync(0xffffffffu, spin(&bars->never, 0, a.probe_cycles)) != 0; };

  if (threadIdx.x == 0) {
    ptx::mbar_init(&bars->qfull, 2);
    ptx::mbar_init(&bars->qempty, 1);
    for (int g = 0; g < 3; ++g) {
      ptx::mbar_init(&bars->kfull[g], 2);
      ptx::mbar_init(&bars->kempty[g], 1);
    }
    for (int g = 0; g < 2; ++g) {
      ptx::mbar_init(&bars->vfull[g], 2);
      ptx::mbar_init(&bars->vempty[g], 1);
      ptx::mbar_init(&bars->vown[g], 1);
      ptx::mbar_init(&bars->sfull[g], 1);
      ptx::mbar_init(&bars->sempty[g], 16);
    }
    ptx::mbar_init(&bars->pfull, 16);
    ptx::mbar_init(&bars->ofree, 1);
    ptx::mbar_init(&bars->done, 1);
    ptx::mbar_init(&bars->never, 1);
    bars->kissued = bars->vissued = 0;
    *abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 11) {
    ptx::tmem_alloc_pair(tmem_holder, 512);
    ptx::tmem_relinquish_pair();
  }
  if (warp == 8 && lane == 0) {
    ptx::prefetch_tmap(&tmap_c);
    ptx::prefetch_tmap(&tmap_r);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // both CTAs' barriers initialised and TMEM allocated
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int c = blockIdx.x >> 1;
  const int4* rec = reinterpret_cast<const int4*>(a.parts + c);
  const int4 r0 = __ldcg(rec), r1 = __ldcg(rec + 1);
  const longlong2 r2 = __ldcg(reinterpret_cast<const longlong2*>(rec + 2));
  const longlong2 r3 = __ldcg(reinterpret_cast<const longlong2*>(rec + 3));
  const long long u_hi = r0.x >= 0 ? r2.y : 0;
  const int box = min(a.page_size, 64);  // rows of one copy
  const int box_log2 = 31 - __clz(box);
  Piece p{r0.x, 0, 0, false, r3.x, r3.y, r0.x >= 0 ? r2.x : 0};
  Tile t{r0.w, r1.x, r1.y, r1.z, r1.w, 0, 0, 0};

  if (warp == 11) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    // S of block k + 1 goes before P . V of block k, whose weights are computed meanwhile.
    if (rank == 0 && ptx::elect_one()) {
      const uint32_t sbase = ptx::smem_u32(smem);
      const uint32_t id1 = ptx::idesc_f32acc(128, kKeys, true);
      const uint32_t id2 = ptx::idesc_f32acc_bf16_bmn(128, 256);
      const uint32_t q0 = ptx::desc_lo(sbase + kOffQ, 16), k0 = ptx::desc_lo(sbase + kOffK, 16);
      const uint32_t p0 = ptx::desc_lo(sbase + kOffP, 16), v0 = ptx::desc_lo(sbase + kOffV, 128 * 128);
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && spin(bar, parity); };
      const uint32_t stop = stop_at(kProbeMma);
      uint32_t n1 = 0, n2 = 0;  // blocks whose S / P . V was issued
      bool more = next_piece(a, p, u_hi, t);
      for (uint32_t seg = 0; ok && more; ++seg) {
        wait(&bars->qfull, seg & 1);
        const int nblk = p.k1 - p.k0;
        for (int i = 0; ok && i <= nblk; ++i) {
          if (i < nblk) {
            const uint32_t d = tmem_base + (n1 & 1) * 64;
            if (kProbe && n1 == stop) ok = ok && spin(&bars->never, 0, a.probe_cycles);
            wait(&bars->sempty[n1 & 1], ((n1 >> 1) & 1) ^ 1);
#pragma unroll
            for (int g = 0; g < 3; ++g) {
              wait(&bars->kfull[g], n1 & 1);
              ptx::tc_fence_after();
              if (ok) {
                uint32_t qa = q0, kb = k0;
                asm volatile("" : "+r"(qa), "+r"(kb));  // descriptors are added up here, not kept over the loop
#pragma unroll
                for (int s = 0; s < 12; ++s) {  // 16 values of K per MMA, four in a column
                  const uint32_t off = ((3 * g + (s >> 2)) * kAtomBytes + (s & 3) * 32) >> 4;
                  ptx::mma_bf16_pair(d, qa + off, kb + off, id1, (g > 0 || s > 0) ? 1u : 0u);
                }
                ptx::mma_commit_pair(&bars->kempty[g], 3);
                if (g == 2) {
                  ptx::mma_commit_pair(&bars->sfull[n1 & 1], 3);
                  if (i + 1 == nblk) ptx::mma_commit_pair(&bars->qempty, 3);
                }
              }
            }
            ++n1;
          }
          if (i == nblk) more = next_piece(a, p, u_hi, t);  // its loads pass behind the last block's softmax
          if (i > 0) {
            wait(&bars->pfull, n2 & 1);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              wait(&bars->vfull[g], n2 & 1);
              ptx::tc_fence_after();
              if (ok) {
                uint32_t pa = p0, vb = v0;
                asm volatile("" : "+r"(pa), "+r"(vb));
#pragma unroll
                for (int s = 0; s < 8; ++s)  // 16 keys per MMA: two 8-key groups of 1024 bytes
                  ptx::mma_bf16_pair(tmem_base + kOCol0 + g * 128,
                                     pa + (((s >> 2) * kAtomBytes + (s & 3) * 32) >> 4),
                                     vb + ((g * kVGroup + s * 2048) >> 4), id2, (i > 1 || s > 0) ? 1u : 0u);
                ptx::mma_commit_pair(&bars->vempty[g], 3);
                if (g == 1) ptx::mma_commit_pair(&bars->ofree, 3);
              }
            }
            ++n2;
          }
        }
      }
      if (!ok) give_up();
      ptx::mma_commit_pair(&bars->done, 3);
      ptx::mbar_spin_drain(&bars->done, 0, a.status, kStatusTimeout, ptx::kWaitCycles / 10);
    }
    __syncwarp();
  } else if (warp == 8) {
    // ------------------------------------------------------------ keys of S: this CTA's 64 of a block
    const int per = 64 / box, j = lane & (per - 1), at = lane / per;  // box of a column, column of a group
    uint32_t n = 0, left = 0;  // left: arrivals when a wait gave up
    bool ok = !probed(kProbeKeys) || run_out();
    while (ok && next_piece(a, p, u_hi, t)) {
      for (int k = p.k0; ok && k < p.k1; ++k, ++n) {
        const Block b = block_at(a, t, k);
        bool bad = false;
        const int row = cache_row(a, t, b, b.s0 + rank * 64 + j * box, box, &bad);
        if (bad) atomicOr(a.status, kStatusBadPage);
#pragma unroll
        for (int g = 0; g < 3; ++g) {
          ok = ok && __all_sync(0xffffffffu, spin(&bars->kempty[g], (n & 1) ^ 1)) != 0;
          if (!ok) {
            left = 3 * n + g;
            break;
          }
          const uint32_t full = ptx::mapa_shared(ptx::smem_u32(&bars->kfull[g]), 0);
          if (lane == 0) ptx::mbar_arrive_expect_tx_cluster(full, kKGroup);
          __syncwarp();
          if (at < 3) {
            uint8_t* dst = smem + kOffK + (3 * g + at) * kAtomBytes + j * box * 128;
            if (3 * g + at < 8) ptx::tma_load_2d_pair(dst, &tmap_c, full, (3 * g + at) * 64, row);
            else ptx::tma_load_2d_pair(dst, &tmap_r, full, 0, row);
          }
        }
      }
    }
    if (!ok) give_up();
    if (lane == 0) bars->kissued = ok ? 3 * n : left;
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ keys of P . V: this CTA's 4 columns, all 128
    const int per = 128 / box, j = lane & (per - 1), at = lane / per;
    uint32_t n = 0, cleared = 0, left = 0;
    bool ok = !probed(kProbeValues) || run_out();
    while (ok && next_piece(a, p, u_hi, t)) {
      for (int k = p.k0; ok && k < p.k1; ++k, ++n) {
        const Block b = block_at(a, t, k);
        bool bad = false;
        const int row = cache_row(a, t, b, b.s0 + j * box, box, &bad);
        // rows that no row of this tile sees may hold anything: their weights are 0, and the
        // values are cleared so that the products are
        const bool clear = b.s0 < b.lo || b.s0 + kKeys > b.hi;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          ok = ok && __all_sync(0xffffffffu, spin(&bars->vempty[g], (n & 1) ^ 1)) != 0;
          if (!ok) {
            left = 2 * n + (clear ? 0 : g);
            if (clear && g > 0)  // the first group's copy lands on this CTA's own barrier
              ptx::mbar_spin_drain(&bars->vown[0], cleared & 1, a.status, kStatusTimeout, ptx::kWaitCycles / 10);
            break;
          }
          const uint32_t full = ptx::mapa_shared(ptx::smem_u32(&bars->vfull[g]), 0);
          if (lane == 0) {
            if (clear) ptx::mbar_arrive_expect_tx(&bars->vown[g], kVGroup);
            else ptx::mbar_arrive_expect_tx_cluster(full, kVGroup);
          }
          __syncwarp();
          if (at < 2) {
            uint8_t* dst = smem + kOffV + g * kVGroup + at * (128 * 128) + j * box * 128;
            const int x = rank * 256 + (2 * g + at) * 64;
            if (clear) ptx::tma_load_2d(dst, &tmap_c, &bars->vown[g], x, row);
            else ptx::tma_load_2d_pair(dst, &tmap_c, full, x, row);
          }
        }
        if (!clear || !ok) continue;
        const int from = min(max(b.lo - b.s0, 0), kKeys), to = max(min(b.hi - b.s0, kKeys), from);  // [from, to) stay
        const int n_clear = from + kKeys - to;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const bool landed = ptx::mbar_spin_drain(&bars->vown[g], cleared & 1, a.status, kStatusTimeout,
                                                   ok ? ptx::kWaitCycles : ptx::kWaitCycles / 10);
          if (!__all_sync(0xffffffffu, landed) && ok) {
            ok = false;
            left = 2 * n + g;
          }
          if (!ok) continue;  // the other group's copy is waited for all the same
          uint8_t* base = smem + kOffV + g * kVGroup;
          for (int e = lane; e < n_clear * 16; e += 32) {  // 16 chunks of 16 bytes a row, in two columns
            const int r = e >> 4, key = r < from ? r : to + (r - from);
            *reinterpret_cast<uint4*>(base + ((e >> 3) & 1) * (128 * 128) + key * 128 + (e & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_u32(&bars->vfull[g]), 0));
        }
        ++cleared;
      }
    }
    if (!ok) give_up();
    if (lane == 0) bars->vissued = ok ? 2 * n : left;
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------ queries: this CTA's 64 rows of the tile
    // (the softmax warps, idle until then, bring the first piece's: 4 x 16 heads behind 1000 took
    // 18.3 us when this warp did, 17.0 now, longer calls the same within 0.6)
    const uint32_t full = ptx::mapa_shared(ptx::smem_u32(&bars->qfull), 0);
    const uint32_t stop = stop_at(kProbeQueries);
    next_piece(a, p, u_hi, t);
    for (uint32_t seg = 1; next_piece(a, p, u_hi, t); ++seg) {
      bool good = !kProbe || seg != stop || spin(&bars->never, 0, a.probe_cycles);
      good = good && spin(&bars->qempty, (seg & 1) ^ 1);
      if (!__all_sync(0xffffffffu, good)) {
        give_up();
        break;
      }
      load_q(a, smem, t, rank, lane >> 3, 4, lane & 7);
      ptx::cp_async_wait_all();
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster(full);
    }
  } else {
    // ------------------------------------------------------------ softmax, rescale, output (warps 0..7)
    const int row = (warp & 1) * 32 + lane, half = (warp >> 1) & 1;  // TMEM lane = 64 half + row
    const int part = warp >> 2, quarter = 2 * half + part;           // columns 32 part of S, 128 part of O
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t row_bar = 2 + (warp & 1);                         // the four warps of the same rows
    const int per = max(32 / box, 1);                                // boxes under this thread's keys
    const uint32_t full = ptx::mapa_shared(ptx::smem_u32(&bars->pfull), 0);
    const uint32_t empty0 = ptx::mapa_shared(ptx::smem_u32(&bars->sempty[0]), 0);
    bool ok = true;
    uint32_t n = 0;
    const int trow = rank * 64 + row;
    auto limit_of = [&](const Tile& tile) {  // keys this row sees
      if (trow >= tile.nrows) return 0;
      const int tq = (tile.row0 + trow) / a.H;
      bool bad = false;  // counted by the plan
      return min(joined(a, tile) ? __ldcg(&a.queries[tq].sees) : sees(a, tile.b, tq, &bad), tile.limit);
    };
    auto row_at = [&](const Tile& tile, int k) {  // cache row of the lane's box under this warp's keys
      const Block b = block_at(a, tile, k);
      const int s0 = b.s0 + half * 64 + part * 32;
      bool bad = false;  // counted by the copies
      return cache_row(a, tile, b, (s0 & ~(box - 1)) + (lane & (per - 1)) * box, box, &bad);
    };
    bool more = next_piece(a, p, u_hi, t);
    if (more) {  // the first piece's queries: eight warps at once
      load_q(a, smem, t, rank, threadIdx.x >> 3, 32, lane & 7);
      ptx::cp_async_wait_all();
      ptx::fence_proxy_async_smem();
      ptx::named_bar_sync(4, 256);
      if (threadIdx.x == 0) ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_u32(&bars->qfull), 0));
    }
    if (probed(kProbeSoftmax) && warp == 0) ok = run_out();
    int lim = more ? limit_of(t) : 0, crow = more ? row_at(t, p.k0) : 0;
    while (more) {
      float m = -INFINITY, l = 0.f;  // reference maximum (scaled, base 2), this quarter's sum
      for (int k = p.k0; k < p.k1; ++k, ++n) {
        const int tb = n & 1;
        const Block b = block_at(a, t, k);
        const int s0 = b.s0 + half * 64 + part * 32;  // this thread's 32 keys
        if (k > p.k0) crow = row_at(t, k);            // passes while S is computed
        const unsigned there = __ballot_sync(0xffffffffu, crow != a.past_row);
        if (ok) ok = __all_sync(0xffffffffu, spin(&bars->sfull[tb], (n >> 1) & 1)) != 0;
        float x[32];
        float mb = -INFINITY;
        if (ok) {
          ptx::tc_fence_after();
          uint32_t xr[32];
          ptx::tmem_ld_32x32b_x32(tmem_base + lane_addr + tb * 64 + part * 32, xr);
          ptx::tmem_ld_wait_regs(xr);
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_cluster(empty0 + tb * 8);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(xr[i]);
          const int end = min(b.hi, lim);
          const unsigned all = (1u << per) - 1u;
          if (s0 < b.lo || s0 + 32 > end || (there & all) != all) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int s = s0 + i;
              const bool v = s >= b.lo && s < end && ((there >> ((i >> box_log2) & (per - 1))) & 1u);
              x[i] = v ? x[i] : -INFINITY;
            }
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) mb = fmaxf(mb, x[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = -INFINITY;
        }
        // the row's block maximum over its quarters
        float* xm = xmax + tb * 256 + row;
        xm[quarter * 64] = mb;
        ptx::named_bar_sync(row_bar, 128);
        mb = fmaxf(fmaxf(xm[0], xm[64]), fmaxf(xm[128], xm[192])) * a.scale_log2;
        // The reference maximum moves only when the block's maximum exceeds it by more than 8
        // (a factor 256 in probability): p stays below 256 and the output, which divides by
        // the sum taken against the same reference, is unchanged.
        float mn = m;
        if (m == -INFINITY || mb > m + 8.f) mn = mb;
        const float cr = (m == -INFINITY || mn == m) ? 1.f : ptx::ex2(m - mn);
        const float off = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: every x is -inf, p = 0
        // P goes into the product as bf16: an MMA's operands are of one type, and V is the cache.  That
        // moves each p by at most 2^-9 of it, the output by about 0.0011 of its size; its own rounding
        // to bf16 makes 0.0017, both together 0.0018 to 0.0020 (the mean error of the listed batches
        // against 64 bits).  P as a sum of two bf16 would take P . V's 1024 of a block's 2284 cycles twice.
        // The sum l takes p unrounded, so that lse has fp32 accuracy.
        float ls[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float p0 = ptx::ex2(fmaf(x[2 * i], a.scale_log2, -off));
          const float p1 = ptx::ex2(fmaf(x[2 * i + 1], a.scale_log2, -off));
          ls[(2 * i) & 3] += p0;
          ls[(2 * i + 1) & 3] += p1;
          const __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
          pk[i] = *reinterpret_cast<const uint32_t*>(&pb);
        }
        l = l * cr + ((ls[0] + ls[1]) + (ls[2] + ls[3]));
        m = mn;
        // P and O are free once the previous block's P . V has completed
        if (n > 0 && ok) ok = __all_sync(0xffffffffu, spin(&bars->ofree, (n - 1) & 1)) != 0;
        if (ok) {
          // row of P: this quarter's 32 keys = 4 chunks of 16 bytes, swizzled by the row
          uint8_t* prow = smem + kOffP + half * kAtomBytes + row * 128;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(prow + (((part * 4 + q) ^ (row & 7)) << 4)) =
                make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
          ptx::fence_proxy_async_smem();
          if (k > p.k0 && __any_sync(0xffffffffu, cr != 1.f)) {
            ptx::tc_fence_after();
            for (int q = 0; q < 4; ++q) {
              const uint32_t col = tmem_base + lane_addr + kOCol0 + part * 128 + q * 32;
              uint32_t r[32];
              ptx::tmem_ld_32x32b_x32(col, r);
              ptx::tmem_ld_wait_regs(r);
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * cr);
              ptx::tmem_st_32x32b_x32(col, r);
            }
            ptx::tmem_st_wait();
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(full);
      }
      // the next piece, its loads behind the last P . V
      const Piece pc = p;
      const Tile tc = t;
      more = next_piece(a, p, u_hi, t);
      lim = more ? limit_of(t) : 0;
      crow = more ? row_at(t, p.k0) : 0;
      // the piece's result
      const bool at_start = pc.k0 == 0;
      const bool direct = pc.whole && !joined(a, tc);
      if (ok) ok = __all_sync(0xffffffffu, spin(&bars->ofree, (n - 1) & 1)) != 0;
      float* xs = xmax + (n & 1) * 256 + row;  // the side that the last block did not use
      xs[quarter * 64] = l;
      ptx::named_bar_sync(row_bar, 128);
      l = (xs[0] + xs[64]) + (xs[128] + xs[192]);
      ptx::named_bar_sync(row_bar, 128);  // read before the next piece writes there
      const bool live = trow < tc.nrows && ok;
      const Place at = place(a, c, at_start, pc.whole, tc.b >= 0, tc.row0 + trow, trow);
      if (live && quarter == 0) {
        if (!direct)
          *reinterpret_cast<float2*>(a.part_ml + (static_cast<long long>(at.slot) * kRows + at.row) * 2) = make_float2(m, l);
        else if (a.lse) a.lse[tc.row0 + trow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;  // no key: 0; a NaN stays one
      ptx::tc_fence_after();
      for (int q = 0; q < 4; ++q) {
        uint32_t r[32];
        ptx::tmem_ld_32x32b_x32(tmem_base + lane_addr + kOCol0 + part * 128 + q * 32, r);
        ptx::tmem_ld_wait_regs(r);
        const int lat = half * 256 + part * 128 + q * 32;
        if (direct) {
          // through the rows' own places in P, so that four lanes write 64 bytes of a row together
          // (a lane's 16 bytes a store, 1024 apart, took the piece's end from 1.5 to 5 us)
          uint8_t* place = smem + kOffP + half * kAtomBytes + row * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(r[8 * i + 2 * j]) * inv,
                                                             __uint_as_float(r[8 * i + 2 * j + 1]) * inv);
              w[j] = *reinterpret_cast<const uint32_t*>(&v);
            }
            *reinterpret_cast<uint4*>(place + (((part * 4 + i) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          ptx::named_bar_sync(row_bar, 128);
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // this warp's 8 rows x 2 halves of 128 bytes, 4 a step
            const int sg = i * 4 + (lane >> 3), hf = sg & 1, ch = lane & 7;
            const int rw = (warp & 1) * 32 + (warp >> 1) * 8 + (sg >> 1);
            const uint4 v = *reinterpret_cast<const uint4*>(smem + kOffP + hf * kAtomBytes + rw * 128 +
                                                            ((ch ^ (rw & 7)) << 4));
            if (ok && rank * 64 + rw < tc.nrows)
              *reinterpret_cast<uint4*>(a.out + (tc.row0 + rank * 64 + rw) * static_cast<long long>(kRank) + hf * 256 +
                                        (ch >> 2) * 128 + q * 32 + (ch & 3) * 8) = v;
          }
          ptx::named_bar_sync(row_bar, 128);  // read before it is written again
        } else if (live) {
          uint4* dst = reinterpret_cast<uint4*>(a.part_o) +
                       (static_cast<long long>(at.slot) * (kRank / 4) + lat / 4) * kRows + at.row;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i * kRows] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        }
      }
      ptx::tc_fence_before();
    }
    if (!ok) give_up();
  }
  ptx::tc_fence_before();
  __syncthreads();
  // the issuer has waited for its last commit in its own CTA; its arrival here comes from outside too
  if (rank != 0 && threadIdx.x == 0)
    ptx::mbar_spin_drain(&bars->done, 0, a.status, kStatusTimeout, ptx::kWaitCycles / 10);
  ptx::cluster_sync();  // no CTA leaves while its peer may still touch its memory, barriers or TMEM
  if (*abort) {
    // Set in both CTAs if in one.  The MMAs have waited for every copy unless a role gave up.  Then a
    // group's last full phase may have the arrival of one CTA only, no more than one phase apart
    // (a copy of a block waits for the MMAs on the block before, and those for both CTAs' copies):
    // arrive for the other, so that the phase ends as soon as the copies that were issued have landed.
    if (rank == 0 && threadIdx.x == 0) {
      const uint32_t k0 = bars->kissued, v0 = bars->vissued;
      const uint32_t k1 = ptx::ld_shared_cluster(ptx::mapa_shared(ptx::smem_u32(&bars->kissued), 1));
      const uint32_t v1 = ptx::ld_shared_cluster(ptx::mapa_shared(ptx::smem_u32(&bars->vissued), 1));
      auto drain = [&](uint64_t* bar, uint32_t n0, uint32_t n1) {  // phases with this and the other CTA's arrival
        if (n0 != n1) ptx::mbar_arrive(bar);
        const uint32_t n = max(n0, n1);
        if (n > 0) ptx::mbar_spin_drain(bar, (n - 1) & 1, a.status, kStatusTimeout, ptx::kWaitCycles / 10);
      };
      for (uint32_t g = 0; g < 3; ++g) drain(&bars->kfull[g], (k0 + 2 - g) / 3, (k1 + 2 - g) / 3);
      for (uint32_t g = 0; g < 2; ++g) drain(&bars->vfull[g], (v0 + 1 - g) / 2, (v1 + 1 - g) / 2);
    }
    ptx::cluster_sync();
  }
  if (warp == 11) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, 512);
  }
}

// ------------------------------------------------------------------ join
// A CTA of 512 threads (128 rows x 4) joins some of the 128 latent columns (of 4) of a tile's rows.
// Packed batches: a row has the pieces of its prefix tile and of one of its request's own tiles;
// blockIdx = per_tile * prefix tile + columns (the grid has room for either kind).  Otherwise blockIdx = 2 * part + columns for every
// part that begins inside a tile; the parts of a tile share its columns (up to 64 of them), so that
// a tile of many pieces has many CTAs.  The four threads of a row split the columns when the pieces
// are few, else the pieces, and meet in shared memory.  About one wave of CTAs, a few trips to L2.
// Tiles without any block get zeros.
constexpr int kBatch = 4, kAcc = 8;  // pieces whose loads go out together, columns (of 4) at once
__global__ void __launch_bounds__(512, 1) prefix_mla_join_kernel(const Args a, int per_tile) {
  extern __shared__ float4 acc_s[];  // [3][kAcc][128]
  __shared__ float2 ml_s[3][kRows];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int r = threadIdx.x & (kRows - 1), y = threadIdx.x >> 7;
  int col0, n_col, row0, nrows;
  bool by_piece;
  // up to two tiles hold a row's pieces: parts a0 .. a1 of tile ta (row r), b0 .. b1 of tb (row rb)
  int ta, a0, a1, tb = 0, rb = 0, b0 = 0, b1 = -1;
  // what a packed batch needs first is read together with whether it is one: one trip to L2
  int packed = 0;
  int4 wa{}, qr{};
  if (a.may_pack) {
    packed = __ldcg(a.head + 2);
    const int rows = a.total_q * a.H;
    const int row_a = min(static_cast<int>(blockIdx.x) / per_tile * kRows + r, rows - 1);
    wa = __ldcg(reinterpret_cast<const int4*>(a.tiles + row_a / kRows) + 1);
    qr = __ldcg(reinterpret_cast<const int4*>(a.queries + row_a / a.H));
  }
  if (packed) {
    ta = blockIdx.x / per_tile;
    if (ta >= a.row_blocks) return;
    const int width = 128 / per_tile;
    by_piece = per_tile == 32;
    col0 = (blockIdx.x - ta * per_tile) * width;
    n_col = by_piece ? width : width / 4;
    if (!by_piece) col0 += y * n_col;
    row0 = ta * kRows;
    nrows = min(kRows, a.total_q * a.H - row0);
    a0 = wa.y;
    a1 = wa.z;
    if (r < nrows) {
      const int local = qr.y + (row0 + r) % a.H;
      tb = qr.x + local / kRows;
      rb = local % kRows;
      if (tb < __ldcg(a.head)) {
        const int4 v = __ldcg(reinterpret_cast<const int4*>(a.tiles + tb) + 1);
        b0 = v.y;
        b1 = v.z;
      }
    }
  } else {
    const int c = min(static_cast<int>(blockIdx.x >> 1), a.G - 1);
    const int4 w = __ldcg(reinterpret_cast<const int4*>(a.parts + c));
    nrows = __ldcg(&a.parts[c].nrows);
    const int n_tiles = __ldcg(a.head);
    if (__ldcg(a.head + 1) > 0) {  // zeros for tiles without blocks
      for (int z = blockIdx.x; z < n_tiles; z += gridDim.x) {
        if (__ldcg(&a.tiles[z].c1) >= 0) continue;
        const int z0 = __ldcg(&a.tiles[z].row0), zn = __ldcg(&a.tiles[z].nrows);
        for (int e = threadIdx.x; e < zn * (kRank / 8); e += blockDim.x)
          reinterpret_cast<uint4*>(a.out + static_cast<long long>(z0) * kRank)[e] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse && threadIdx.x < zn) a.lse[z0 + threadIdx.x] = -INFINITY;
      }
    }
    if (w.x < 0 || blockIdx.x >= 2 * a.G) return;
    ta = w.x;
    a0 = w.y;
    a1 = w.z;
    row0 = w.w;
    const int first = c - a0 - 1;  // which of the parts that begin inside the tile's blocks
    const int pieces = a1 - a0 + 1;
    const int share = pieces > 64 ? 64 : (pieces > 16 ? 16 : (pieces > 4 ? 4 : (pieces > 2 ? 2 : 1)));
    if (first < 0 || first >= share) return;  // begins with the tile (first < 0), or not needed
    const int width = 64 / share;
    by_piece = pieces > 4;
    n_col = by_piece ? width : width / 4;
    col0 = ((blockIdx.x & 1) * share + first) * width + (by_piece ? 0 : y * n_col);
  }
  const int row = row0 + r;
  const bool live = r < nrows;
  const int na = a1 - a0 + 1, np = live ? na + b1 - b0 + 1 : 0;
  const int k0 = by_piece ? y : 0, step = by_piece ? 4 : 1;
  const float2* part_ml = reinterpret_cast<const float2*>(a.part_ml);
  const float4* part_o = reinterpret_cast<const float4*>(a.part_o);
  // the same places as the pieces were left in; a whole tile's by the rows of the batch (packed: row0 = 128 ta)
  const int whole = 2 * a.G + ta, whole_b = whole + a.row_blocks;
  if (b0 == b1) rb = r;
  auto place_of = [&](int k) -> Place {  // of piece k
    const bool in_a = k < na;
    const int kk = in_a ? k : k - na, first = in_a ? a0 : b0;
    if (first == (in_a ? a1 : b1)) return {in_a ? whole : whole_b, in_a ? r : rb};
    return {2 * (first + kk) + (kk == 0 ? 1 : 0), in_a ? r : rb};
  };

  for (int q0 = 0; q0 < n_col; q0 += kAcc) {
    // running maximum, sum and columns over this thread's pieces
    float M = -INFINITY, L = 0.f;
    float4 acc[kAcc];
#pragma unroll
    for (int q = 0; q < kAcc; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = k0; k < np; k += kBatch * step) {
      float2 ml[kBatch];
      const float4* src[kBatch];
      float w[kBatch];
#pragma unroll
      for (int h = 0; h < kBatch; ++h) {
        const int kk = k + h * step;
        const Place at = place_of(min(kk, np - 1));
        const long long slot = at.slot;
        ml[h] = part_ml[slot * kRows + at.row];
        if (kk >= np) ml[h] = make_float2(-INFINITY, 0.f);
        src[h] = part_o + (slot * (kRank / 4) + col0 + q0) * kRows + at.row;
      }
      float Mn = M;
#pragma unroll
      for (int h = 0; h < kBatch; ++h) Mn = fmaxf(Mn, ml[h].x);
      const float base = Mn == -INFINITY ? 0.f : Mn;  // nothing seen so far: every weight is 0
      const float f = ptx::ex2(M - base);
      M = Mn;
      L *= f;
#pragma unroll
      for (int h = 0; h < kBatch; ++h) {
        w[h] = ptx::ex2(ml[h].x - base);
        L = fmaf(w[h], ml[h].y, L);
      }
#pragma unroll
      for (int q = 0; q < kAcc; q += 2) {
        if (q0 + q >= n_col) break;
        float4 o[kBatch][2];
#pragma unroll
        for (int h = 0; h < kBatch; ++h) {
          const bool in = k + h * step < np;
          o[h][0] = in ? src[h][q * kRows] : make_float4(0.f, 0.f, 0.f, 0.f);
          o[h][1] = in && q0 + q + 1 < n_col ? src[h][(q + 1) * kRows] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float4 v = make_float4(acc[q + e].x * f, acc[q + e].y * f, acc[q + e].z * f, acc[q + e].w * f);
#pragma unroll
          for (int h = 0; h < kBatch; ++h) {
            v.x = fmaf(w[h], o[h][e].x, v.x);
            v.y = fmaf(w[h], o[h][e].y, v.y);
            v.z = fmaf(w[h], o[h][e].z, v.z);
            v.w = fmaf(w[h], o[h][e].w, v.w);
          }
          acc[q + e] = v;
        }
      }
    }
    if (by_piece) {  // the four threads of a row meet
      if (y > 0) {
        ml_s[y - 1][r] = make_float2(M, L);
#pragma unroll
        for (int q = 0; q < kAcc; ++q)
          if (q0 + q < n_col) acc_s[((y - 1) * kAcc + q) * kRows + r] = acc[q];
      }
      __syncthreads();
      if (y == 0) {
        float Mn = M;
#pragma unroll
        for (int h = 0; h < 3; ++h) Mn = fmaxf(Mn, ml_s[h][r].x);
        const float base = Mn == -INFINITY ? 0.f : Mn;
        const float f = ptx::ex2(M - base);
        M = Mn;
        L *= f;
#pragma unroll
        for (int q = 0; q < kAcc; ++q) acc[q] = make_float4(acc[q].x * f, acc[q].y * f, acc[q].z * f, acc[q].w * f);
#pragma unroll
        for (int h = 0; h < 3; ++h) {
          const float w = ptx::ex2(ml_s[h][r].x - base);
          L = fmaf(w, ml_s[h][r].y, L);
#pragma unroll
          for (int q = 0; q < kAcc; ++q) {
            if (q0 + q >= n_col) break;
            const float4 v = acc_s[(h * kAcc + q) * kRows + r];
            acc[q].x = fmaf(w, v.x, acc[q].x);
            acc[q].y = fmaf(w, v.y, acc[q].y);
            acc[q].z = fmaf(w, v.z, acc[q].z);
            acc[q].w = fmaf(w, v.w, acc[q].w);
          }
        }
      }
      __syncthreads();
    }
    if (!live || (by_piece && y > 0)) continue;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint2* dst = reinterpret_cast<uint2*>(a.out + static_cast<long long>(row) * kRank + (col0 + q0) * 4);
    auto packed = [&](const float4& v) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * inv, v.y * inv), hi = __floats2bfloat162_rn(v.z * inv, v.w * inv);
      return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    };
#pragma unroll
    for (int q = 0; q < kAcc; q += 2) {  // columns come in pairs, but for a single one
      if (q0 + q >= n_col) break;
      const uint2 u = packed(acc[q]), v = packed(acc[q + 1]);
      if (n_col == 1) dst[q] = u;
      else *reinterpret_cast<uint4*>(dst + q) = make_uint4(u.x, u.y, v.x, v.y);
    }
    if (a.lse && col0 + q0 == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
  }
}
constexpr int kJoinSmem = 3 * kAcc * kRows * 16;

// CTA pairs that run at once (one per two SMs, less where a cluster does not fit), per device.
int pair_count() {
  int dev = 0;
  static int cached[64] = {};
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 76;
  if (cached[dev] == 0) {
    int n = 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(prefix_mla_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmem)) != cudaSuccess ||
        cudaFuncSetAttribute(prefix_mla_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmem)) != cudaSuccess ||
        cudaFuncSetAttribute(prefix_mla_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kJoinSmem) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, prefix_mla_kernel<false>, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      return 76;
    }
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
  // rows, cache rows and positions are counted in 32 bits, with room for a tile or block behind them
  if (static_cast<long long>(a->total_q) * a->H > 0x7FFFFFFFLL - kRows ||
      static_cast<long long>(a->num_pages) * a->page_size > 0x7FFFFFFFLL - kKeys || a->prefix_len > kMaxKeys)
    return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

struct Layout {
  int may_pack, max_tiles, G;
  size_t off_tiles, off_u0, off_head, off_parts, off_queries, off_ml, off_o, total;
};

Layout layout(const dsa_prefix_mla_args* a) {
  Layout p{};
  const long long rows = static_cast<long long>(a->total_q) * a->H;
  // Whether requests share prefix tiles is for the plan to say, from the lengths: where their own
  // tiles, sum ceil(rows / 128), come to more than 1.15 times the rows.  That sum is at most
  // (rows + 127 B) / 128, so batches of 15 rows > 12700 B never do, and need no room for it.
  p.may_pack = a->prefix_len > 0 && a->B > 1 && a->H % kRows != 0 && 15 * rows <= 12700LL * a->B ? 1 : 0;
  p.max_tiles = static_cast<int>((p.may_pack ? 2 : 1) * (rows / kRows + 1) + a->B + 1);
  p.G = pair_count();
  const size_t slots = 2 * static_cast<size_t>(p.G) + (p.may_pack ? 2 * ((rows + kRows - 1) / kRows) : 0);
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  p.off_tiles = 0;
  p.off_u0 = up(p.off_tiles + sizeof(Tile) * p.max_tiles);
  p.off_head = up(p.off_u0 + 8 * (static_cast<size_t>(p.max_tiles) + 1));
  p.off_parts = up(p.off_head + 4 * (static_cast<size_t>(a->B) + 4));
  p.off_queries = up(p.off_parts + sizeof(Part) * p.G);
  p.off_ml = up(p.off_queries + (p.may_pack ? sizeof(Query) * a->total_q : 0));
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
  // (strides of one query, of one head, lead nowhere)
  if ((a->total_q > 1 && (a->qn_stride_t % 8 || a->qr_stride_t % 8)) ||
      (a->H > 1 && (a->qn_stride_h % 8 || a->qr_stride_h % 8)))
    return DSA_ERR_INVALID_ARGUMENT;
  const Layout p = layout(a);
  if (!a->workspace || a->workspace_bytes < p.total || !al(a->workspace, 16)) return DSA_ERR_WORKSPACE;
  unsigned* status = device_status_ptr();
  if (!status) return DSA_ERR_CUDA;
  CUtensorMap tc, tr;
  const long long slots = std::max(1LL, static_cast<long long>(a->num_pages) * a->page_size);
  const int box = std::min(a->page_size, 64);
  if (!make_map_2d(&tc, a->cache_c, false, kRank, slots, box) || !make_map_2d(&tr, a->cache_r, false, kRope, slots, box))
    return DSA_ERR_CUDA;
  Args k{};
  k.B = a->B;
  k.total_q = a->total_q;
  k.H = a->H;
  k.page_size = a->page_size;
  k.page_log2 = a->page_size == 16 ? 4 : (a->page_size == 32 ? 5 : (a->page_size == 64 ? 6 : 7));
  k.num_pages = a->num_pages;
  k.max_pages = a->max_pages_per_seq;
  k.prefix_len = a->prefix_len;
  k.num_prefix_pages = a->num_prefix_pages;
  k.may_pack = p.may_pack;
  k.max_tiles = p.max_tiles;
  k.G = p.G;
  k.past_row = static_cast<int>(slots);
  const long long groups = (static_cast<long long>(a->total_q) * a->H + kRows - 1) / kRows;
  k.row_blocks = static_cast<int>(groups);
  k.room = static_cast<int>(std::min(std::max(static_cast<long long>(a->max_pages_per_seq) * a->page_size,
                                              static_cast<long long>(a->prefix_len)), static_cast<long long>(kMaxKeys)));
  const long long most = k.room / kKeys + 2 + kSetup;
  k.narrow = most * p.max_tiles < (1LL << 31) ? 1 : 0;
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
  k.parts = reinterpret_cast<Part*>(ws + p.off_parts);
  k.queries = reinterpret_cast<Query*>(ws + p.off_queries);
  k.part_ml = reinterpret_cast<float*>(ws + p.off_ml);
  k.part_o = reinterpret_cast<float*>(ws + p.off_o);
  k.status = status;
  const Probe probe = armed_probe();
  armed_probe() = Probe{0, 0, 0};
  k.probe_site = probe.site;
  k.probe_at = probe.at;
  k.probe_cycles = 2 * static_cast<long long>(probe.limit_ns);  // some 2 cycles a nanosecond
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_pdl(prefix_mla_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, k);
  if (e != cudaSuccess) return DSA_ERR_CUDA;
  e = launch_pdl(probe.site != 0 ? prefix_mla_kernel<true> : prefix_mla_kernel<false>, dim3(2 * p.G), dim3(kThreads), kSmem, s, tc, tr, k);
  if (e != cudaSuccess) return DSA_ERR_CUDA;
  // Few packed tiles have many pieces each: 32 CTAs a tile, which split them.
  const int per_tile = groups * 32 <= 2LL * p.G ? 32 : (groups * 8 <= 2LL * p.G ? 8 : 4);
  const long long ctas = std::max(p.may_pack ? groups * per_tile : 0LL, p.G * 2LL);
  e = launch_pdl(prefix_mla_join_kernel, dim3(static_cast<unsigned>(ctas)), dim3(512), kJoinSmem, s, k, per_tile);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

dsa_status dsa_test_arm_prefix_mla_timeout(int site, unsigned at, unsigned long long limit_ns) {
  const int role = site & ~kProbeOdd;
  if (role < kProbeMma || role > kProbeSoftmax || site == kProbeMma + kProbeOdd || limit_ns > 1000000000ull)
    return DSA_ERR_INVALID_ARGUMENT;
  armed_probe() = limit_ns == 0 ? Probe{0, 0, 0} : Probe{site, at, limit_ns};
  return DSA_OK;
}

}  // extern "C"
