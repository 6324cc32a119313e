// quant_mla.cu -- multi-head latent attention over the quantised latent cache.
//
//     logit[t, h, s] = scale * (q_nope[t, h] . c[s] + q_rope[t, h] . r[s])
//     out[t, h]      = sum_s softmax_s(logit[t, h, :]) c[s],   lse[t, h] = ln sum_s exp(logit[t, h, s])
//
// over the selected positions s = topk[t, j] of the query's sequence, or over every position up to its own.
//
// Both formats are e4m3 numbers times a row's power of two, c[s] = 2^E c8[s], r[s] = 2^E r8[s], so the tensor
// cores take the cache's codes as they are, and nothing is converted to bf16:
//   q = 2^-a (hi + 2^-4 lo) in two e4m3 rows, the largest value of a row in [128, 256): exact for what lies within 2^13
//   of that, 2^-21 of it off otherwise:
//       S = hi . c8 + 2^-4 lo . c8 + (2^a q_rope) . r8,   x = S 2^(E - a) scale log2(e)
//   x' = x + E - kExpRef,  m' its running maximum,  p = 2^(x' - m' + kPShift) in an e4m3 and an e5m2 term (two_terms):
//       O = sum p c8,  L = sum p 2^(kExpRef - E) (fp32, of the unrounded p),  out = 2^kExpRef O / L
// Two 8-bit planes cost the tensor cores what one bf16 plane does and half the shared memory traffic.  Taking E
// into the maximum keeps p in range whatever the rows' scales are.  On random rows, against 64 bits, the output's root mean
// square error is 0.0017 to 0.0021 of its size (the most with few keys), 0.00166 of which is its own rounding to bf16; lse is
// off by 2e-6 at most, 3e-7 to 5e-7 on average.
//
// Work: a tile is a query and up to 64 heads, its keys are cut into blocks of 64; how tiles come to CTAs stands at Pieces.
// A tile done in one piece is normalised and written; the pieces of the others, (O, m', L) in fp32, are joined by the CTAs of
// a cluster that hold them, or else go through memory to a second kernel.  Roles of a CTA:
//   warps 0..7    softmax, two groups that take 32 keys each of every block.  Rows of S alternate between 16 hi and
//                 16 lo rows, so that a lane and the one 16 further hold a head's two planes; each adds the planes
//                 for half of its group's keys.  (Alternate blocks to the groups took 1 % less for the first figure
//                 below, but 6 % more for 62 x 128 heads x 1001 keys in 4 bits, and 4 % more for the other 4-bit
//                 cases: there the time from S to P is what counts);
//   warps 8..11   query rows: bf16 -> hi, lo in TMEM (A operand), 2^a q_rope in shared memory;
//                 4-bit rows also: codes from the staged rows to e4m3 tiles;
//   warps 12, 15  rows of the cache by gathering TMA: e4m3 tiles in 128-byte columns, 4-bit rows whole;
//   warp 13       TMEM, MMAs:  S [128 x 64 keys] = Q (TMEM) . K^T,  O^T [512 x heads] += V^T (the same tile,
//                 MN-major) . P^T;
//   warp 14       where the rows lie, four blocks at a time; e4m3: their scales.
// A tile in shared memory serves both products, so a key is fetched once for 64 heads: at 64 heads an e4m3 row of 656
// bytes meets 128 x 576 + 2 x 64 x 512 multiplications.
//
// What bounds it (GB300, 1.9 GHz, captured in a graph):
//   block     the MMAs of a block take the tensor pipe for 1150 cycles.  e4m3: 2070 a block, by the softmax (some 350
//             instructions a warp, each waiting for the one before, and a barrier) and the four tiles in flight: a tile is gathered
//             (950 cycles from L2, 1430 with one issuing warp less), waits its turn, is multiplied twice and freed; 2430 a
//             block when rows come from DRAM.  1127 queries x 64 heads x 2048 keys: 316 us, the tensor pipe active for 46 % of
//             them, 166 at the tensor cores' rate.  4 bits: three tiles, and decoding stands in the round: 2600 a block.
//   piece     some 8000 to 10000 cycles before a CTA's first MMA (launch, queries, look-up, first rows), 10000 from a
//             piece's last product to the next one's first (next queries 6000, then their first block's softmax; the
//             output, 6000, beside them).  64 queries x 64 heads x 2048 keys: 44.5 us (e4m3) and 43 (4 bits), 14 and 9 at
//             the copy bandwidth.
//   join      in a cluster 3 us; through memory 7 to 14, 2 of which its CTAs wait for room.
// Every wait is bounded; after one gives up, every role stops, the MMAs and copies in flight are drained (bounded; with any
// role's wait made to run out, a call ends some 0.1 ms later), the CTAs of a cluster meet all the same and TMEM is freed.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "internal.h"
#include "ptx.cuh"
#include "quant_rows.cuh"

namespace dsa {
namespace {

using namespace quant;

constexpr int kHeads = 64;                                // heads per tile
constexpr int kKeys = 64;                                 // keys per block
constexpr int kThreads = 512;
constexpr uint32_t kAtom = kKeys * 128;                   // 64 rows of 128 bytes
constexpr uint32_t kTile = 5 * kAtom;                     // 4 columns of 128 codes, one of 64 bf16
constexpr uint32_t kStaged = kKeys * kRow4;               // a block of 4-bit rows
constexpr uint32_t kQRope = 128 * 128, kPBytes = kHeads * 128;
constexpr uint32_t kQStride = 80, kQBuf = 4 * 32 * kQStride;  // 64 codes of 32 query rows a warp, 16 bytes apart further
constexpr uint32_t kBe5m2 = 1u << 10;                     // instruction descriptor: B holds e5m2
constexpr uint32_t kColQ = 0, kColS = 128, kColO = 256;   // TMEM columns
constexpr int kPShift = 5;                                // p = 2^5 at the reference maximum
constexpr float kMove = 3.f;                              // the reference moves when passed by more: p <= 2^8
constexpr int kFewHeads = 12;                             // rescaled one by one (130 cycles each; all at once 2000)
constexpr int kLoShift = 4;                               // lo = 2^4 (x - hi): below 2^4 of its step it is exact, and 2^7 at most
constexpr int kExpRef = -7;                               // E of normalised rows: x' counts from there, so that it does not lose x's bits
constexpr float kLn2 = 0.6931471805599453f;
constexpr long long kMostKeys = 0x7FFFFF00ll;             // that a query sees: a key of its last blocks fits 32 bits, and of three behind them
constexpr int kMaxStages = 4;
constexpr int kQRing = 4;                                 // scales of the queries of consecutive pieces
constexpr int kBatch = 4, kBatches = 4, kRing = kBatch * kBatches;  // blocks of a piece whose rows are looked up together

template <bool FP4>
struct Smem {
  static constexpr int kStages = FP4 ? 3 : 4;             // tiles
  static constexpr int kAhead = kStages - 2;              // blocks that S runs ahead of P . V: a tile is always left to fill
  static constexpr int kPBufs = kAhead + 1;               // S of block b is issued behind P . V of b - kPBufs, whose P it then replaces
  static constexpr int kStagedBufs = FP4 ? 2 : 0;
  static constexpr int kScRing = FP4 ? kStages : kRing;   // blocks whose scales are held
  static constexpr uint32_t kOffTile = 0, kOffQr = kOffTile + kStages * kTile, kOffP = kOffQr + kQRope;
  static constexpr uint32_t kOffStaged = kOffP + kPBufs * kPBytes, kOffQ = kOffStaged + kStagedBufs * kStaged;
  static constexpr uint32_t kOffMisc = kOffQ + kQBuf, kOffRows = kOffMisc + 5120, kOffSc = kOffRows + kRing * kKeys * 4;
  static constexpr uint32_t kOffLevels = kOffSc + kScRing * kKeys * 8;  // 4 bits: magnitudes by the scale's byte
  static constexpr uint32_t kBytes = kOffLevels + (FP4 ? 256 * 8 : 0);
};
static_assert(Smem<false>::kBytes <= 232448 && Smem<true>::kBytes <= 232448, "shared memory of a CTA");

struct Args {
  int B, total_q, H, groups, page_size, num_pages, max_pages, topk_width;
  int nb;                  // blocks of a tile (selected keys)
  int most_live;           // total_q; 0 without requests, where there are no lengths to look at
  int parts;               // CTAs
  int whole, rest, split;  // selected keys: whole tiles a CTA, tiles behind them, pieces of each
  int cluster;             // CTAs that hold the pieces of a tile and join them among themselves (1: the pieces go through memory)
  int past_row;            // a row past the cache: copies from there are zeros
  unsigned long long page_mul;  // position / page_size = position * page_mul >> page_shift
  int page_shift;
  float scale_log2;        // scale * log2(e)
  const __nv_bfloat16 *qn, *qr;
  long long qn_t, qn_h, qr_t, qr_h;
  const uint8_t* cache;
  const int32_t *block_tables, *cu, *lens, *topk;
  const long long* cum;    // [total_q + 1] blocks before each query (every position)
  __nv_bfloat16* out;
  float* lse;
  float *part_o, *part_ml; // pieces: [slot][4][16][128][4] (latent chunk, four heads, latent, head), [slot][64][2]
  int2* joins;             // [parts] the tile that a part begins inside, if no earlier one does (-1: none), its last part
  unsigned* status;
  // failure-path test hook: a role waits, at probe_at, for what never comes
  int probe_site;
  uint32_t probe_at;
  long long probe_cycles;
};

// Roles whose waits the test hook can let run out: before a block (MMAs; either copying warp; decoding; softmax), a batch of
// look-ups or a piece's queries, in the CTAs of even number; + kProbeOdd: in the others.
enum : int { kProbeMma = 1, kProbeCopy = 2, kProbeCopy2 = 3, kProbeRows = 4, kProbeQueries = 5, kProbeDecode = 6, kProbeSoftmax = 7, kProbeOdd = 8 };
struct Probe {
  int site;
  uint32_t at;
  unsigned long long limit_ns;
};
Probe& armed_probe() {
  static thread_local Probe p{0, 0, 0};
  return p;
}

struct Bars {
  uint64_t tfull[kMaxStages], tempty[kMaxStages];
  uint64_t rfull[kBatches], bempty[kBatches], scfull[kBatches];
  uint64_t gfull[2], gempty[2];           // staged 4-bit rows
  uint64_t qfull[kQRing], qfree;
  uint64_t sfull[2], sempty[2], pfull[2], pvdone[2], odrained, done;
  uint64_t never;                         // test hook: nothing arrives
};

// Rows of queries; the others are padding.
__device__ __forceinline__ int live_rows(const Args& a) { return min(__ldg(a.cu + a.B), a.most_live); }

// Keys that a query at place i of the last q of n tokens sees (every position): those up to its own that the table
// covers.
__device__ __forceinline__ long long keys_seen(const Args& a, long long pos, bool report) {
  const long long n = pos + 1, room = min(static_cast<long long>(a.max_pages) * a.page_size, kMostKeys);
  if (n > room && report) atomicOr(a.status, kStatusUncovered);
  return max(0ll, min(n, room));
}

// Tile w: query w / groups, its heads 64 (w % groups) ..  How the tiles come to the CTAs:
//
// Selected keys (every tile of nb blocks): CTA c takes the whole tiles c * whole .. and then, of the `rest` tiles that
// do not fill a round of all CTAs, piece c % split of tile c / split.  Cutting no more tiles than that: a piece costs
// some six blocks beside its own (its queries, its output), and a cut one is read again by the join.
//
// Every position (blocks by the queries' lengths): the blocks of all tiles stand in one line, tile w at the places
// tile_begin(w) .. tile_begin(w + 1) - 1, cut into parts of `size` places, the first `more` of them of one more.
struct Line {
  long long size;
  int more, parts;
  __device__ __forceinline__ long long begin(int c) const { return size * c + min(c, more); }
  __device__ __forceinline__ int part_at(long long u) const {
    const long long first = (size + 1) * more;
    return static_cast<int>(u < first ? u / (size + 1) : more + (u - first) / size);
  }
};
__device__ __forceinline__ long long tile_begin(const Args& a, int w) {
  const int t = w / a.groups, g = w - t * a.groups;
  const long long c0 = __ldg(a.cum + t);
  return c0 * a.groups + (g ? g * (__ldg(a.cum + t + 1) - c0) : 0);
}
__device__ __forceinline__ Line line_of(const Args& a) {
  const long long total = tile_begin(a, a.total_q * a.groups);
  Line l;
  l.parts = static_cast<int>(min(static_cast<long long>(a.parts), total));
  l.size = total / l.parts;
  l.more = static_cast<int>(total - l.size * l.parts);
  return l;
}
// The tile that holds place u.
__device__ __forceinline__ int tile_at(const Args& a, long long u) {
  int lo = 0, hi = a.total_q * a.groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile_begin(a, mid) <= u) lo = mid; else hi = mid;
  }
  return lo;
}

// The pieces of a CTA, in order; every role walks them by itself.
template <bool ALL>
struct Pieces;
template <>
struct Pieces<false> {
  int w, t, g, k0, k1 = 0, blocks;  // the current piece: blocks k0 .. k1 - 1 of `blocks`
  int c, q = 0;
  __device__ __forceinline__ Pieces(const Args& a, int part) : blocks(a.nb), c(part) {}
  __device__ __forceinline__ bool next(const Args& a) {
    k0 = 0;
    k1 = blocks;
    if (q < a.whole) {
      w = c * a.whole + q;
    } else {
      if (q > a.whole || c >= a.rest * a.split) return false;
      const int r = c / a.split, j = c - r * a.split;
      w = a.parts * a.whole + r;
      k0 = static_cast<int>(static_cast<long long>(blocks) * j / a.split);
      k1 = static_cast<int>(static_cast<long long>(blocks) * (j + 1) / a.split);
    }
    ++q;
    t = w / a.groups;
    g = w - t * a.groups;
    return true;
  }
};
template <>
struct Pieces<true> {
  long long u, end, t_end;  // the next piece's first place, the part's end, its tile's end
  int w, t, g, k0, k1 = 0, blocks;
  __device__ __forceinline__ Pieces(const Args& a, int part) {
    const Line l = line_of(a);
    u = part < l.parts ? l.begin(part) : 0;
    end = part < l.parts ? l.begin(part + 1) : 0;
    w = u < end ? tile_at(a, u) : 0;
    --w;
  }
  __device__ __forceinline__ bool next(const Args& a) {
    if (u >= end) return false;
    ++w;
    const long long b = tile_begin(a, w);
    t_end = tile_begin(a, w + 1);
    t = w / a.groups;
    g = w - t * a.groups;
    blocks = static_cast<int>(t_end - b);
    k0 = static_cast<int>(u - b);
    k1 = static_cast<int>(min(end, t_end) - b);
    u = b + k1;
    return true;
  }
};

// A piece's blocks are looked up in batches: how many, and whether block i (from the piece's first) ends one.
template <typename P>
__device__ __forceinline__ int batches(const P& p) { return (p.k1 - p.k0 + kBatch - 1) / kBatch; }
template <typename P>
__device__ __forceinline__ bool last_of_batch(const P& p, int i) { return i % kBatch == kBatch - 1 || i == p.k1 - p.k0 - 1; }
// The request of query t: the last b < B with cu[b] <= t, by a whole warp, 32 places a look.
__device__ __forceinline__ int request_of(const int32_t* cu, int B, int t, int lane) {
  int lo = 0, n = B;  // among lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 31) >> 5, at = lane * step;
    const unsigned below = __ballot_sync(0xffffffffu, at < n && __ldg(cu + lo + at) <= t);
    const int last = below ? 31 - __clz(below) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}
// The keys of a query.  Queries come in ascending order, so the request is searched for once and then walked to.
struct Keys {
  int t = -1, b = -1, hi = 0, len = 0, live = 0;
  long long n = 0;  // keys
  __device__ __forceinline__ void move(const Args& a, bool all, int query, int lane) {
    if (query == t) return;
    t = query;
    if (b < 0) {
      live = live_rows(a);
      b = t < live ? request_of(a.cu, a.B, t, lane) : 0;
      hi = t;
    } else {
      while (t < live && t >= hi && b + 1 < a.B && __ldg(a.cu + b + 1) <= t) ++b;
    }
    if (t < live && t >= hi) {
      hi = __ldg(a.cu + b + 1);
      len = __ldg(a.lens + b);
    }
    n = t >= live ? 0 : all ? keys_seen(a, static_cast<long long>(len) - hi + t, lane == 0) : a.topk_width;
  }
};
// The cache row of a position, through a request's table; a.past_row where there is none (*bad: its page is not there).
__device__ __forceinline__ int row_of(const Args& a, const int32_t* table, int pos, bool* bad) {
  const int lp = static_cast<int>(static_cast<unsigned long long>(static_cast<unsigned>(pos)) * a.page_mul >> a.page_shift);
  const int page = pos >= 0 && lp < a.max_pages ? __ldg(table + lp) : -1;
  const bool there = static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages);
  *bad |= pos >= 0 && !there;
  return there ? page * a.page_size + (pos - lp * a.page_size) : a.past_row;
}

// D[tmem] (+)= A . B[smem]^T: A e4m3 in TMEM, e4m3 or bf16 in shared memory.  Operands in shared memory are given by the
// low words of their descriptors; the high word is the same for all (128-byte swizzle, K-major or MN-major).
__device__ __forceinline__ void mma_f8_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tmov.b64 db, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], db, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b_lo), "r"(idesc),
      "r"(accumulate), "n"(ptx::kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_f8_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d), "r"(a_lo),
      "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(ptx::kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_bf16_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d), "r"(a_lo),
      "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(ptx::kDescHi)
      : "memory");
}
// Four rows of 128 bytes from column x on, into 512 bytes of a 128-byte swizzled tile.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* m, uint64_t* bar, int x, const int (&y)[4]) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(ptx::smem_u32(bar)), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
      : "memory");
}

// A wait that did not succeed at once (one copy of its code for all of them).
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* status) {
  return ptx::mbar_spin(bar, parity, abort, status, kStatusTimeout);
}
// Whether v is non-zero in any of the 256 threads at named barrier `id`.
__device__ __forceinline__ bool bar_any(uint32_t id, uint32_t v) {
  uint32_t any;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.or.pred p, %2, 256, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(any) : "r"(v), "r"(id) : "memory");
  return any != 0;
}
// One column of 32 lanes.
__device__ __forceinline__ float tmem_ld_x1(uint32_t taddr) {
  float r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=f"(r) : "r"(taddr));
  return r;
}
__device__ __forceinline__ void tmem_st_x1(uint32_t taddr, float r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "f"(r) : "memory");
}
__device__ __forceinline__ void tmem_ld_wait4(float (&r)[4]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]) : : "memory");
}
// Four values 0 <= p <= 2^8 in fp16 as e4m3 codes (x) and the e5m2 codes of what they leave (y).
// 2^-8 p has e4m3's exponents as its low four and its subnormals where e4m3 has them, so rounding its bits to three
// of the mantissa is the code; e5m2 is the upper half of fp16.  (Conversions take the slow pipe, integers do not.)
// Together they are within 2^-7 of p.  Below e4m3's normal numbers, p < 2^-6, the second term's two bits are all that
// counts, and its step is 2^-12 to 2^-16.  Thousands of such keys behind a large one may be alike, and their errors with them, or
// all less than half a step, so there the rounding goes up for as many keys as it should: a key's threshold among the 256 that
// fp16 has in a step is 16 times its place among 16 in bit-reversed order (`at`: of the first of the four), its bits changed by
// the hash of the sixteen (`change`), so that keys at a regular distance are not rounded alike.  What is lost is fp16's: p
// below 2^-25, 2^-30 of the largest, and up to 2^-25 of others.
__device__ __forceinline__ constexpr uint32_t round_at(int i) {  // 16 thresholds of a step, in bit-reversed order
  return 16u * ((i & 1) << 3 | (i & 2) << 1 | (i & 4) >> 1 | (i & 8) >> 3);
}
__device__ __forceinline__ uint32_t threshold_change(int sixteen) {
  return __byte_perm(static_cast<uint32_t>(sixteen) * 0x9E3779B9u, 0u, 0x4242);  // (2^32 over the golden ratio)
}
__device__ __forceinline__ uint32_t first_term(__half2 p) {  // in 2^-8
  const __half2 v = __hmul2(p, __float2half2_rn(0.00390625f));
  return (*reinterpret_cast<const uint32_t*>(&v) + 0x00400040u) & 0x7F807F80u;
}
__device__ __forceinline__ uint32_t second_term(__half2 p, uint32_t first, int at, uint32_t change) {
  const __half2 left = __hfma2(*reinterpret_cast<const __half2*>(&first), __float2half2_rn(-256.f), p);  // (exact)
  const uint32_t small = __hlt2_mask(p, __float2half2_rn(0.015625f));  // p < 2^-6
  const uint32_t spread = (round_at(at) | round_at(at + 1) << 16) ^ 0x00800080u;
  return *reinterpret_cast<const uint32_t*>(&left) + ((small & (spread ^ change)) ^ 0x00800080u);
}
__device__ __forceinline__ uint2 two_terms(__half2 a, __half2 b, int at, uint32_t change) {
  const uint32_t fa = first_term(a), fb = first_term(b);
  return make_uint2(__byte_perm(fa << 1, fb << 1, 0x7531),
                    __byte_perm(second_term(a, fa, at, change), second_term(b, fb, at + 2, change), 0x7531));
}
// Four values |x| < 2^8 as e4m3 codes (x) and as those of 2^kLoShift times what they leave (y).  (By conversions, which are
// fewer instructions: the warps that do this have a scheduler each, and the softmax is not at work beside them.)
__device__ __forceinline__ uint32_t to_e4m3x2(__half2 v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&v)));
  return r;
}
__device__ __forceinline__ __half2 half2_of_e4m3x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return *reinterpret_cast<const __half2*>(&r);
}
__device__ __forceinline__ uint2 two_planes(__half2 a, __half2 b) {
  const uint32_t ha = to_e4m3x2(a), hb = to_e4m3x2(b);
  const __half2 up = __float2half2_rn(1 << kLoShift);
  return make_uint2(ha | hb << 16, to_e4m3x2(__hmul2(__hsub2(a, half2_of_e4m3x2(ha)), up)) |
                                       to_e4m3x2(__hmul2(__hsub2(b, half2_of_e4m3x2(hb)), up)) << 16);
}
// The largest magnitudes among 8 bf16 values, in two halves.
__device__ __forceinline__ __nv_bfloat162 most(const uint4& v) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
  return __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])), __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
}
// The top bits of four bytes, the first byte's lowest.
__device__ __forceinline__ int top_bits(uint32_t x) { return static_cast<int>((x >> 7 & 0x01010101u) * 0x01020408u >> 24 & 15u); }
// Scale u = 2^E of a block's row `key` (0: no row, which takes no weight).
__device__ __forceinline__ void put_scale(float4* block, int key, float u) {
  float* pair = reinterpret_cast<float*>(block + (key >> 1)) + (key & 1);
  pair[0] = u;
  pair[2] = u > 0.f ? static_cast<float>(static_cast<int>(__float_as_uint(u) >> 23) - 127 - kExpRef) : -INFINITY;
}
// The same of a row of zeros.  Its own E is 0, which stays in u (its rotary part is in these units), marked by the last bit;
// in x' it takes kZeroExp: it adds nothing to O, and with E = 0, seven octaves above normalised rows, one that is ahead would
// push the others' p below the smallest that the product takes.
constexpr int kZeroExp = -kMaxExp;
__device__ __forceinline__ void put_scale_of_zeros(float4* block, int key) {
  float* pair = reinterpret_cast<float*>(block + (key >> 1)) + (key & 1);
  pair[0] = __uint_as_float(0x3F800001u);
  pair[2] = static_cast<float>(kZeroExp - kExpRef);
}
// Of the rows `rows[32 j + lane]` (e4m3) whose bits j are set in a lane's `of`, those whose codes are all zeros.  Only rows of
// E = 0 are asked about.  Another row of that scale is told by its first codes as a rule; the rest are looked at by the
// whole warp, eight at a time.  (1100 x 64 heads x 2048 keys: 3 % more time where every row has E = 0, 4 % where one in a hundred
// is zeros, three times as much where all are.)
__device__ __noinline__ unsigned rows_of_zeros(const uint8_t* cache, const int* rows, unsigned of, int lane) {
  uint4 first[2 * kBatch];
#pragma unroll
  for (int j = 0; j < 2 * kBatch; ++j) {
    first[j] = make_uint4(0u, 0u, 0u, 0u);
    if (of >> j & 1) first[j] = __ldg(reinterpret_cast<const uint4*>(cache + static_cast<long long>(rows[32 * j + lane]) * kRow8));
  }
#pragma unroll
  for (int j = 0; j < 2 * kBatch; ++j)
    if ((first[j].x | first[j].y | first[j].z | first[j].w) & 0x7F7F7F7Fu) of &= ~(1u << j);
  unsigned found = 0u;
#pragma unroll 1
  for (int j = 0; j < 2 * kBatch; ++j) {
    unsigned left = __ballot_sync(0xffffffffu, of >> j & 1u);
    while (left) {
      uint4 v[8];
      int at[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        at[i] = left ? __ffs(static_cast<int>(left)) - 1 : -1;
        left &= left - 1;
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (at[i] >= 0) v[i] = __ldg(reinterpret_cast<const uint4*>(cache + static_cast<long long>(rows[32 * j + at[i]]) * kRow8) + lane);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool some = __any_sync(0xffffffffu, ((v[i].x | v[i].y | v[i].z | v[i].w) & 0x7F7F7F7Fu) != 0u);
        if (at[i] == lane && !some) found |= 1u << j;
      }
    }
  }
  return found;
}
__device__ __forceinline__ float2 add2(float2 a, float b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b));
  return d;
}
// 16 columns of 32 lanes, and the wait for earlier loads (the registers tied to it).
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16], uint32_t (&q)[16]) {
  tmem_ld_wait16(r);
  tmem_ld_wait16(q);
}
// 64 codes of 32 rows: thread i writes 16 columns of lane (base + i).
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// out = sum_j 2^(m_j - M) O_j / sum_j 2^(m_j - M) L_j over the pieces j of a tile, in their order, which the CTAs of a cluster
// hold: each takes a part of the heads and gets the others' O for it through distributed shared memory (their tiles are
// free by then), so that the pieces are neither written to memory nor joined by another launch.  All threads.
struct Held {
  float m, sum;
};
__device__ __noinline__ void join_in_cluster(const Args& a, uint8_t* tiles, uint8_t* room, uint32_t* to, const Held* held, uint32_t tmem) {
  const int C = a.cluster, rank = static_cast<int>(ptx::cluster_ctarank()), tid = threadIdx.x;
  const int tile = a.parts * a.whole + static_cast<int>(blockIdx.x) / C;
  const int t = tile / a.groups, g = tile - t * a.groups, hg = min(kHeads, a.H - g * kHeads), per = (hg + C - 1) / C;
  float* got = reinterpret_cast<float*>(tiles);                 // [C - 1][per][512], the others' in their order
  Held* stats = reinterpret_cast<Held*>(room);                  // [C][64]
  float* weights = reinterpret_cast<float*>(stats + C * kHeads);  // [C][64]
  ptx::cluster_sync();  // every CTA is done with its tiles
  if (tid < C * kHeads) {
    const int h = tid & (kHeads - 1), dst = tid / kHeads;
    const uint32_t at = ptx::mapa_shared(ptx::smem_u32(stats + rank * kHeads + h), dst);
    ptx::st_shared_cluster(at, __float_as_uint(held[h].m));
    ptx::st_shared_cluster(at + 4, __float_as_uint(held[h].sum));
  }
  if (tid < kHeads) {
    const int dst = tid / per, slot = rank < dst ? rank : rank - 1;
    to[tid] = tid < hg && dst != rank ? ptx::mapa_shared(ptx::smem_u32(got + (slot * per + tid - dst * per) * kRank), dst) : 0u;
  }
  __syncthreads();
  const int lane = tid & 31, quarter = (tid >> 5) & 3, chunk = tid >> 7, lat = chunk * 128 + quarter * 32 + lane;
  const uint32_t o = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + kColO + chunk * kHeads;
#pragma unroll 1
  for (int h0 = 0; h0 < hg; h0 += 16) {
    uint32_t r[16];
    tmem_ld_x16(o + h0, r);
    tmem_ld_wait16(r);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t at = to[h0 + j];
      if (at) ptx::st_shared_cluster(at + lat * 4, r[j]);
    }
  }
  ptx::cluster_sync();  // (nothing is written to another CTA from here on)
  const int first = rank * per, mine = min(per, hg - first);
  if (tid < mine) {
    const int h = first + tid;
    float M = -INFINITY, total = 0.f;
    for (int j = 0; j < C; ++j) M = fmaxf(M, stats[j * kHeads + h].m);
    for (int j = 0; j < C; ++j) {
      const Held s = stats[j * kHeads + h];
      const float f = s.m == -INFINITY ? 0.f : exp2f(s.m - M);
      total += f == 0.f ? 0.f : f * s.sum;
      weights[j * kHeads + tid] = f;
    }
    for (int j = 0; j < C; ++j) weights[j * kHeads + tid] = total == 0.f ? 0.f : weights[j * kHeads + tid] * (pow2f(kExpRef) / total);
    if (a.lse) a.lse[static_cast<long long>(t) * a.H + g * kHeads + h] = total == 0.f ? -INFINITY : (M - kPShift + log2f(total)) * kLn2;
  }
  __syncthreads();
  const bool odd = lane & 1;
  __nv_bfloat16* out = a.out + (static_cast<long long>(t) * a.H + g * kHeads + first + odd) * kRank + (lat & ~1);
#pragma unroll 1
  for (int i0 = 0; i0 < mine; i0 += 4) {
    float own[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) own[i] = tmem_ld_x1(o + min(first + i0 + i, kHeads - 1));
    tmem_ld_wait4(own);
#pragma unroll 1
    for (int j = 0; j < C; ++j) {
      const float* v = got + (j < rank ? j : j - 1) * per * kRank + lat;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = min(i0 + i, mine - 1);
        const float f = weights[j * kHeads + h];
        acc[i] = fmaf(f, f == 0.f ? 0.f : j == rank ? own[i] : v[h * kRank], acc[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const float x = __shfl_xor_sync(0xffffffffu, odd ? acc[i] : acc[i + 1], 1);
      const uint32_t v = odd ? pack_bf16(x, acc[i + 1]) : pack_bf16(acc[i], x);
      if (i0 + i + odd < mine) *reinterpret_cast<uint32_t*>(out + (i0 + i) * kRank) = v;
    }
  }
}

// What the rows of zeros among a lane's 16 keys add to L: p 2^(kExpRef - kZeroExp) each.  (The loop over all keys takes E from u:
// 2^kExpRef of these p, 2^-60 of what is added here.  Beside that loop, not in it: few blocks have such rows.)
__device__ __noinline__ float sum_of_zeros(const float4* scp, float ref, float x0, float x1, float x2, float x3, float x4, float x5, float x6,
                                           float x7, float x8, float x9, float x10, float x11, float x12, float x13, float x14, float x15) {
  const float x[16] = {x0, x1, x2, x3, x4, x5, x6, x7, x8, x9, x10, x11, x12, x13, x14, x15};
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (__float_as_uint(reinterpret_cast<const float*>(scp + (j >> 1))[j & 1]) & 1u) s += ptx::ex2(x[j] + ref);
  static_assert(kExpRef - kZeroExp == 53, "the factor");
  return s * 0x1p53f;
}

// kProbe: with the test hook's waits.
template <bool FP4, bool ALL, bool kProbe>
__global__ void __launch_bounds__(kThreads, 1) quant_mla_kernel(const __grid_constant__ CUtensorMap tmap, const Args a) {
  using L = Smem<FP4>;
  constexpr int kStages = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((ptx::smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusSmemAlign);
    return;
  }
  uint8_t* misc = smem + L::kOffMisc;
  Bars* bars = reinterpret_cast<Bars*>(misc);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(misc + 512);
  volatile int* abort = reinterpret_cast<volatile int*>(misc + 516);
  volatile int* stopped = reinterpret_cast<volatile int*>(misc + 520);  // [2] blocks that either copying warp came to
  uint2* levels = reinterpret_cast<uint2*>(smem + L::kOffLevels);       // [256] the eight magnitudes that codes stand for
  float* linv = reinterpret_cast<float*>(misc + 768);                   // [64] of the piece that is written
  float* corr = reinterpret_cast<float*>(misc + 1024);                  // [2][64] factors of a block's heads
  float* top = reinterpret_cast<float*>(misc + 4096);                   // [2][2][64] a block's maxima over each group's keys
  uint32_t* movedv = reinterpret_cast<uint32_t*>(misc + 640);           // [2][4] a block's moved heads, by 16
  uint32_t* zeros = reinterpret_cast<uint32_t*>(misc + 672);            // [kScRing] whether a block has rows of zeros (4 bits: by 16 rows)
  float* lsum = reinterpret_cast<float*>(misc + 2048);                  // [2][64]
  Held* held = reinterpret_cast<Held*>(misc + 2560);                    // [64] of the piece that the cluster joins
  float* qscale = reinterpret_cast<float*>(held + kHeads);             // [kQRing][64]
  int* rows = reinterpret_cast<int*>(smem + L::kOffRows);               // [kRing][64] rows of a block's keys
  float4* sc = reinterpret_cast<float4*>(smem + L::kOffSc);             // [kScRing][32] two rows' 2^E, then their E - kExpRef
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&bars->tfull[s], FP4 ? 4 : 2);
      ptx::mbar_init(&bars->tempty[s], 1);
    }
    for (int s = 0; s < kBatches; ++s) {
      ptx::mbar_init(&bars->rfull[s], 1);
      ptx::mbar_init(&bars->bempty[s], FP4 ? 2 + 4 : 2 + 8);  // the copying warps; who reads validity or scales
      ptx::mbar_init(&bars->scfull[s], FP4 ? 4 : 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&bars->gfull[s], 2);
      ptx::mbar_init(&bars->gempty[s], 4);
      ptx::mbar_init(&bars->sfull[s], 1);
      ptx::mbar_init(&bars->sempty[s], 8);
      ptx::mbar_init(&bars->pfull[s], 8);
      ptx::mbar_init(&bars->pvdone[s], 1);
    }
    for (int s = 0; s < kQRing; ++s) ptx::mbar_init(&bars->qfull[s], 4);
    ptx::mbar_init(&bars->qfree, 1);
    ptx::mbar_init(&bars->odrained, 8);
    ptx::mbar_init(&bars->done, 1);
    if (kProbe) ptx::mbar_init(&bars->never, 1);
    *abort = 0;
    ptx::fence_mbar_init();
  }
  if (FP4 && threadIdx.x < 256) levels[threadIdx.x] = levels_at(levels_base(threadIdx.x & 7), threadIdx.x & 127);
  if (warp == 13) {
    ptx::tmem_alloc(tmem_holder, 512);
    ptx::tmem_relinquish();
  }
  if (warp == 12 && lane == 0) ptx::prefetch_tmap(&tmap);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();

  const int part = blockIdx.x;
  Pieces<ALL> pc(a, part);
  auto wait = [&](uint64_t* bar, uint32_t parity) { return ptx::mbar_try_wait(bar, parity) || wait_on(bar, parity, abort, a.status); };
  // Two at once: a try takes some 100 cycles even when it succeeds.
  auto wait2 = [&](uint64_t* bar0, uint32_t parity0, uint64_t* bar1, uint32_t parity1) {
    const bool r0 = ptx::mbar_try_wait(bar0, parity0), r1 = ptx::mbar_try_wait(bar1, parity1);
    return (r0 || wait_on(bar0, parity0, abort, a.status)) && (r1 || wait_on(bar1, parity1, abort, a.status));
  };
  const uint32_t sbase = ptx::smem_u32(smem);
  auto stop_at = [&](int site) { return kProbe && a.probe_site == site + (blockIdx.x & 1 ? kProbeOdd : 0) ? a.probe_at : ~0u; };
  auto run_out = [&]() { return ptx::mbar_spin(&bars->never, 0, abort, a.status, kStatusTimeout, a.probe_cycles); };

  if (warp == 13) {
    // ------------------------------------------------------------ MMAs
    // One elected lane runs the whole loop, its waits too: under any condition that the compiler cannot see to be
    // the same for the warp, an MMA takes some 90 cycles to issue.
    if (ptx::elect_one()) {
      const uint32_t id_qk = ptx::idesc_f32acc(128, kKeys, false), id_qr = ptx::idesc_f32acc(128, kKeys, true);
      const uint32_t tile0 = ptx::desc_lo(sbase + L::kOffTile, kAtom), rope0 = ptx::desc_lo(sbase + L::kOffQr, 16);
      const uint32_t p0 = ptx::desc_lo(sbase + L::kOffP, 16);
      const uint32_t stop = stop_at(kProbeMma);
      int it = 0, n = 0;  // blocks, pieces
      bool ok = true;
      while (ok && pc.next(a)) {
        const int cnt = pc.k1 - pc.k0, hg = min(kHeads, a.H - pc.g * kHeads);
        const uint32_t id_pv = ptx::idesc_f32acc(128, (hg + 15) & ~15, false) | (1u << 15);
        ok = wait(&bars->qfull[n % kQRing], (n / kQRing) & 1);
        for (int i = 0; i < cnt + L::kAhead && ok; ++i) {
          if (i < cnt) {  // S of block i
            const int b = it + i;
            if (kProbe && static_cast<uint32_t>(b) == stop && !run_out()) {
              ok = false;
              break;
            }
            // (one block ahead, P of the block that S's place was last for has been waited for already)
            ok = b < 2 || L::kAhead == 1 ? wait(&bars->tfull[b % kStages], (b / kStages) & 1)
                                         : wait2(&bars->tfull[b % kStages], (b / kStages) & 1, &bars->sempty[b & 1], ((b >> 1) & 1) ^ 1);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t d = tmem + kColS + (b & 1) * kKeys;
            uint32_t kd = tile0 + (b % kStages) * (kTile >> 4), qd = rope0;
            asm volatile("" : "+r"(kd), "+r"(qd));  // descriptors are added up here, not kept over the loop
#pragma unroll 1
            for (int at = 0; at < 4; ++at) {
#pragma unroll
              for (int s = 0; s < 4; ++s)  // 32 codes of K per MMA, four in a column
                mma_f8_ts(d, tmem + kColQ + (4 * at + s) * 8, kd + ((at * kAtom + s * 32) >> 4), id_qk, at + s);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) mma_bf16_ss(d, qd + 2 * s, kd + ((4 * kAtom) >> 4) + 2 * s, id_qr, 1u);
            ptx::mma_commit(&bars->sfull[b & 1]);
            if (i == cnt - 1) ptx::mma_commit(&bars->qfree);
          }
          const int j = i - L::kAhead;  // P . V of an earlier block
          if (j < 0) continue;
          const int b = it + j;
          ok = wait(&bars->pfull[b & 1], (b >> 1) & 1) && (j > 0 || n == 0 || wait(&bars->odrained, (n - 1) & 1));
          if (!ok) break;
          ptx::tc_fence_after();
          uint32_t vd = tile0 + (b % kStages) * (kTile >> 4), pd = p0 + (b % L::kPBufs) * (kPBytes >> 4);
          asm volatile("" : "+r"(vd), "+r"(pd));
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {  // 32 keys per MMA
              const uint32_t ad = vd + ((c * kAtom + s * 4096) >> 4);
              mma_f8_ss(tmem + kColO + c * kHeads, ad, pd + 2 * s, id_pv, (j > 0 || s > 0) ? 1u : 0u);
              mma_f8_ss(tmem + kColO + c * kHeads, ad, pd + 4 + 2 * s, id_pv | kBe5m2, 1u);
            }
          }
          ptx::mma_commit(&bars->tempty[b % kStages]);
          ptx::mma_commit(&bars->pvdone[b & 1]);
        }
        it += cnt;
        ++n;
      }
      ptx::mma_commit(&bars->done);
      ptx::mbar_spin_drain(&bars->done, 0, a.status, kStatusTimeout, 400000000ll);
    }
    __syncwarp();
  } else if (warp == 12 || warp == 15) {
    // ------------------------------------------------------------ rows of the cache, half of each block
    const int first = warp == 12 ? 0 : 8;  // groups of four rows
    constexpr int kBufs = FP4 ? 2 : kStages;
    const uint32_t stop = stop_at(warp == 12 ? kProbeCopy : kProbeCopy2);
    int it = 0, bn = 0;  // blocks, batches before this piece
    bool ok = true;
    for (; ok && pc.next(a); bn += batches(pc)) {
      for (int i = 0; i < pc.k1 - pc.k0; ++i, ++it) {
        const int bi = bn + i / kBatch, bt = bi % kBatches, st = it % kBufs;
        uint64_t* full = FP4 ? &bars->gfull[st] : &bars->tfull[st];
        ok = (i % kBatch || wait(&bars->rfull[bt], (bi / kBatches) & 1)) &&
             (it < kBufs || wait(FP4 ? &bars->gempty[st] : &bars->tempty[st], ((it / kBufs) & 1) ^ 1));
        if (kProbe && static_cast<uint32_t>(it) == stop) ok = ok && run_out();
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (ptx::elect_one()) {
          ptx::mbar_arrive_expect_tx(full, (FP4 ? kStaged : kTile) / 2);
          const int4* y4 = reinterpret_cast<const int4*>(rows + (bt * kBatch + i % kBatch) * kKeys) + first;
          int4 v = y4[0];
#pragma unroll 1
          for (int g = 0; g < 8; ++g) {
            const int y[4] = {v.x, v.y, v.z, v.w};
            if (g < 7) v = y4[g + 1];  // (ahead of the copies, which nothing is moved across)
            if (FP4) {
              tma_gather4(smem + L::kOffStaged + st * kStaged + (first + g) * 4 * kRow4, &tmap, full, 0, y);
            } else {
#pragma unroll
              for (int c = 0; c < 5; ++c)
                tma_gather4(smem + L::kOffTile + st * kTile + c * kAtom + (first + g) * 512, &tmap, full, c * 64, y);
            }
          }
          if (last_of_batch(pc, i)) ptx::mbar_arrive(&bars->bempty[bt]);
        }
        __syncwarp();
      }
    }
    // Copies in flight land before the CTA can exit, whatever happened.  A block's barrier counts both warps; where one gave up,
    // the other may have gone up to kBufs blocks further, and arrives in its place for those once both have stopped, so that
    // their drain ends when they have landed, not at its limit.  (A block that was issued kBufs after another shows that one done.)
    if (lane == 0) stopped[warp == 12 ? 0 : 1] = it;
    ptx::named_bar_sync(5, 64);
    const int other = stopped[warp == 12 ? 1 : 0];
    auto full = [&](int i) { return FP4 ? &bars->gfull[i % kBufs] : &bars->tfull[i % kBufs]; };
    if (lane == 0)
      for (int i = other; i < it; ++i) ptx::mbar_arrive(full(i));
    for (int i = max(0, max(it, other) - kBufs); i < it; ++i)
      ptx::mbar_spin_drain(full(i), (i / kBufs) & 1, a.status, kStatusTimeout, 400000000ll);
  } else if (warp == 14) {
    // ------------------------------------------------------------ where the rows lie; scales of e4m3 rows
    // A batch's loads pass behind each other: positions of the next batch and pages of this one together, then the
    // scales of this one behind the next one's.
    Keys keys;
    int k = 0, bi = 0;
    int pos[2 * kBatch];
    float u[2 * kBatch];
    const int32_t* table = nullptr;
    auto scales = [&](int bt) {
      unsigned z = 0u, some = 0u;
#pragma unroll
      for (int j = 0; j < 2 * kBatch; ++j) {
        put_scale(sc + (bt * kBatch + (j >> 1)) * (kKeys / 2), 32 * (j & 1) + lane, u[j]);
        z |= (u[j] == 1.f ? 1u : 0u) << j;
      }
      if (__builtin_expect(__any_sync(0xffffffffu, z != 0u), 0)) {
        z = rows_of_zeros(a.cache, rows + bt * kBatch * kKeys, z, lane);
        __syncwarp();
        some = __reduce_or_sync(0xffffffffu, z);
        for (; z; z &= z - 1) {
          const int j = __ffs(z) - 1;
          put_scale_of_zeros(sc + (bt * kBatch + (j >> 1)) * (kKeys / 2), 32 * (j & 1) + lane);
        }
      }
      if (lane < kBatch) zeros[bt * kBatch + lane] = some >> (2 * lane) & 3u;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars->scfull[bt]);
    };
    bool have = false, ok = true, bad = false;
    for (;;) {
      int y[2 * kBatch];
#pragma unroll
      for (int j = 0; j < 2 * kBatch; ++j) y[j] = pos[j];
      const int32_t* rows_of = table;
      bool more = true;  // the next batch's positions
      if (k >= pc.k1) {
        more = pc.next(a);
        k = pc.k0;
        if constexpr (ALL) {
          if (more && !have && part > 0 && lane == 0) {  // the join's part of the plan
            const Line line = line_of(a);
            const bool inside = k > 0 && line.begin(part - 1) <= pc.t_end - pc.blocks;
            a.joins[part] = inside ? make_int2(pc.w, line.part_at(pc.t_end - 1)) : make_int2(-1, 0);
          }
        }
      }
      if (more) {
        if (!ALL) {  // (read before it is known what the query sees: one trip to memory less)
          const int32_t* sel = a.topk + static_cast<long long>(pc.t) * a.topk_width;
#pragma unroll
          for (int j = 0; j < 2 * kBatch; ++j) {
            const int key = (k + (j >> 1)) * kKeys + 32 * (j & 1) + lane;
            pos[j] = k + (j >> 1) < pc.k1 && key < a.topk_width ? __ldg(sel + key) : -1;
          }
        }
        keys.move(a, ALL, pc.t, lane);
        table = a.block_tables + static_cast<long long>(keys.b) * a.max_pages;
#pragma unroll
        for (int j = 0; j < 2 * kBatch; ++j) {
          const int key = (k + (j >> 1)) * kKeys + 32 * (j & 1) + lane;
          if (ALL) pos[j] = k + (j >> 1) < pc.k1 && key < keys.n ? key : -1;
          else if (keys.n == 0 || pos[j] >= keys.len) pos[j] = -1;
        }
        k += kBatch;
      }
      if (have) {
#pragma unroll
        for (int j = 0; j < 2 * kBatch; ++j) y[j] = row_of(a, rows_of, y[j], &bad);
        const int bt = bi % kBatches;
        if (!FP4 && bi) scales((bt + kBatches - 1) % kBatches);
        ok = bi < kBatches || wait(&bars->bempty[bt], ((bi / kBatches) & 1) ^ 1);
        if (kProbe && static_cast<uint32_t>(bi) == stop_at(kProbeRows)) ok = ok && run_out();
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < 2 * kBatch; ++j) rows[(bt * kBatch + (j >> 1)) * kKeys + 32 * (j & 1) + lane] = y[j];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->rfull[bt]);
        if constexpr (!FP4) {
#pragma unroll
          for (int j = 0; j < 2 * kBatch; ++j)
            u[j] = y[j] != a.past_row ? __ldg(reinterpret_cast<const float*>(a.cache + static_cast<long long>(y[j]) * kRow8 + kScale8)) : 0.f;
        }
        ++bi;
      }
      have = more;
      if (!more) break;
    }
    if (!FP4 && ok && bi) scales((bi + kBatches - 1) % kBatches);
    if (bad) atomicOr(a.status, kStatusBadPage);
  } else if (warp >= 8) {
    // ------------------------------------------------------------ queries; tiles of 4-bit rows
    const int w = warp - 8;
    const uint32_t lane_addr = static_cast<uint32_t>(w * 32) << 16;
    uint8_t* qbuf = smem + L::kOffQ + w * 32 * kQStride;
    const int l8 = lane & 7, hr = lane >> 3;  // a lane takes 8 of 64 values of the heads 16 w + hr + 0, 4, 8, 12
    {
      // the lo rows take no part in the rotary product
      uint4* qr = reinterpret_cast<uint4*>(smem + L::kOffQr + (w * 32 + 16) * 128);
#pragma unroll
      for (int c = 0; c < 4; ++c) qr[c * 32 + lane] = make_uint4(0u, 0u, 0u, 0u);
    }
    int it = 0, n = 0, bn = 0;
    bool ok = true;
    for (; ok && pc.next(a); bn += batches(pc)) {
      if (kProbe && w == 0 && static_cast<uint32_t>(n) == stop_at(kProbeQueries)) ok = __all_sync(0xffffffffu, run_out());
      if (kProbe && !ok) break;
      const uint4* src[4];
      bool live[4];
      uint4 rp[4], r[4][4];
      __nv_bfloat162 am[4];
      const uint32_t keep = pc.t < live_rows(a) ? 0xffffffffu : 0u;  // rows of padding may hold anything: taken as zeros
      auto kept = [&](const uint4& v) { return make_uint4(v.x & keep, v.y & keep, v.z & keep, v.w & keep); };
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = pc.g * kHeads + w * 16 + 4 * i + hr;
        live[i] = h < a.H;
        src[i] = reinterpret_cast<const uint4*>(a.qn + pc.t * a.qn_t + (live[i] ? h : 0) * a.qn_h) + l8;
        rp[i] = live[i] ? __ldg(reinterpret_cast<const uint4*>(a.qr + pc.t * a.qr_t + h * a.qr_h) + l8) : make_uint4(0u, 0u, 0u, 0u);
        am[i] = most(rp[i]);
      }
      auto load = [&](int c, uint4 (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = live[i] ? __ldg(src[i] + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
      };
#pragma unroll 1
      for (int c = 4; c >= 0; c -= 4) {  // (the chunks that the conversion begins with come last, and stay)
#pragma unroll
        for (int q = 0; q < 4; ++q) load(c + q, r[q]);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) am[i] = __hmax2_nan(am[i], most(r[q][i]));
      }
      // the power of two that takes the row's largest value to [128, 256)
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t m = max(__float_as_uint(__low2float(am[i])), __float_as_uint(__high2float(am[i]))) & keep;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int e = m > 0u ? min(126, 7 - (static_cast<int>(m >> 23) - 127)) : 0;
        f[i] = pow2f(e);
        if (l8 == 0) qscale[(n % kQRing) * kHeads + w * 16 + 4 * i + hr] = m < 0x7F800000u ? a.scale_log2 * pow2f(-e) : NAN;  // (its codes would hide it)
      }
      if (n > 0) {
        ok = wait(&bars->qfree, (n - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      ptx::tc_fence_after();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = w * 32 + 4 * i + hr;
        float x[8];
        unpack_bf16(kept(rp[i]), x);
        *reinterpret_cast<uint4*>(smem + L::kOffQr + r * 128 + ((l8 ^ (r & 7)) << 4)) =
            make_uint4(pack_bf16(x[0] * f[i], x[1] * f[i]), pack_bf16(x[2] * f[i], x[3] * f[i]),
                       pack_bf16(x[4] * f[i], x[5] * f[i]), pack_bf16(x[6] * f[i], x[7] * f[i]));
      }
      // 64 values of every row at a time: codes to shared memory, from there by rows to TMEM
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x[8];
          unpack_bf16(kept(r[0][i]), x);
          const float g = f[i];
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint2 p = two_planes(__floats2half2_rn(x[4 * j] * g, x[4 * j + 1] * g), __floats2half2_rn(x[4 * j + 2] * g, x[4 * j + 3] * g));
            hi[j] = p.x;
            lo[j] = p.y;
          }
          *reinterpret_cast<uint2*>(qbuf + (4 * i + hr) * kQStride + l8 * 8) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(qbuf + (16 + 4 * i + hr) * kQStride + l8 * 8) = make_uint2(lo[0], lo[1]);
#pragma unroll
          for (int q = 0; q < 3; ++q) r[q][i] = r[q + 1][i];
        }
        if (c < 4) load(4 + c, r[3]);
        __syncwarp();
        uint32_t t[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 q = *reinterpret_cast<const uint4*>(qbuf + lane * kQStride + 16 * j);
          t[4 * j] = q.x, t[4 * j + 1] = q.y, t[4 * j + 2] = q.z, t[4 * j + 3] = q.w;
        }
        tmem_st_32x32b_x16(tmem + lane_addr + kColQ + 16 * c, t);
        __syncwarp();
      }
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars->qfull[n % kQRing]);
      ++n;
      if constexpr (FP4) {
        // 4-bit rows: a warp takes 16 rows of a block, a lane a block of 16 values
        for (int i = 0; i < pc.k1 - pc.k0; ++i, ++it) {
          const int st = it % kStages, gs = it & 1, bt = (bn + i / kBatch) % kBatches;
          ok = wait(&bars->gfull[gs], (it >> 1) & 1) && (it < kStages || wait(&bars->tempty[st], ((it / kStages) & 1) ^ 1));
          if (kProbe && w == 1 && static_cast<uint32_t>(it) == stop_at(kProbeDecode)) ok = ok && run_out();
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const bool there = rows[(bt * kBatch + i % kBatch) * kKeys + w * 16 + (lane & 15)] != a.past_row;  // of key 16 w + lane
          const uint8_t* staged = smem + L::kOffStaged + gs * kStaged + w * 16 * kRow4;
          uint8_t* tile = smem + L::kOffTile + st * kTile;
#pragma unroll 1
          for (int i0 = 0; i0 < 16; i0 += 8) {
            uint2 q[8], lv[8];
            int byte[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              byte[j] = staged[(i0 + j) * kRow4 + kScale4 + lane];
              q[j] = reinterpret_cast<const uint2*>(staged + (i0 + j) * kRow4)[lane];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) lv[j] = levels[byte[j]];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int key = w * 16 + i0 + j;
              const uint2 c0 = codes4_to_e4m3(q[j].x, lv[j]), c1 = codes4_to_e4m3(q[j].y, lv[j]);
              *reinterpret_cast<uint4*>(tile + (lane >> 3) * kAtom + key * 128 + ((l8 ^ (key & 7)) << 4)) =
                  make_uint4(c0.x, c0.y, c1.x, c1.y);
            }
          }
          uint4 rr[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) rr[j] = reinterpret_cast<const uint4*>(staged + (4 * j + hr) * kRow4 + kRope4)[l8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = w * 16 + 4 * j + hr;
            *reinterpret_cast<uint4*>(tile + 4 * kAtom + key * 128 + ((l8 ^ (key & 7)) << 4)) = rr[j];
          }
          bool none = false;
          if (lane < 16) {  // (the row's exponent from the top bits of its first eight scales; of zeros: E = 0, the smallest scales)
            const uint4 lo = *reinterpret_cast<const uint4*>(staged + lane * kRow4 + kScale4);
            const uint4 hi = *reinterpret_cast<const uint4*>(staged + lane * kRow4 + kScale4 + 16);
            none = there && ((lo.x | (lo.y ^ 0x80000000u)) | (lo.z | lo.w) | (hi.x | hi.y) | (hi.z | hi.w)) == 0u;
            put_scale(sc + st * (kKeys / 2), w * 16 + lane, there ? pow2f(top_bits(lo.x) + 16 * top_bits(lo.y) - 128) : 0.f);
            if (none) put_scale_of_zeros(sc + st * (kKeys / 2), w * 16 + lane);
          }
          none = __any_sync(0xffffffffu, none);
          if (lane == 0) reinterpret_cast<uint8_t*>(zeros + st)[w] = none;
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(&bars->gempty[gs]);
            ptx::mbar_arrive(&bars->scfull[st]);
            ptx::mbar_arrive(&bars->tfull[st]);
            if (last_of_batch(pc, i)) ptx::mbar_arrive(&bars->bempty[bt]);
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax, rescale, output
    // Group g takes the keys 32 g .. of every block, of which the hi lane has the first 16 and the lo lane the others.
    const int grp = warp >> 2, w = warp & 3, half = lane >> 4, hl = w * 16 + (lane & 15);
    const uint32_t lane_addr = static_cast<uint32_t>(w * 32) << 16;
    int it = 0, n = 0, bn = 0;
    bool ok = true;
    // Every piece and block runs its named barriers whatever happened, so that a wait that gave up leaves no
    // warp behind at one.
    while (pc.next(a)) {
      const int cnt = pc.k1 - pc.k0, hg = min(kHeads, a.H - pc.g * kHeads), end = it + cnt;
      float m = -INFINITY;  // the reference, the same in both groups
      float2 l = make_float2(0.f, 0.f), qm = l, qo = l;  // the sum, in two parts; the planes' scales
      if (ok) ok = __all_sync(0xffffffffu, wait(&bars->qfull[n % kQRing], (n / kQRing) & 1)) != 0;
      if (ok) {
        const float qs = qscale[(n % kQRing) * kHeads + hl];
        qm.x = qm.y = half ? qs * (1.f / (1 << kLoShift)) : qs;  // of this lane's plane, and of the other's
        qo.x = qo.y = half ? qs : qs * (1.f / (1 << kLoShift));
      }
      for (int b = it; b < end; ++b) {
        const int bi = bn + (b - it) / kBatch, bt = bi % kBatches, s2 = b & 1;
        const int ss = FP4 ? b % kStages : bt * kBatch + (b - it) % kBatch;
        const float4* scp = sc + ss * (kKeys / 2) + grp * 16 + half * 8;
        float x[16];
        float mb = -INFINITY;
        uint32_t none = 0u;  // rows of zeros in the block
        if (kProbe && ok && warp == 0 && static_cast<uint32_t>(b) == stop_at(kProbeSoftmax)) ok = __all_sync(0xffffffffu, run_out()) != 0;
        if (ok)
          ok = __all_sync(0xffffffffu, FP4 ? wait2(&bars->sfull[s2], (b >> 1) & 1, &bars->scfull[ss], (b / kStages) & 1)
                                       : (b - it) % kBatch ? wait(&bars->sfull[s2], (b >> 1) & 1)
                                       : wait2(&bars->sfull[s2], (b >> 1) & 1, &bars->scfull[bt], (bi / kBatches) & 1)) != 0;
        if (ok) {
          ptx::tc_fence_after();
          const uint32_t col = tmem + lane_addr + kColS + s2 * kKeys + grp * 32;
          uint32_t s0[16], s1[16];
          tmem_ld_x16(col, s0);
          tmem_ld_x16(col + 16, s1);
          tmem_ld_wait16(s0, s1);
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&bars->sempty[s2]);
          none = zeros[ss];
          float2 mx = make_float2(-INFINITY, -INFINITY);
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float2 keep, got;
            keep.x = __uint_as_float(half ? s1[j] : s0[j]);
            keep.y = __uint_as_float(half ? s1[j + 1] : s0[j + 1]);
            got.x = __uint_as_float(__shfl_xor_sync(0xffffffffu, half ? s0[j] : s1[j], 16));
            got.y = __uint_as_float(__shfl_xor_sync(0xffffffffu, half ? s0[j + 1] : s1[j + 1], 16));
            const float4 v = scp[j >> 1];
            float2 y = mul2(keep, qm);
            ptx::ffma2(y, got, qo);
            float2 z = make_float2(v.z, v.w);
            ptx::ffma2(z, y, make_float2(v.x, v.y));
            mx.x = fmaxf(mx.x, z.x);
            mx.y = fmaxf(mx.y, z.y);
            x[j] = z.x;
            x[j + 1] = z.y;
          }
          mb = fmaxf(mx.x, mx.y);
        }
        mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 16));
        if (!half) top[(s2 * 2 + grp) * kHeads + hl] = mb;
        // The reference moves only when it is passed by more than kMove, so that most blocks leave O as it is.
        const bool any = bar_any(2, m != -INFINITY && mb > m + kMove && hl < hg);
        mb = fmaxf(mb, top[(s2 * 2 + (grp ^ 1)) * kHeads + hl]);
        const float before = m;
        if (m == -INFINITY || mb > m + kMove) m = mb;
        const float cr = before == -INFINITY ? 1.f : ptx::ex2(before - m);
        float2 lb = make_float2(0.f, 0.f);  // the block's sum, by itself first: a long row's has 16 times fewer terms
        if (ok) {
          const float ref = m == -INFINITY ? 0.f : kPShift - m;
          const uint32_t change = threshold_change((pc.k0 + b - it) * 4 + grp * 2 + half);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float2 p[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint2 u = *reinterpret_cast<const uint2*>(scp + 2 * j + q);
              constexpr uint32_t kInv = static_cast<uint32_t>(254 + kExpRef) << 23;
              p[q] = add2(make_float2(x[4 * j + 2 * q], x[4 * j + 2 * q + 1]), ref);
              p[q] = make_float2(ptx::ex2(p[q].x), ptx::ex2(p[q].y));
              ptx::ffma2(lb, p[q], make_float2(__uint_as_float(kInv - u.x), __uint_as_float(kInv - u.y)));  // p 2^(kExpRef - E)
            }
            const uint2 t = two_terms(__floats2half2_rn(p[0].x, p[0].y), __floats2half2_rn(p[1].x, p[1].y), 4 * j, change);
            hi[j] = t.x;
            lo[j] = t.y;
          }
          ptx::ffma2(lb, l, make_float2(cr, cr));
          l = lb;
          const int ch = grp * 2 + half;
          // (its buffer is free: this block's S was issued behind the products that read it, and has been done)
          uint8_t* prow = smem + L::kOffP + (b % L::kPBufs) * kPBytes + hl * 128;
          *reinterpret_cast<uint4*>(prow + ((ch ^ (hl & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(prow + (((4 + ch) ^ (hl & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          if (__builtin_expect(none != 0u, 0))
            l.x += sum_of_zeros(scp, ref, x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], x[8], x[9], x[10], x[11], x[12], x[13], x[14],
                                x[15]);
          ptx::fence_proxy_async_smem();
        }
        // Heads whose reference moved: their columns of O are rescaled when the products of the block before are
        // done and before those of this one begin (which wait for them in any case), each group's two latent chunks.
        // (corr and movedv are read before the barrier of the next block, and rewritten behind it.)
        if (any) {
          const unsigned moved = __ballot_sync(0xffffffffu, !half && hl < hg && cr != 1.f);
          if (grp == 0) {
            if (!half) corr[s2 * kHeads + hl] = cr;
            if (lane == 0) movedv[s2 * 4 + w] = moved;
          }
          ptx::named_bar_sync(3, 256);
          if (ok) ok = __all_sync(0xffffffffu, wait(&bars->pvdone[s2 ^ 1], ((b - 1) >> 1) & 1)) != 0;
          if (ok) {
            ptx::tc_fence_after();
            const uint2 m01 = *reinterpret_cast<const uint2*>(movedv + s2 * 4), m23 = *reinterpret_cast<const uint2*>(movedv + s2 * 4 + 2);
            uint64_t todo = (m01.x | m01.y << 16) | static_cast<uint64_t>(m23.x | m23.y << 16) << 32;
            const uint32_t o = tmem + lane_addr + kColO + grp * 2 * kHeads;
            const float* f = corr + s2 * kHeads;
            if (__popcll(todo) <= kFewHeads) {
              for (; todo; todo &= todo - 1) {
                const int h = __ffsll(static_cast<long long>(todo)) - 1;
                float r0 = tmem_ld_x1(o + h), r1 = tmem_ld_x1(o + kHeads + h);
                asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(r0), "+f"(r1) : : "memory");
                tmem_st_x1(o + h, r0 * f[h]);
                tmem_st_x1(o + kHeads + h, r1 * f[h]);
              }
            } else {
#pragma unroll 1
              for (int q = 0; q < 8; ++q) {
                uint32_t r[16];
                tmem_ld_x16(o + q * 16, r);
                tmem_ld_wait16(r);
#pragma unroll
                for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * f[(q & 3) * 16 + j]);
                tmem_st_32x32b_x16(o + q * 16, r);
              }
            }
            ptx::tmem_st_wait();
          }
        }
        if (ok) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(&bars->pfull[s2]);
            if (!FP4 && last_of_batch(pc, b - it)) ptx::mbar_arrive(&bars->bempty[bt]);
          }
        }
      }
      it = end;
      ++n;
      bn += batches(pc);
      // the piece's output: the sums of both groups
      const int last = (end - 1) & 1;
      if (ok) ok = __all_sync(0xffffffffu, wait(&bars->pvdone[last], ((end - 1) >> 1) & 1)) != 0;
      const float fin = m;
      float sum = l.x + l.y;
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      if (!half) lsum[grp * kHeads + hl] = sum;
      ptx::named_bar_sync(4, 256);
      const bool whole = pc.k0 == 0 && pc.k1 == pc.blocks;
      const int slot = 2 * part + (pc.k0 == 0 ? 1 : 0);
      if (grp == 0 && !half) {
        sum = lsum[hl] + lsum[kHeads + hl];
        linv[hl] = sum == 0.f ? 0.f : pow2f(kExpRef) / sum;
        if (hl < hg && ok) {
          if (!ALL && !whole && a.cluster > 1) {
            held[hl] = {fin + 0.f * sum, sum};
          } else if (!whole) {
            a.part_ml[(static_cast<long long>(slot) * kHeads + hl) * 2] = fin + 0.f * sum;  // (not a number if the sum is not)
            a.part_ml[(static_cast<long long>(slot) * kHeads + hl) * 2 + 1] = sum;
          } else if (a.lse) {
            a.lse[static_cast<long long>(pc.t) * a.H + pc.g * kHeads + hl] = sum == 0.f ? -INFINITY : (fin - kPShift + log2f(sum)) * kLn2;
          }
        }
      }
      ptx::named_bar_sync(4, 256);
      if (ok && (ALL || whole || a.cluster == 1)) {
        ptx::tc_fence_after();
        const int lat = w * 32 + lane;
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {  // this group's two latent chunks, 16 heads at a time
          const int c = 2 * grp + (q >> 2), h0 = (q & 3) * 16;
          if (h0 >= hg) continue;
          uint32_t r[16];
          tmem_ld_x16(tmem + lane_addr + kColO + c * kHeads + h0, r);
          tmem_ld_wait16(r);
          if (whole) {
            // neighbouring lanes exchange heads, so that a store takes two latent values: the even lane head j, the odd one j + 1
            const bool odd = lane & 1;
            __nv_bfloat16* o = a.out + (static_cast<long long>(pc.t) * a.H + pc.g * kHeads + h0 + odd) * kRank + c * 128 + w * 32 + (lane & 30);
            const int heads = hg - h0 - odd;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float2 f = *reinterpret_cast<const float2*>(linv + h0 + j);
              const float x = __uint_as_float(r[j]) * f.x, y = __uint_as_float(r[j + 1]) * f.y;
              const float got = __shfl_xor_sync(0xffffffffu, odd ? x : y, 1);
              const uint32_t v = odd ? pack_bf16(got, y) : pack_bf16(x, got);
              if (j < heads) *reinterpret_cast<uint32_t*>(o + j * kRank) = v;
            }
          } else {
            float4* o = reinterpret_cast<float4*>(a.part_o) + ((static_cast<long long>(slot) * 4 + c) * 16 + h0 / 4) * 128 + lat;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (h0 + 4 * j < hg)
                o[j * 128] = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]), __uint_as_float(r[4 * j + 2]),
                                         __uint_as_float(r[4 * j + 3]));
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->odrained);
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (!ALL) {
    if (a.cluster > 1 && static_cast<int>(blockIdx.x) < a.rest * a.cluster) {  // (the same in all CTAs of a cluster)
      ptx::tc_fence_after();
      join_in_cluster(a, smem + L::kOffTile, smem + L::kOffP, reinterpret_cast<uint32_t*>(smem + L::kOffQ), held, tmem);
      ptx::tc_fence_before();
      __syncthreads();
    }
  }
  if (warp == 13) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// The same of pieces that went through memory.  The tiles are listed by
// the parts that begin inside them.  Of a tile of few pieces a warp takes four heads of a latent chunk, a lane four
// latent values of each; of many, a CTA, its warps four chunks of every fourth piece.
constexpr int kJoinThreads = 512, kFewPieces = 16, kMaxParts = 512;
__device__ __forceinline__ void add_piece(float4& acc, float4 f, float4 v) {  // (a piece without keys may hold anything)
  acc.x = fmaf(f.x, f.x == 0.f ? 0.f : v.x, acc.x);
  acc.y = fmaf(f.y, f.y == 0.f ? 0.f : v.y, acc.y);
  acc.z = fmaf(f.z, f.z == 0.f ? 0.f : v.z, acc.z);
  acc.w = fmaf(f.w, f.w == 0.f ? 0.f : v.w, acc.w);
}
__device__ __forceinline__ float4 warp_sum4(float4 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
    v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
  }
  return v;
}
__device__ __forceinline__ float4 warp_max4(float4 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x = fmaxf(v.x, __shfl_xor_sync(0xffffffffu, v.x, o));
    v.y = fmaxf(v.y, __shfl_xor_sync(0xffffffffu, v.y, o));
    v.z = fmaxf(v.z, __shfl_xor_sync(0xffffffffu, v.z, o));
    v.w = fmaxf(v.w, __shfl_xor_sync(0xffffffffu, v.w, o));
  }
  return v;
}
template <bool ALL>
__global__ void __launch_bounds__(kJoinThreads) quant_join_kernel(const Args a) {
  __shared__ int2 joins[kMaxParts];
  __shared__ int4 few[kMaxParts], many[kMaxParts];  // tile, first part, pieces
  __shared__ float4 weights[kMaxParts], sums[4][128];
  __shared__ int n_few, n_many;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  if constexpr (ALL) {
    const int parts = line_of(a).parts;
    if (tid < parts) joins[tid] = tid ? a.joins[tid] : make_int2(-1, 0);
    __syncthreads();
    if (warp == 0) {
      int nf = 0, nm = 0;
      for (int c0 = 0; c0 < parts; c0 += 32) {
        const int c = c0 + lane;
        const int2 r = c < parts ? joins[c] : make_int2(-1, 0);
        const int n = r.y - c + 2;
        const unsigned f = __ballot_sync(0xffffffffu, r.x >= 0 && n <= kFewPieces), m = __ballot_sync(0xffffffffu, r.x >= 0 && n > kFewPieces);
        const unsigned below = (1u << lane) - 1;
        if (f >> lane & 1) few[nf + __popc(f & below)] = make_int4(r.x, c - 1, n, 0);
        if (m >> lane & 1) many[nm + __popc(m & below)] = make_int4(r.x, c - 1, n, 0);
        nf += __popc(f);
        nm += __popc(m);
      }
      if (lane == 0) n_few = nf, n_many = nm;
    }
    __syncthreads();
  }
  const int tiles_few = ALL ? n_few : a.split <= kFewPieces ? a.rest : 0, tiles_many = ALL ? n_many : a.rest - tiles_few;
  auto tile_of = [&](const int4* list, int i) { return ALL ? list[i] : make_int4(a.parts * a.whole + i, i * a.split, a.split, 0); };
  auto slot = [](int c0, int j) { return static_cast<long long>(2 * (c0 + j) + (j == 0 ? 1 : 0)); };
  auto stats = [&](int c0, int j, int quad, float4* m, float4* l) {
    const float4* ml = reinterpret_cast<const float4*>(a.part_ml + (slot(c0, j) * kHeads + quad * 4) * 2);
    const float4 x = ml[0], y = ml[1];
    *m = make_float4(x.x, x.z, y.x, y.z);
    *l = make_float4(x.y, x.w, y.y, y.w);
  };
  // weight of a piece against the tile's maximum, and its part of the sum
  auto weigh = [](float4 m, float4 M, float4 l, float4* f) {
    *f = make_float4(m.x == -INFINITY ? 0.f : exp2f(m.x - M.x), m.y == -INFINITY ? 0.f : exp2f(m.y - M.y),
                     m.z == -INFINITY ? 0.f : exp2f(m.z - M.z), m.w == -INFINITY ? 0.f : exp2f(m.w - M.w));
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    add_piece(s, *f, l);
    return s;
  };
  auto store = [&](int t, int h0, int lat, float4 acc, float4 total) {
    const float v[4] = {acc.x, acc.y, acc.z, acc.w}, s[4] = {total.x, total.y, total.z, total.w};
    __nv_bfloat16* dst = a.out + (static_cast<long long>(t) * a.H + h0) * kRank + lat;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (h0 + i < a.H) dst[i * kRank] = __float2bfloat16_rn(s[i] == 0.f ? 0.f : v[i] / s[i] * pow2f(kExpRef));
  };
  auto store_lse = [&](int t, int h0, float4 M, float4 total) {
    const float m[4] = {M.x, M.y, M.z, M.w}, s[4] = {total.x, total.y, total.z, total.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (a.lse && h0 + i < a.H)
        a.lse[static_cast<long long>(t) * a.H + h0 + i] = s[i] == 0.f ? -INFINITY : (m[i] - kPShift + log2f(s[i])) * kLn2;
  };
  const float4 none = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY), zero = make_float4(0.f, 0.f, 0.f, 0.f);

  for (int item = blockIdx.x * (kJoinThreads / 32) + warp; item < tiles_few * 64; item += gridDim.x * (kJoinThreads / 32)) {
    const int4 tile = tile_of(few, item >> 6);
    const int quad = item & 15, chunk = (item >> 4) & 3, n = tile.z;
    const int t = tile.x / a.groups, h0 = (tile.x - t * a.groups) * kHeads + quad * 4;
    if (h0 >= a.H) continue;
    float4 m = none, l = zero, f;  // lane j: piece j
    if (lane < n) stats(tile.y, lane, quad, &m, &l);
    const float4* o = reinterpret_cast<const float4*>(a.part_o) + (static_cast<long long>(chunk) * 16 + quad) * 128 + lane;
    const float4 M = warp_max4(m);
    const float4 total = warp_sum4(weigh(m, M, l, &f));
    float4 acc[4] = {zero, zero, zero, zero};
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const float4 fj = make_float4(__shfl_sync(0xffffffffu, f.x, j), __shfl_sync(0xffffffffu, f.y, j),
                                    __shfl_sync(0xffffffffu, f.z, j), __shfl_sync(0xffffffffu, f.w, j));
#pragma unroll
      for (int i = 0; i < 4; ++i) add_piece(acc[i], fj, o[slot(tile.y, j) * (4 * 16 * 128) + 32 * i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) store(t, h0, chunk * 128 + 32 * i + lane, acc[i], total);
    if (chunk == 0 && lane == 0) store_lse(t, h0, M, total);
  }

  for (int item = blockIdx.x; item < tiles_many * 64; item += gridDim.x) {
    const int4 tile = tile_of(many, item >> 6);
    const int quad = item & 15, chunk = (item >> 4) & 3, n = tile.z, grp = tid >> 7, lat = tid & 127;
    const int t = tile.x / a.groups, h0 = (tile.x - t * a.groups) * kHeads + quad * 4;
    if (h0 >= a.H) continue;  // the same in the whole CTA
    __syncthreads();
    if (warp == 0) {
      float4 M = none, total = zero, m, l, f;
      for (int j = lane; j < n; j += 32) {
        stats(tile.y, j, quad, &m, &l);
        M = make_float4(fmaxf(M.x, m.x), fmaxf(M.y, m.y), fmaxf(M.z, m.z), fmaxf(M.w, m.w));
      }
      M = warp_max4(M);
      for (int j = lane; j < n; j += 32) {
        stats(tile.y, j, quad, &m, &l);
        const float4 s = weigh(m, M, l, &f);
        total = make_float4(total.x + s.x, total.y + s.y, total.z + s.z, total.w + s.w);
        weights[j] = f;
      }
      total = warp_sum4(total);
      if (lane == 0) {
        sums[3][0] = total;
        if (chunk == 0) store_lse(t, h0, M, total);
      }
    }
    __syncthreads();
    const float4 total = sums[3][0];
    const float4* o = reinterpret_cast<const float4*>(a.part_o) + (static_cast<long long>(chunk) * 16 + quad) * 128 + lat;
    float4 acc = zero;
#pragma unroll 4
    for (int j = grp; j < n; j += 4) add_piece(acc, weights[j], o[slot(tile.y, j) * (4 * 16 * 128)]);
    if (grp) sums[grp - 1][lat] = acc;
    __syncthreads();
    if (!grp) {
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const float4 x = sums[q][lat];
        acc = make_float4(acc.x + x.x, acc.y + x.y, acc.z + x.z, acc.w + x.w);
      }
      store(t, h0, chunk * 128 + lat, acc, total);
    }
  }
}

// Blocks before each query (every position): at least one a query, so that each has a tile that writes it.
constexpr int kPlanRequests = 4096;
__global__ void __launch_bounds__(1024) quant_plan_kernel(const Args a, long long* cum) {
  __shared__ long long sums[32];
  __shared__ int32_t first[kPlanRequests + 1];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool held = a.B <= kPlanRequests;  // else from memory
  if (held)
    for (int b = threadIdx.x; b <= a.B; b += 1024) first[b] = __ldg(a.cu + b);
  __syncthreads();
  auto cu = [&](int b) { return held ? first[b] : __ldg(a.cu + b); };
  const int rows = min(cu(a.B), a.most_live);
  long long before = 0;
  for (int t0 = 0; t0 < a.total_q; t0 += 1024) {
    const int t = t0 + threadIdx.x;
    long long v = t < a.total_q ? 1 : 0;
    if (t < a.total_q && t < rows) {
      int lo = 0, hi = a.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu(mid) <= t) lo = mid; else hi = mid;
      }
      v = max(1ll, (keys_seen(a, static_cast<long long>(__ldg(a.lens + lo)) - cu(lo + 1) + t, false) + kKeys - 1) / kKeys);
    }
    long long s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += x;
    }
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    long long w = sums[lane];  // every warp scans the warps' sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += x;
    }
    const long long add = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
    if (t < a.total_q) cum[t] = before + add + s - v;
    before += __shfl_sync(0xffffffffu, w, 31);
    __syncthreads();
  }
  if (threadIdx.x == 0) cum[a.total_q] = before;
}

dsa_status validate(const dsa_quant_mla_args* a) {
  if (!a) return DSA_ERR_INVALID_ARGUMENT;
  if (a->B < 0 || a->total_q < 0 || a->H <= 0 || a->topk_width < 0 || a->page_size <= 0 || a->num_pages < 0 ||
      a->max_pages_per_seq < 0 || !(a->scale > 0.f) || !(a->scale < INFINITY))
    return DSA_ERR_INVALID_ARGUMENT;
  if (a->kv_rank != quant::kRank || a->rope_dim != quant::kRope || quant::row_bytes(a->format) == 0 || a->H > 128)
    return DSA_ERR_UNSUPPORTED;
  if (a->topk_width > kMostKeys) return DSA_ERR_UNSUPPORTED;
  if (static_cast<long long>(a->total_q) * a->H >= 0x7FFFFF80LL || static_cast<long long>(a->num_pages) * a->page_size >= 0x7FFFFF80LL)
    return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

// SMs of the current device, asked for once (148 where there is no device to ask: a workspace size).
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

struct Plan {
  int groups, nb, parts, whole, rest, split, cluster;
  size_t off_ml, off_joins, off_cum, total;
};
Plan plan_of(const dsa_quant_mla_args* a) {
  Plan p{};
  p.cluster = 1;
  p.groups = (a->H + kHeads - 1) / kHeads;
  p.nb = (a->topk_width + kKeys - 1) / kKeys;
  p.parts = std::min(sm_count(), kMaxParts);
  if (p.nb) {
    const int tiles = static_cast<int>(static_cast<long long>(a->total_q) * p.groups);
    p.whole = tiles / p.parts;
    p.rest = tiles - p.whole * p.parts;
    // pieces of two blocks at least: of one, 4 tiles of 32 blocks take as long, and the join longer
    p.split = p.rest ? std::max(1, std::min(p.parts / p.rest, p.nb / 2)) : 1;
    // Pieces of a tile in a cluster (as many as it has CTAs) where that is faster than more pieces, joined through memory, and
    // all clusters find room at once: 15 of 8, 32 of 4, 76 of 2 (16 of 8: 46.0 us instead of 23.6; with whole tiles every SM is
    // taken).  The cluster's join saves a launch, some 3 us; it adds blocks to a CTA, 1.0 to 1.4 us each; and with many heads it
    // takes longer than a join through memory of few pieces.  us in a cluster, through memory; 2048 keys in 8 bits (4 bits alike):
    //   4 tiles of 16 heads    8 or 16 pieces  17.0, 18.0      of 64 heads           23.4, 21.6
    //   24 tiles of 16 heads   4 or 6          21.1, 21.1      17 tiles, 4 or 8      20.5, 19.6 (four blocks more)
    //   32 tiles of 32 heads   4               23.7, 23.4      of 48 heads           26.3, 24.6
    //   64 tiles of 8 heads    2               28.4, 32.3      of 64 heads           35.8, 37.6
    //   48 tiles of 64 heads   2 or 3          35.5, 32.8 (five blocks more)
    //   64 tiles behind 152    2               76.4, 81.1      40 tiles, 2 or 3      75.5, 74.4
    //   33 tiles of 64 heads, 256 keys, 2  19.5, 17.9      1 tile of 64, 65536 keys, 8 or 152  164, 28.8
    const int most = !p.whole && p.split >= 8 && p.rest <= 15 ? 8 : !p.whole && p.split >= 4 && p.rest <= 32 ? 4 : 2;
    const int added = (p.nb + most - 1) / most - (p.nb + p.split - 1) / p.split;
    if (p.split >= 2 && added <= 2 && (a->H <= 32 || (most == 2 && 3 * p.rest > p.parts)) && p.rest * most <= p.parts && p.parts % (p.whole ? most : 1) == 0)
      p.cluster = most;
    if (p.cluster > 1) p.split = p.cluster;
    if (!p.whole) p.parts = p.rest * p.split;
    if (p.split == 1 || p.cluster > 1) return p;  // no workspace
  }
  p.off_ml = static_cast<size_t>(2) * p.parts * kHeads * kRank * 4;
  p.off_joins = p.off_ml + static_cast<size_t>(2) * p.parts * kHeads * 2 * 4;
  p.off_cum = p.off_joins + static_cast<size_t>(p.parts) * 8;
  p.total = p.off_cum + (p.nb ? 0 : (static_cast<size_t>(a->total_q) + 1) * 8);
  return p;
}

template <bool FP4, bool ALL, bool kProbe>
cudaError_t launch_kernel(const CUtensorMap& map, const Args& k, cudaStream_t s) {
  static std::atomic<unsigned long long> set{0};  // devices whose kernel has its shared memory size
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto* kern = quant_mla_kernel<FP4, ALL, kProbe>;
  if (dev >= 64 || !(set.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<FP4>::kBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) set.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  return launch_pdl_cluster(kern, dim3(k.parts), dim3(kThreads), Smem<FP4>::kBytes, ALL ? 1 : k.cluster, s, map, k);
}
template <bool FP4, bool ALL>
cudaError_t launch_attend(const CUtensorMap& map, const Args& k, cudaStream_t s) {
  return k.probe_site != 0 ? launch_kernel<FP4, ALL, true>(map, k, s) : launch_kernel<FP4, ALL, false>(map, k, s);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_quant_mla_workspace_size(const dsa_quant_mla_args* a, size_t* bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARGUMENT;
  const dsa_status st = validate(a);
  if (st != DSA_OK) return st;
  *bytes = plan_of(a).total;
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
  const Plan p = plan_of(a);
  if (p.total && (!a->workspace || a->workspace_bytes < p.total || !al(a->workspace, 16))) return DSA_ERR_WORKSPACE;
  unsigned* status = device_status_ptr();
  if (!status) return DSA_ERR_CUDA;
  Args k{};
  k.B = a->B;
  k.total_q = a->total_q;
  k.H = a->H;
  k.groups = p.groups;
  k.page_size = a->page_size;
  // d <= 2^s: m = ceil(2^(32 + s) / d) exceeds 2^(32 + s) / d by less than 2^s / d, too little to matter below 2^32
  int s2 = 0;
  while (1ll << s2 < a->page_size) ++s2;
  k.page_mul = ((1ull << (32 + s2)) + a->page_size - 1) / a->page_size;
  k.page_shift = 32 + s2;
  k.num_pages = a->num_pages;
  k.max_pages = a->max_pages_per_seq;
  k.topk_width = a->topk_width;
  k.nb = p.nb;
  k.most_live = a->B > 0 ? a->total_q : 0;
  k.parts = p.parts;
  k.whole = p.whole;
  k.rest = p.rest;
  k.split = p.split;
  k.cluster = p.cluster;
  k.past_row = std::max(1, a->num_pages * a->page_size);
  k.scale_log2 = a->scale * 1.4426950408889634f;
  k.qn = static_cast<const __nv_bfloat16*>(a->q_nope);
  k.qr = static_cast<const __nv_bfloat16*>(a->q_rope);
  k.qn_t = a->qn_stride_t;
  k.qn_h = a->qn_stride_h;
  k.qr_t = a->qr_stride_t;
  k.qr_h = a->qr_stride_h;
  k.cache = static_cast<const uint8_t*>(a->cache);
  k.block_tables = a->block_tables;
  k.cu = a->cu_q_lens;
  k.lens = a->seq_lens;
  k.topk = a->topk;
  k.out = static_cast<__nv_bfloat16*>(a->out);
  k.lse = a->lse;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  k.part_o = reinterpret_cast<float*>(ws);
  k.part_ml = reinterpret_cast<float*>(ws + p.off_ml);
  k.joins = reinterpret_cast<int2*>(ws + p.off_joins);
  k.status = status;
  const Probe probe = armed_probe();
  armed_probe() = Probe{0, 0, 0};
  k.probe_site = probe.site;
  k.probe_at = probe.at;
  k.probe_cycles = 2 * static_cast<long long>(probe.limit_ns);  // some 2 cycles a nanosecond
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (!p.nb) {
    long long* cum = reinterpret_cast<long long*>(ws + p.off_cum);
    e = launch_pdl(quant_plan_kernel, dim3(1), dim3(1024), 0, s, k, cum);
    if (e != cudaSuccess) return DSA_ERR_CUDA;
    k.cum = cum;
  }
  // (a cache without pages: a map of one row, past which every copy lies)
  CUtensorMap map;
  const bool fp4 = a->format == DSA_FP4_E2M1;
  if (!make_gather_map(&map, a->cache ? a->cache : a->q_nope, fp4, quant::row_bytes(a->format), k.past_row)) return DSA_ERR_CUDA;
  const bool all = p.nb == 0;
  e = fp4 ? (all ? launch_attend<true, true>(map, k, s) : launch_attend<true, false>(map, k, s))
          : (all ? launch_attend<false, true>(map, k, s) : launch_attend<false, false>(map, k, s));
  if (e != cudaSuccess) return DSA_ERR_CUDA;
  // two CTAs of the join fill an SM; of selected keys it is known how many it takes, and whether any
  const int per = p.split <= kFewPieces ? kJoinThreads / 32 : 1;
  const int blocks = all ? 2 * sm_count() : p.split > 1 && p.cluster == 1 ? std::min(2 * sm_count(), (p.rest * 64 + per - 1) / per) : 0;
  if (blocks) e = launch_pdl(all ? quant_join_kernel<true> : quant_join_kernel<false>, dim3(blocks), dim3(kJoinThreads), 0, s, k);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

dsa_status dsa_test_arm_quant_mla_timeout(int site, unsigned at, unsigned long long limit_ns) {
  const int role = site & ~kProbeOdd;
  if (role < kProbeMma || role > kProbeSoftmax || site < 0 || limit_ns > 1000000000ull) return DSA_ERR_INVALID_ARGUMENT;
  armed_probe() = limit_ns == 0 ? Probe{0, 0, 0} : Probe{site, at, limit_ns};
  return DSA_OK;
}

}  // extern "C"
