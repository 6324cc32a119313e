// quant_mla.cu -- multi-head latent attention over the quantised latent cache.
//
//     logit[t, h, s] = scale * (q_nope[t, h] . c[s] + q_rope[t, h] . r[s])
//     out[t, h]      = sum_s softmax_s(logit[t, h, :]) c[s],   lse[t, h] = ln sum_s exp(logit[t, h, s])
//
// over the selected positions s = topk[t, j] of the query's sequence, or over every position up to its own.
//
// Both formats are e4m3 numbers times a row's power of two, c[s] = 2^E c8[s], r[s] = 2^E r8[s], so the tensor
// cores take the cache's codes as they are, and nothing is converted to bf16:
//   q = 2^-a (hi + lo) in two e4m3 rows (exact for what lies within 2^9 of the row's largest value, and within
//   2^-17 of that otherwise):      S = hi . c8 + lo . c8 + (2^a q_rope) . r8,   logit log2(e) = 2^-a 2^E S scale log2(e)
//   x' = logit log2(e) + E,  m' its running maximum,  p = 2^(x' - m' + 5) in two e4m3 terms (2^-8 relative,
//   2^-15 of the largest):         O = sum p c8,  L = sum p 2^-E (fp32),  out = O / L
// Two e4m3 planes cost the tensor cores what one bf16 plane does and half the shared memory traffic.  Taking E
// into the maximum keeps p in e4m3's range whatever the rows' scales are.
//
// Work: a tile is a query and up to 64 heads, its keys are cut into blocks of 64.  The blocks of all tiles stand
// in one line, cut into equal parts, one per CTA: a part may start and end inside a tile.  A tile done in one
// piece is normalised and written, the pieces of the others leave (O, m', L) in fp32 and a second kernel joins them.
// Roles of a CTA:
//   warps 0..7    softmax, two groups that take alternate blocks and hand the reference on.  Rows of S alternate
//                 between 16 hi and 16 lo rows, so that a lane and the one 16 further hold a head's two planes;
//                 each adds the planes for half of the block's keys;
//   warps 8..11   query rows: bf16 -> hi, lo in TMEM (A operand), 2^a q_rope in shared memory;
//                 4-bit rows also: codes from the staged rows to e4m3 tiles;
//   warps 12, 15  rows of the cache by gathering TMA: e4m3 tiles in 128-byte columns, 4-bit rows whole;
//   warp 13       TMEM, MMAs:  S [128 x 64 keys] = Q (TMEM) . K^T,  O^T [512 x heads] += V^T (the same tile,
//                 MN-major) . P^T;
//   warp 14       where the rows lie, four blocks at a time; e4m3: their scales.
// Every wait is bounded; after one gives up, every role stops, the MMAs and copies in flight are drained
// (bounded) and TMEM is freed.
#include <cuda_runtime.h>

#include <algorithm>

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
constexpr long long kMostKeys = 0x7FFFFF00ll;             // that a query sees: a block's last key fits 32 bits
constexpr int kMaxStages = 4;
constexpr int kQRing = 4;                                 // scales of the queries of consecutive pieces
constexpr int kBatch = 4, kBatches = 4, kRing = kBatch * kBatches;  // blocks whose rows are looked up together

template <bool FP4>
struct Smem {
  static constexpr int kStages = FP4 ? 3 : 4;             // tiles
  static constexpr int kStagedBufs = FP4 ? 2 : 0;
  static constexpr int kScRing = FP4 ? kStages : kRing;   // blocks whose scales are held
  static constexpr uint32_t kOffTile = 0, kOffQr = kOffTile + kStages * kTile, kOffP = kOffQr + kQRope;
  static constexpr uint32_t kOffStaged = kOffP + 2 * kPBytes, kOffQ = kOffStaged + kStagedBufs * kStaged;
  static constexpr uint32_t kOffMisc = kOffQ + kQBuf, kOffRows = kOffMisc + 4096, kOffSc = kOffRows + kRing * kKeys * 4;
  static constexpr uint32_t kBytes = kOffSc + kScRing * kKeys * 8;
};
static_assert(Smem<false>::kBytes <= 232448 && Smem<true>::kBytes <= 232448, "shared memory of a CTA");

struct Args {
  int B, total_q, H, groups, page_size, page_log2, num_pages, max_pages, topk_width;
  int nb;                  // blocks of a tile (selected keys); 0: from the plan
  int parts;               // CTAs
  int past_row;            // a row past the cache: copies from there are zeros
  float scale_log2;        // scale * log2(e)
  const __nv_bfloat16 *qn, *qr;
  long long qn_t, qn_h, qr_t, qr_h;
  const uint8_t* cache;
  const int32_t *block_tables, *cu, *lens, *topk;
  const long long* cum;    // [total_q + 1] blocks before each query (every position)
  __nv_bfloat16* out;
  float* lse;
  float *part_o, *part_ml; // pieces: [slot][4][16][128][4] (latent chunk, four heads, latent, head), [slot][64][2]
  unsigned* status;
};

struct Bars {
  uint64_t tfull[kMaxStages], tempty[kMaxStages];
  uint64_t rfull[kBatches], bempty[kBatches], scfull[kBatches];
  uint64_t gfull[2], gempty[2];           // staged 4-bit rows
  uint64_t qfull[kQRing], qfree;
  uint64_t sfull[2], sempty[2], pfull[2], pvdone[2], odrained, done;
  uint64_t hand0[4], hand1[4];            // the reference after a block of group 0, 1, to the other group's warp
};

// Keys of query t (every position): those up to its own that the table covers.
__device__ __forceinline__ long long keys_of(const Args& a, int t, int* b_out, unsigned* bad) {
  if (t >= __ldg(a.cu + a.B)) {
    *b_out = 0;
    return 0;
  }
  const int b = sequence_of(a.cu, a.B, t);
  *b_out = b;
  long long n = static_cast<long long>(__ldg(a.lens + b)) - __ldg(a.cu + b + 1) + t + 1;
  const long long room = min(static_cast<long long>(a.max_pages) * a.page_size, kMostKeys);
  if (n > room) {
    *bad = 1;
    n = room;
  }
  return n < 0 ? 0 : n;
}

// The line of all blocks: tile w = (query w / groups, heads 64 (w % groups) ..) holds the places
// tile_begin(w) .. tile_begin(w + 1) - 1, part c the places part_begin(c) .. part_begin(c + 1) - 1.
struct Line {
  long long total;
  int parts;
};
__device__ __forceinline__ long long tile_begin(const Args& a, int w) {
  if (a.nb) return static_cast<long long>(w) * a.nb;
  const int t = w / a.groups, g = w - t * a.groups;
  const long long c0 = __ldg(a.cum + t);
  return c0 * a.groups + (g ? g * (__ldg(a.cum + t + 1) - c0) : 0);
}
__device__ __forceinline__ Line line_of(const Args& a) {
  Line l;
  l.total = tile_begin(a, a.total_q * a.groups);
  l.parts = static_cast<int>(min(static_cast<long long>(a.parts), l.total));
  return l;
}
__device__ __forceinline__ long long part_begin(const Line& l, int c) { return l.total * c / l.parts; }
// The tile that holds place u.
__device__ __forceinline__ int tile_at(const Args& a, long long u) {
  if (a.nb) return static_cast<int>(u / a.nb);
  int lo = 0, hi = a.total_q * a.groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile_begin(a, mid) <= u) lo = mid; else hi = mid;
  }
  return lo;
}

// The pieces of a part, in order; every role walks them by itself.
struct Pieces {
  long long u, end, t_end;  // the next piece's first place, the part's end, its tile's end
  int w, t, g, k0, k1, blocks;  // the current piece: blocks k0 .. k1 - 1 of `blocks`
  __device__ __forceinline__ Pieces(const Args& a, const Line& l, int c) {
    u = c < l.parts ? part_begin(l, c) : 0;
    end = c < l.parts ? part_begin(l, c + 1) : 0;
    w = u < end ? tile_at(a, u) : 0;
    --w;
    t_end = u;
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

// The keys of a query: the position of each, -1 where there is none.
struct Keys {
  int b, len;
  long long n;  // keys (every position)
  const int32_t* sel;
  const int32_t* table;
  __device__ __forceinline__ Keys(const Args& a, int t, bool report) {
    unsigned bad = 0;
    if (a.nb) {
      const bool live = t < __ldg(a.cu + a.B);
      b = live ? sequence_of(a.cu, a.B, t) : 0;
      len = live ? __ldg(a.lens + b) : 0;
      n = a.topk_width;
      sel = a.topk + static_cast<long long>(t) * a.topk_width;
    } else {
      n = keys_of(a, t, &b, &bad);
      len = 0;
      sel = nullptr;
    }
    if (bad && report) atomicOr(a.status, kStatusUncovered);
    table = a.block_tables + static_cast<long long>(b) * a.max_pages;
  }
  __device__ __forceinline__ int position(const Args& a, int key) const {
    if (key >= n) return -1;
    if (!a.nb) return key;
    const int s = __ldg(sel + key);
    return s < len ? s : -1;
  }
};
// The cache row of a position, through a request's table; a.past_row where there is none.
__device__ __forceinline__ int row_of(const Args& a, const int32_t* table, int pos) {
  if (pos < 0) return a.past_row;
  const int lp = a.page_log2 >= 0 ? pos >> a.page_log2 : pos / a.page_size;
  const int page = lp < a.max_pages ? __ldg(table + lp) : -1;
  if (page < 0 || page >= a.num_pages) {
    atomicOr(a.status, kStatusBadPage);
    return a.past_row;
  }
  return page * a.page_size + (pos - lp * a.page_size);
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
// Whether v is non-zero in any of the 128 threads at named barrier `id`.
__device__ __forceinline__ bool bar_any(uint32_t id, uint32_t v) {
  uint32_t any;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.or.pred p, %2, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
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
// Four values 0 <= p <= 2^8, given as 2^-8 p in fp16, as e4m3 codes (x) and the e5m2 codes of what they leave (y).
// 2^-8 p has e4m3's exponents as its low four and its subnormals where e4m3 has them, so rounding its bits to three
// of the mantissa is the code; e5m2 is the upper half of fp16.  (Conversions take the slow pipe, integers do not.)
__device__ __forceinline__ uint2 two_terms(__half2 a, __half2 b) {
  const uint32_t ua = *reinterpret_cast<const uint32_t*>(&a), ub = *reinterpret_cast<const uint32_t*>(&b);
  const uint32_t ra = (ua + 0x00400040u) & 0x7F807F80u, rb = (ub + 0x00400040u) & 0x7F807F80u;
  const __half2 up = __float2half2_rn(256.f);
  const __half2 la = __hmul2(__hsub2(a, *reinterpret_cast<const __half2*>(&ra)), up);
  const __half2 lb = __hmul2(__hsub2(b, *reinterpret_cast<const __half2*>(&rb)), up);
  return make_uint2(__byte_perm(ra << 1, rb << 1, 0x7531),
                    __byte_perm(*reinterpret_cast<const uint32_t*>(&la) + 0x00800080u,
                                *reinterpret_cast<const uint32_t*>(&lb) + 0x00800080u, 0x7531));
}
// Scale u = 2^E of a block's row `key` (0: no row, which takes no weight).
__device__ __forceinline__ void put_scale(float4* block, int key, float u) {
  float* pair = reinterpret_cast<float*>(block + (key >> 1)) + (key & 1);
  pair[0] = u;
  pair[2] = u > 0.f ? static_cast<float>(static_cast<int>(__float_as_uint(u) >> 23) - 127 - kExpRef) : -INFINITY;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
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

template <bool FP4>
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
  uint2* levels = reinterpret_cast<uint2*>(misc + 576);                 // [8] magnitudes of the 4-bit codes
  float* linv = reinterpret_cast<float*>(misc + 768);                   // [64] of the piece that is written
  float* corr = reinterpret_cast<float*>(misc + 1024);                  // [2][64] each group's
  float* refv = reinterpret_cast<float*>(misc + 1536);                  // [2][64] the reference after its last block
  uint32_t* movedv = reinterpret_cast<uint32_t*>(misc + 640);           // [2][4] moved heads of each group's warps
  float* lsum = reinterpret_cast<float*>(misc + 2048);                  // [2][64]
  float* qscale = reinterpret_cast<float*>(misc + 3072);                // [kQRing][64]
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
      ptx::mbar_init(&bars->sempty[s], 4);
      ptx::mbar_init(&bars->pfull[s], 4);
      ptx::mbar_init(&bars->pvdone[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      ptx::mbar_init(&bars->hand0[s], 1);
      ptx::mbar_init(&bars->hand1[s], 1);
    }
    for (int s = 0; s < kQRing; ++s) ptx::mbar_init(&bars->qfull[s], 4);
    ptx::mbar_init(&bars->qfree, 1);
    ptx::mbar_init(&bars->odrained, 8);
    ptx::mbar_init(&bars->done, 1);
    *abort = 0;
    ptx::fence_mbar_init();
  }
  if (FP4 && threadIdx.x < 8) levels[threadIdx.x] = levels_base(threadIdx.x);
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

  const Line line = line_of(a);
  const int part = blockIdx.x;
  Pieces pc(a, line, part);
  auto wait = [&](uint64_t* bar, uint32_t parity) { return ptx::mbar_try_wait(bar, parity) || wait_on(bar, parity, abort, a.status); };
  const uint32_t sbase = ptx::smem_u32(smem);

  if (warp == 13) {
    // ------------------------------------------------------------ MMAs
    // One elected lane runs the whole loop, its waits too: under any condition that the compiler cannot see to be
    // the same for the warp, an MMA takes some 90 cycles to issue.
    if (ptx::elect_one()) {
      const uint32_t id_qk = ptx::idesc_f32acc(128, kKeys, false), id_qr = ptx::idesc_f32acc(128, kKeys, true);
      const uint32_t tile0 = ptx::desc_lo(sbase + L::kOffTile, kAtom), rope0 = ptx::desc_lo(sbase + L::kOffQr, 16);
      const uint32_t p0 = ptx::desc_lo(sbase + L::kOffP, 16);
      int it = 0, n = 0;  // blocks, pieces
      bool ok = true;
      while (ok && pc.next(a)) {
        const int cnt = pc.k1 - pc.k0, hg = min(kHeads, a.H - pc.g * kHeads);
        const uint32_t id_pv = ptx::idesc_f32acc(128, (hg + 15) & ~15, false) | (1u << 15);
        ok = wait(&bars->qfull[n % kQRing], (n / kQRing) & 1);
        // S runs two blocks ahead: both groups of softmax warps have their next block when they are done with one.
        for (int i = 0; i < cnt + 2 && ok; ++i) {
          if (i < cnt) {  // S of block i
            const int b = it + i;
            ok = wait(&bars->tfull[b % kStages], (b / kStages) & 1) && (b < 2 || wait(&bars->sempty[b & 1], ((b >> 1) & 1) ^ 1));
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t d = tmem + kColS + (b & 1) * kKeys;
            uint32_t kd = tile0 + (b % kStages) * (kTile >> 4), qd = rope0;
            asm volatile("" : "+r"(kd), "+r"(qd));  // descriptors are added up here, not kept over the loop
#pragma unroll
            for (int s = 0; s < 16; ++s)  // 32 codes of K per MMA, four in a column
              mma_f8_ts(d, tmem + kColQ + s * 8, kd + (((s >> 2) * kAtom + (s & 3) * 32) >> 4), id_qk, s > 0 ? 1u : 0u);
#pragma unroll
            for (int s = 0; s < 4; ++s) mma_bf16_ss(d, qd + 2 * s, kd + ((4 * kAtom) >> 4) + 2 * s, id_qr, 1u);
            ptx::mma_commit(&bars->sfull[b & 1]);
            if (i == cnt - 1) ptx::mma_commit(&bars->qfree);
          }
          if (i < 2) continue;
          const int b = it + i - 2;  // P . V of the block before the last
          ok = wait(&bars->pfull[b & 1], (b >> 1) & 1) && (i > 2 || n == 0 || wait(&bars->odrained, (n - 1) & 1));
          if (!ok) break;
          ptx::tc_fence_after();
          uint32_t vd = tile0 + (b % kStages) * (kTile >> 4), pd = p0 + (b & 1) * (kPBytes >> 4);
          asm volatile("" : "+r"(vd), "+r"(pd));
#pragma unroll
          for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {  // 32 keys per MMA
              const uint32_t ad = vd + ((c * kAtom + s * 4096) >> 4);
              mma_f8_ss(tmem + kColO + c * kHeads, ad, pd + 2 * s, id_pv, (i > 2 || s > 0) ? 1u : 0u);
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
    int it = 0;
    bool ok = true;
    while (ok && pc.next(a)) {
      for (int k = pc.k0; k < pc.k1; ++k, ++it) {
        const int bt = (it / kBatch) % kBatches, st = it % kBufs;
        uint64_t* full = FP4 ? &bars->gfull[st] : &bars->tfull[st];
        ok = wait(&bars->rfull[bt], (it / kRing) & 1) &&
             (it < kBufs || wait(FP4 ? &bars->gempty[st] : &bars->tempty[st], ((it / kBufs) & 1) ^ 1));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (ptx::elect_one()) {
          ptx::mbar_arrive_expect_tx(full, (FP4 ? kStaged : kTile) / 2);
          const int4* y4 = reinterpret_cast<const int4*>(rows + (it % kRing) * kKeys) + first;
#pragma unroll 4
          for (int g = 0; g < 8; ++g) {
            const int4 v = y4[g];
            const int y[4] = {v.x, v.y, v.z, v.w};
            if (FP4) {
              tma_gather4(smem + L::kOffStaged + st * kStaged + (first + g) * 4 * kRow4, &tmap, full, 0, y);
            } else {
#pragma unroll
              for (int c = 0; c < 5; ++c)
                tma_gather4(smem + L::kOffTile + st * kTile + c * kAtom + (first + g) * 512, &tmap, full, c * 64, y);
            }
          }
          if (it % kBatch == kBatch - 1) ptx::mbar_arrive(&bars->bempty[bt]);
        }
        __syncwarp();
      }
    }
    // copies in flight land before the CTA can exit, whatever happened
    for (int i = max(0, it - kBufs); i < it; ++i)
      ptx::mbar_spin_drain(FP4 ? &bars->gfull[i % kBufs] : &bars->tfull[i % kBufs], (i / kBufs) & 1, a.status, kStatusTimeout, 400000000ll);
  } else if (warp == 14) {
    // ------------------------------------------------------------ where the rows lie; scales of e4m3 rows
    bool more = pc.next(a);
    Keys keys(a, more ? pc.t : 0, lane == 0 && more);
    int k = pc.k0;
    for (int it = 0; more; it += kBatch) {
      int y[2 * kBatch];
      const int32_t* table[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        y[2 * j] = y[2 * j + 1] = -1;
        table[j] = keys.table;
        if (!more) continue;
        y[2 * j] = keys.position(a, k * kKeys + lane);
        y[2 * j + 1] = keys.position(a, k * kKeys + 32 + lane);
        if (++k == pc.k1) {
          more = pc.next(a);
          if (more) keys = Keys(a, pc.t, lane == 0);
          k = pc.k0;
        }
      }
#pragma unroll
      for (int j = 0; j < 2 * kBatch; ++j) y[j] = row_of(a, table[j >> 1], y[j]);
      const int bt = (it / kBatch) % kBatches;
      bool ok = it < kRing || wait(&bars->bempty[bt], ((it / kRing) & 1) ^ 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
#pragma unroll
      for (int j = 0; j < 2 * kBatch; ++j) rows[(bt * kBatch + (j >> 1)) * kKeys + 32 * (j & 1) + lane] = y[j];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars->rfull[bt]);
      if constexpr (!FP4) {
        float u[2 * kBatch];
  #pragma unroll
        for (int j = 0; j < 2 * kBatch; ++j)
          u[j] = y[j] != a.past_row ? __ldg(reinterpret_cast<const float*>(a.cache + static_cast<long long>(y[j]) * kRow8 + kScale8)) : 0.f;
  #pragma unroll
        for (int j = 0; j < 2 * kBatch; ++j)
          put_scale(sc + (bt * kBatch + (j >> 1)) * (kKeys / 2), 32 * (j & 1) + lane, u[j]);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->scfull[bt]);
      }
    }
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
    int it = 0, n = 0;
    bool ok = true;
    while (ok && pc.next(a)) {
      const uint4* src[4];
      bool live[4];
      uint4 rp[4];
      float am[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = pc.g * kHeads + w * 16 + 4 * i + hr;
        live[i] = h < a.H;
        src[i] = reinterpret_cast<const uint4*>(a.qn + pc.t * a.qn_t + (live[i] ? h : 0) * a.qn_h) + l8;
        rp[i] = live[i] ? __ldg(reinterpret_cast<const uint4*>(a.qr + pc.t * a.qr_t + h * a.qr_h) + l8) : make_uint4(0u, 0u, 0u, 0u);
        am[i] = 0.f;
      }
      auto load = [&](int c, uint4 (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = live[i] ? __ldg(src[i] + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
      };
      auto most = [&](const uint4 (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x[8];
          unpack_bf16(v[i], x);
#pragma unroll
          for (int j = 0; j < 8; ++j) am[i] = fmaxf(am[i], fabsf(x[j]));
        }
      };
      // (the chunks that the conversion begins with come last)
      uint4 v[2][4];
#pragma unroll 1
      for (int c = 6; c >= 0; c -= 2) {
        load(c, v[0]);
        load(c + 1, v[1]);
        most(v[0]);
        most(v[1]);
      }
      most(rp);
      // the power of two that takes the row's largest value to [128, 256)
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) am[i] = fmaxf(am[i], __shfl_xor_sync(0xffffffffu, am[i], o));
        const int e = am[i] > 0.f ? max(-60, min(60, 7 - (static_cast<int>(__float_as_uint(am[i]) >> 23) - 127))) : 0;
        f[i] = pow2f(e);
        if (l8 == 0) qscale[(n % kQRing) * kHeads + w * 16 + 4 * i + hr] = a.scale_log2 * pow2f(-e);
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
        unpack_bf16(rp[i], x);
        *reinterpret_cast<uint4*>(smem + L::kOffQr + r * 128 + ((l8 ^ (r & 7)) << 4)) =
            make_uint4(pack_bf16(x[0] * f[i], x[1] * f[i]), pack_bf16(x[2] * f[i], x[3] * f[i]),
                       pack_bf16(x[4] * f[i], x[5] * f[i]), pack_bf16(x[6] * f[i], x[7] * f[i]));
      }
      // 64 values of every row at a time: codes to shared memory, from there by rows to TMEM
      auto convert = [&](int c, const uint4 (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x[8];
          unpack_bf16(v[i], x);
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float v0 = x[4 * j] * f[i], v1 = x[4 * j + 1] * f[i], v2 = x[4 * j + 2] * f[i], v3 = x[4 * j + 3] * f[i];
            const uint32_t h01 = e4m3x2(v0, v1), h23 = e4m3x2(v2, v3);
            const float2 b01 = from_e4m3x2(h01), b23 = from_e4m3x2(h23);
            constexpr float up = 1 << kLoShift;
            hi[j] = h01 | (h23 << 16);
            lo[j] = e4m3x2((v0 - b01.x) * up, (v1 - b01.y) * up) | (e4m3x2((v2 - b23.x) * up, (v3 - b23.y) * up) << 16);
          }
          *reinterpret_cast<uint2*>(qbuf + (4 * i + hr) * kQStride + l8 * 8) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(qbuf + (16 + 4 * i + hr) * kQStride + l8 * 8) = make_uint2(lo[0], lo[1]);
        }
        __syncwarp();
        uint32_t r[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 q = *reinterpret_cast<const uint4*>(qbuf + lane * kQStride + 16 * j);
          r[4 * j] = q.x, r[4 * j + 1] = q.y, r[4 * j + 2] = q.z, r[4 * j + 3] = q.w;
        }
        tmem_st_32x32b_x16(tmem + lane_addr + kColQ + 16 * c, r);
        __syncwarp();
      };
#pragma unroll 1
      for (int c = 0; c < 8; c += 2) {
        convert(c, v[0]);
        if (c < 6) load(c + 2, v[0]);
        convert(c + 1, v[1]);
        if (c < 6) load(c + 3, v[1]);
      }
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars->qfull[n % kQRing]);
      ++n;
      if constexpr (FP4) {
        // 4-bit rows: a warp takes 16 rows of a block, a lane a block of 16 values
        for (int k = pc.k0; k < pc.k1; ++k, ++it) {
          const int st = it % kStages, gs = it & 1, bt = (it / kBatch) % kBatches;
          ok = wait(&bars->gfull[gs], (it >> 1) & 1) && (it < kStages || wait(&bars->tempty[st], ((it / kStages) & 1) ^ 1));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const bool there = rows[(it % kRing) * kKeys + w * 16 + (lane & 15)] != a.past_row;  // of key 16 w + lane
          const uint8_t* staged = smem + L::kOffStaged + gs * kStaged + w * 16 * kRow4;
          uint8_t* tile = smem + L::kOffTile + st * kTile;
          int E = 0;
  #pragma unroll
          for (int i0 = 0; i0 < 16; i0 += 8) {
            uint2 q[8], lv[8];
            int byte[8];
  #pragma unroll
            for (int i = 0; i < 8; ++i) {
              byte[i] = staged[(i0 + i) * kRow4 + kScale4 + lane];
              q[i] = reinterpret_cast<const uint2*>(staged + (i0 + i) * kRow4)[lane];
            }
  #pragma unroll
            for (int i = 0; i < 8; ++i) lv[i] = levels[byte[i] & 7];
  #pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int key = w * 16 + i0 + i;
              const int e = static_cast<int>(__ballot_sync(0xffffffffu, byte[i] >> 7) & 0xFFu) - 128;
              if (lane == i0 + i) E = e;
              const uint2 l2 = levels_at(lv[i], byte[i] & 127);
              const uint2 c0 = codes4_to_e4m3(q[i].x, l2), c1 = codes4_to_e4m3(q[i].y, l2);
              *reinterpret_cast<uint4*>(tile + (lane >> 3) * kAtom + key * 128 + ((l8 ^ (key & 7)) << 4)) =
                  make_uint4(c0.x, c0.y, c1.x, c1.y);
            }
          }
          uint4 rr[4];
  #pragma unroll
          for (int i = 0; i < 4; ++i) rr[i] = reinterpret_cast<const uint4*>(staged + (4 * i + hr) * kRow4 + kRope4)[l8];
  #pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = w * 16 + 4 * i + hr;
            *reinterpret_cast<uint4*>(tile + 4 * kAtom + key * 128 + ((l8 ^ (key & 7)) << 4)) = rr[i];
          }
          if (lane < 16) put_scale(sc + st * (kKeys / 2), w * 16 + lane, there ? pow2f(E) : 0.f);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(&bars->gempty[gs]);
            ptx::mbar_arrive(&bars->scfull[st]);
            ptx::mbar_arrive(&bars->tfull[st]);
            if (it % kBatch == kBatch - 1) ptx::mbar_arrive(&bars->bempty[bt]);
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax, rescale, output
    const int grp = warp >> 2, w = warp & 3, half = lane >> 4, hl = w * 16 + (lane & 15);
    const uint32_t lane_addr = static_cast<uint32_t>(w * 32) << 16;
    uint64_t* mine = grp ? &bars->hand1[w] : &bars->hand0[w];
    uint64_t* other = grp ? &bars->hand0[w] : &bars->hand1[w];
    int it = 0, n = 0;
    bool ok = true;
    // Every piece and block runs its named barriers whatever happened, so that a wait that gave up leaves no
    // warp behind at one.
    while (pc.next(a)) {
      const int cnt = pc.k1 - pc.k0, hg = min(kHeads, a.H - pc.g * kHeads), end = it + cnt;
      float m = -INFINITY;  // the group's reference at its last block
      float2 l = make_float2(0.f, 0.f), qm = l, qo = l;  // its sum, in two parts; the planes' scales
      if (ok) ok = __all_sync(0xffffffffu, wait(&bars->qfull[n % kQRing], (n / kQRing) & 1)) != 0;
      if (ok) {
        const float qs = qscale[(n % kQRing) * kHeads + hl];
        qm.x = qm.y = half ? qs * (1.f / (1 << kLoShift)) : qs;  // of this lane's plane, and of the other's
        qo.x = qo.y = half ? qs : qs * (1.f / (1 << kLoShift));
      }
      for (int b = it + ((it ^ grp) & 1); b < end; b += 2) {
        const int ss = FP4 ? b % kStages : b % kRing;
        const uint32_t col = tmem + lane_addr + kColS + grp * kKeys;
        const float4* scp = sc + ss * (kKeys / 2) + half * 16;
        float cr = 1.f;
        if (ok)
          ok = __all_sync(0xffffffffu, wait(&bars->sfull[grp], (b >> 1) & 1) &&
                                           (FP4 ? wait(&bars->scfull[ss], (b / kStages) & 1)
                                                : wait(&bars->scfull[(b / kBatch) % kBatches], (b / kRing) & 1))) != 0;
        if (ok) {
          // x' of the block, 16 keys at a time (the hi lane takes keys 0..31, the lo lane 32..63), back over S.
          // Both passes are loops: as straight code the two groups' block is more than an SM's schedulers hold of
          // instructions (a third of the cycles went by waiting for them).
          ptx::tc_fence_after();
          float2 mx = make_float2(-INFINITY, -INFINITY);
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t s0[16], s1[16], x[16];
            tmem_ld_x16(col + 16 * c, s0);
            tmem_ld_x16(col + 32 + 16 * c, s1);
            tmem_ld_wait16(s0, s1);
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              float2 keep, got;
              keep.x = __uint_as_float(half ? s1[j] : s0[j]);
              keep.y = __uint_as_float(half ? s1[j + 1] : s0[j + 1]);
              got.x = __uint_as_float(__shfl_xor_sync(0xffffffffu, half ? s0[j] : s1[j], 16));
              got.y = __uint_as_float(__shfl_xor_sync(0xffffffffu, half ? s0[j + 1] : s1[j + 1], 16));
              const float4 v = scp[8 * c + (j >> 1)];
              float2 y = mul2(keep, qm);
              ptx::ffma2(y, got, qo);
              float2 z = make_float2(v.z, v.w);
              ptx::ffma2(z, y, make_float2(v.x, v.y));
              mx.x = fmaxf(mx.x, z.x);
              mx.y = fmaxf(mx.y, z.y);
              x[j] = __float_as_uint(z.x);
              x[j + 1] = __float_as_uint(z.y);
            }
            tmem_st_32x32b_x16(col + 16 * c, x);
          }
          ptx::tmem_st_wait();
          float mb = fmaxf(mx.x, mx.y);
          mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 16));
          if (b > 0) ok = __all_sync(0xffffffffu, wait(other, ((b - 1) >> 1) & 1)) != 0;
          if (ok) {
            const float before = b == end - cnt ? -INFINITY : refv[(grp ^ 1) * kHeads + hl];
            // The reference moves only when it is passed by more than kMove, so that most blocks leave O as it is.
            float mn = before;
            if (before == -INFINITY || mb > before + kMove) mn = mb;
            cr = before == -INFINITY ? 1.f : ptx::ex2(before - mn);
            const float f = m == -INFINITY ? 0.f : ptx::ex2(m - mn);
            l.x *= f;
            l.y *= f;
            m = mn;
            if (!half) {
              refv[grp * kHeads + hl] = mn;
              corr[grp * kHeads + hl] = cr;
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(mine);
          }
          // the group's P is free once the products of its block before have been done
          if (ok && b > 1) ok = __all_sync(0xffffffffu, wait(&bars->pvdone[grp], ((b >> 1) & 1) ^ 1)) != 0;
        }
        if (ok) {
          const float ref = m == -INFINITY ? 0.f : (kPShift - 8) - m;
          uint8_t* prow = smem + L::kOffP + grp * kPBytes + hl * 128;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t x[16], hi[4], lo[4];
            tmem_ld_x16(col + 16 * c, x);
            tmem_ld_wait16(x);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float2 p[2];
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const uint2 u = *reinterpret_cast<const uint2*>(scp + 8 * c + 2 * j + q);
                constexpr uint32_t kInv = static_cast<uint32_t>(254 + kExpRef) << 23;
                p[q] = add2(make_float2(__uint_as_float(x[4 * j + 2 * q]), __uint_as_float(x[4 * j + 2 * q + 1])), ref);
                p[q] = make_float2(ptx::ex2(p[q].x), ptx::ex2(p[q].y));  // 2^-8 p
                ptx::ffma2(l, p[q], make_float2(__uint_as_float(kInv - u.x), __uint_as_float(kInv - u.y)));  // 2^-8 p 2^(kExpRef - E)
              }
              const uint2 t = two_terms(__floats2half2_rn(p[0].x, p[0].y), __floats2half2_rn(p[1].x, p[1].y));
              hi[j] = t.x;
              lo[j] = t.y;
            }
            const int ch = half * 2 + c;
            *reinterpret_cast<uint4*>(prow + ((ch ^ (hl & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(prow + (((4 + ch) ^ (hl & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
          ptx::tc_fence_before();
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&bars->sempty[grp]);
        }
        // Heads whose reference moved: their columns of O are rescaled when the products of the block before are
        // done and before those of this one begin (which wait for them in any case).
        const unsigned moved = __ballot_sync(0xffffffffu, !half && hl < hg && cr != 1.f);
        if (lane == 0) movedv[grp * 4 + w] = moved;
        if (bar_any(2 + grp, moved)) {
          if (ok) ok = __all_sync(0xffffffffu, wait(&bars->pvdone[grp ^ 1], ((b - 1) >> 1) & 1)) != 0;
          if (ok) {
            ptx::tc_fence_after();
            const uint2 m01 = *reinterpret_cast<const uint2*>(movedv + grp * 4), m23 = *reinterpret_cast<const uint2*>(movedv + grp * 4 + 2);
            uint64_t todo = (m01.x | m01.y << 16) | static_cast<uint64_t>(m23.x | m23.y << 16) << 32;
            const uint32_t o = tmem + lane_addr + kColO;
            const float* f = corr + grp * kHeads;
            if (__popcll(todo) <= kFewHeads) {
              for (; todo; todo &= todo - 1) {
                const int h = __ffsll(static_cast<long long>(todo)) - 1;
                float r[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) r[c] = tmem_ld_x1(o + c * kHeads + h);
                tmem_ld_wait4(r);
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_st_x1(o + c * kHeads + h, r[c] * f[h]);
              }
            } else {
#pragma unroll 1
              for (int q = 0; q < 16; ++q) {
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
          ptx::named_bar_sync(2 + grp, 128);  // corr is read before the group's next block rewrites it
        }
        if (ok) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(&bars->pfull[grp]);
            if (!FP4 && (b % kBatch) >> 1 == kBatch / 2 - 1) ptx::mbar_arrive(&bars->bempty[(b / kBatch) % kBatches]);
          }
        }
      }
      it = end;
      ++n;
      // the piece's output: the sums of both groups against the last reference
      const int last = (end - 1) & 1;
      if (ok)
        ok = __all_sync(0xffffffffu, (last == grp || wait(other, ((end - 1) >> 1) & 1)) &&
                                         wait(&bars->pvdone[last], ((end - 1) >> 1) & 1)) != 0;
      const float fin = refv[last * kHeads + hl];
      float sum = m == -INFINITY ? 0.f : (l.x + l.y) * ptx::ex2(m - fin);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      if (!half) lsum[grp * kHeads + hl] = sum;
      ptx::named_bar_sync(4, 256);
      const bool whole = pc.k0 == 0 && pc.k1 == pc.blocks;
      const int slot = 2 * part + (pc.k0 == 0 ? 1 : 0);
      if (grp == 0 && !half) {
        sum = lsum[hl] + lsum[kHeads + hl];
        linv[hl] = sum == 0.f ? 0.f : pow2f(kExpRef - 8) / sum;
        if (hl < hg && ok) {
          if (!whole) {
            a.part_ml[(static_cast<long long>(slot) * kHeads + hl) * 2] = fin;
            a.part_ml[(static_cast<long long>(slot) * kHeads + hl) * 2 + 1] = sum;
          } else if (a.lse) {
            a.lse[static_cast<long long>(pc.t) * a.H + pc.g * kHeads + hl] = sum == 0.f ? -INFINITY : (fin - (kPShift - 8) + log2f(sum)) * kLn2;
          }
        }
      }
      ptx::named_bar_sync(4, 256);
      if (ok) {
        ptx::tc_fence_after();
        const int lat = w * 32 + lane;
        const bool odd = lane & 1;
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {  // this group's two latent chunks, 16 heads at a time
          const int c = 2 * grp + (q >> 2), h0 = (q & 3) * 16;
          if (h0 >= hg) continue;
          uint32_t r[16];
          tmem_ld_x16(tmem + lane_addr + kColO + c * kHeads + h0, r);
          tmem_ld_wait16(r);
          if (whole) {
            // pairs of lanes swap, so that each stores two latent values of one head
            uint32_t* o = reinterpret_cast<uint32_t*>(a.out + (static_cast<long long>(pc.t) * a.H + pc.g * kHeads + h0 + odd) * kRank + c * 128) + (lat >> 1);
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float2 f = *reinterpret_cast<const float2*>(linv + h0 + j);
              const float v0 = __uint_as_float(r[j]) * f.x, v1 = __uint_as_float(r[j + 1]) * f.y;
              const float got = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
              if (h0 + j + odd < hg) o[j * (kRank / 2)] = odd ? pack_bf16(got, v1) : pack_bf16(v0, got);
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
  if (warp == 13) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// out = sum_j 2^(m_j - M) O_j / sum_j 2^(m_j - M) L_j over the pieces of a tile, in their order.  Block (c - 1, y): the
// tile that part c begins inside, if no earlier part does; y: four heads, a latent chunk.
__global__ void __launch_bounds__(128) quant_join_kernel(const Args a) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const Line line = line_of(a);
  const int c = blockIdx.x + 1, quad = blockIdx.y & 15, chunk = blockIdx.y >> 4;
  if (c >= line.parts) return;
  const long long u = part_begin(line, c);
  const int w = tile_at(a, u);
  const long long b = tile_begin(a, w), e = tile_begin(a, w + 1);
  if (b == u || part_begin(line, c - 1) > b) return;
  const int t = w / a.groups, g = w - t * a.groups, h0 = g * kHeads + quad * 4;
  if (h0 >= a.H) return;
  int last = c;
  while (last + 1 < line.parts && part_begin(line, last + 1) < e) ++last;
  float M[4], W[4] = {0.f, 0.f, 0.f, 0.f}, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) M[i] = -INFINITY;
  for (int j = c - 1; j <= last; ++j) {
    const float* ml = a.part_ml + (static_cast<long long>(2 * j + (j == c - 1 ? 1 : 0)) * kHeads + quad * 4) * 2;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (h0 + i < a.H) M[i] = fmaxf(M[i], ml[2 * i]);
  }
  for (int j = c - 1; j <= last; ++j) {
    const long long slot = 2 * j + (j == c - 1 ? 1 : 0);
    const float* ml = a.part_ml + (slot * kHeads + quad * 4) * 2;
    const float4 o = reinterpret_cast<const float4*>(a.part_o)[((slot * 4 + chunk) * 16 + quad) * 128 + threadIdx.x];
    const float v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (h0 + i >= a.H) continue;
      const float mj = ml[2 * i];
      if (mj == -INFINITY) continue;
      const float f = exp2f(mj - M[i]);
      W[i] += f * ml[2 * i + 1];
      acc[i] += f * v[i];
    }
  }
  const long long row = static_cast<long long>(t) * a.H + h0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (h0 + i >= a.H) continue;
    a.out[(row + i) * kRank + chunk * 128 + threadIdx.x] = __float2bfloat16_rn(W[i] == 0.f ? 0.f : ldexpf(acc[i] / W[i], kExpRef - 8));
    if (chunk == 0 && threadIdx.x == i && a.lse) a.lse[row + i] = W[i] == 0.f ? -INFINITY : (M[i] - (kPShift - 8) + log2f(W[i])) * kLn2;
  }
}

// Blocks before each query (every position): at least one a query, so that each has a tile that writes it.
__global__ void __launch_bounds__(1024) quant_plan_kernel(const Args a, long long* cum) {
  __shared__ long long sums[32];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long before = 0;
  for (int t0 = 0; t0 < a.total_q; t0 += 1024) {
    const int t = t0 + threadIdx.x;
    long long v = 0;
    if (t < a.total_q) {
      int b;
      unsigned bad = 0;
      v = max(1ll, (keys_of(a, t, &b, &bad) + kKeys - 1) / kKeys);
    }
    long long s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += x;
    }
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    long long w = sums[lane], add = 0;
    for (int i = 0; i < 32; ++i) {
      const long long x = __shfl_sync(0xffffffffu, w, i);
      if (i < warp) add += x;
    }
    if (t < a.total_q) cum[t] = before + add + s - v;
    long long total = 0;
    for (int i = 0; i < 32; ++i) total += __shfl_sync(0xffffffffu, w, i);
    before += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) cum[a.total_q] = before;
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

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return n > 0 ? n : 148;
}

struct Plan {
  int groups, nb, parts;
  size_t off_ml, off_cum, total;
};
Plan plan_of(const dsa_quant_mla_args* a) {
  Plan p{};
  p.groups = (a->H + kHeads - 1) / kHeads;
  p.nb = (a->topk_width + kKeys - 1) / kKeys;
  long long parts = sm_count();
  if (p.nb) parts = std::min<long long>(parts, static_cast<long long>(a->total_q) * p.groups * p.nb);
  p.parts = static_cast<int>(std::max<long long>(1, parts));
  p.off_ml = static_cast<size_t>(2) * p.parts * kHeads * kRank * 4;
  p.off_cum = p.off_ml + static_cast<size_t>(2) * p.parts * kHeads * 2 * 4;
  p.total = p.off_cum + (p.nb ? 0 : (static_cast<size_t>(a->total_q) + 1) * 8);
  return p;
}

template <bool FP4>
cudaError_t launch_attend(const CUtensorMap& map, const Args& k, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(quant_mla_kernel<FP4>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<FP4>::kBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(quant_mla_kernel<FP4>, dim3(k.parts), dim3(kThreads), Smem<FP4>::kBytes, s, map, k);
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
  if (!a->workspace || a->workspace_bytes < p.total || !al(a->workspace, 16)) return DSA_ERR_WORKSPACE;
  unsigned* status = device_status_ptr();
  if (!status) return DSA_ERR_CUDA;
  Args k{};
  k.B = a->B;
  k.total_q = a->total_q;
  k.H = a->H;
  k.groups = p.groups;
  k.page_size = a->page_size;
  k.page_log2 = -1;
  for (int i = 0; i < 31; ++i)
    if (a->page_size == 1 << i) k.page_log2 = i;
  k.num_pages = a->num_pages;
  k.max_pages = a->max_pages_per_seq;
  k.topk_width = a->topk_width;
  k.nb = p.nb;
  k.parts = p.parts;
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
  k.status = status;
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
  e = fp4 ? launch_attend<true>(map, k, s) : launch_attend<false>(map, k, s);
  if (e != cudaSuccess) return DSA_ERR_CUDA;
  if (p.parts > 1) e = launch_pdl(quant_join_kernel, dim3(p.parts - 1, 64), dim3(128), 0, s, k);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
