// quant_append.cu -- the step's latent rows (norm, RoPE) in 8 or 4 bits through slot_mapping into the paged cache.
//
//     c = w * x / sqrt(mean(x^2) + eps),   r = RoPE(r, position),   row = codes of c / 2^E, r / 2^E, scales
//
// A code is that of c in exact arithmetic.  In fp32, c is off by up to 13 * 2^-24 (12 roundings of the sum of squares
// and eps count half through the root, which is 2 * 2^-24 off itself; then two products and the three of its scaling),
// which moves a value next to a border between two codes over it: once in some 10^5 values, by a whole step of the code.
// So each decision (the row's exponent, a block's scale, every code) is taken for c (1 - 2^-20) and for c (1 + 2^-20);
// where the two differ, one row in some 100, the warp takes the row again with two floats a value.  Without norm c is the
// input and fp32 is exact.
//
// One warp takes a token: lane i holds the values 16 i .. 16 i + 15, which are one block of the 4-bit format.
// In a graph with the read-back of the same rows: 64 tokens 6.2 us (latency: launch, slot, row, reductions, store; rows
// that are taken again 1 us of it), 8193 tokens in 8 bits 12.4 (4.7 at the copy bandwidth), 74968 in 4 bits 78 (38): there
// the arithmetic of the decisions, some 90 instructions a value pair, takes longer than the bytes.
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"
#include "quant_rows.cuh"

namespace dsa {
namespace {

using namespace quant;

constexpr int kWarps = 4;
constexpr float kSlack = 1.f / 1048576.f;  // 2^-20

// The smallest E with amax <= TOP 2^E, within +-kMaxExp; 0 for a row of zeros.
template <bool FP4>
__device__ __forceinline__ int row_exponent(float amax) {
  constexpr uint32_t kTopMantissa = FP4 ? 0x580000u : 0x600000u;  // 432 = 1.6875 * 2^8, 448 = 1.75 * 2^8
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > kTopMantissa ? 1 : 0);
  return b == 0u ? 0 : max(-kMaxExp, min(kMaxExp, e));
}
// A block's scale: the smallest s of 4 significant bits, 2^-5 at least, with 6 s >= a.
__device__ __forceinline__ float block_scale(float a) {
  uint32_t s = __float_as_uint(fmaxf(a * (0.9999995f / 6.f), 0.03125f)) & 0xFFF00000u;  // at most the scale, two steps below at most
  if (6.f * __uint_as_float(s) < a) s += 0x100000u;
  if (6.f * __uint_as_float(s) < a) s += 0x100000u;
  return fminf(__uint_as_float(s), 72.f);
}
// Sums and products of two floats that carry what one loses.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {  // exact
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two two_prod(float a, float b) {  // exact
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Two add(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi);
  const float e = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)), h = __fadd_rn(s.hi, e);
  return {h, __fsub_rn(e, __fsub_rn(h, s.hi))};
}
// hi + lo as one float whose last bit is set where it was cut: rounding this to fewer bits rounds the sum.
__device__ __forceinline__ float to_odd(float hi, float lo) {
  const float s = __fadd_rn(hi, lo), e = __fsub_rn(lo, __fsub_rn(s, hi));
  if (e == 0.f) return __uint_as_float(__float_as_uint(s) | (__float_as_uint(hi) & 0x80000000u));  // (-0 + 0 is -0 here)
  const uint32_t b = __float_as_uint(s);
  return __uint_as_float(((e > 0.f) == (s > 0.f) ? b : b - 1u) | 1u);
}
// Standard nibbles (sign on top of each) to the row's order of signs.
__device__ __forceinline__ uint32_t place_signs(uint32_t w) {
  return (w & 0x77777777u) | ((w & 0x8u) << 4) | ((w & 0x80u) << 8) | ((w & 0x800u) << 12) | ((w & 0x8000u) << 16) |
         ((w >> 16) & 0x8u) | ((w >> 12) & 0x800u) | ((w >> 8) & 0x80000u) | ((w >> 4) & 0x8000000u);
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// What a lane stores of a row: its 16 codes (four words, or two and a scale), and the row's exponent.
struct Codes {
  uint32_t w[4];
  int scale;
  int E;
};

template <bool FP4>
__device__ __forceinline__ float amax16(const float (&v)[16]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(v[i]));
  return a;
}

// Codes of v, exact fp32 values (NORM off); with NORM, v is off by up to kSlack and *near is set where that may have
// changed a decision.
template <bool FP4, bool NORM>
__device__ __forceinline__ Codes encode(const float (&v)[16], bool* near) {
  Codes r;
  const float block = amax16<FP4>(v), amax = warp_max(block);
  const float lo = 1.f - kSlack, hi = 1.f + kSlack;
  r.E = row_exponent<FP4>(NORM ? amax * hi : amax);
  // the scales are chosen for the larger value; would the smaller one take less?
  bool off = NORM && amax > 0.f && amax * lo <= (FP4 ? kTop4 : kTop8) * pow2f(r.E - 1) && r.E > -kMaxExp;
  const float f = pow2f(-r.E);
  if (FP4) {
    const float a = block * f;
    const float s = block_scale(NORM ? a * hi : a);
    if (NORM) off |= a * lo <= 6.f * __uint_as_float(__float_as_uint(s) - 0x100000u) && s > 0.03125f;
    r.scale = static_cast<int>(__float_as_uint(s) >> 20) - (122 << 3);
    const float g = NORM ? f * __frcp_rn(s) : f;
    const float2 gl = make_float2(g * lo, g * lo), gh = make_float2(g * hi, g * hi);
    uint32_t differ = 0u;
    r.w[0] = r.w[1] = r.w[2] = r.w[3] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = make_float2(v[2 * i], v[2 * i + 1]);
      uint32_t c;
      if (NORM) {
        const float2 l = mul2(x, gl), h = mul2(x, gh);
        c = e2m1x2(l.x, l.y);
        differ |= c ^ e2m1x2(h.x, h.y);
      } else {
        c = e2m1x2(__fdiv_rn(x.x * g, s), __fdiv_rn(x.y * g, s));  // a tie divides exactly, and nothing else rounds to one
      }
      r.w[i >> 2] |= c << (8 * (i & 3));
    }
    if (NORM) off |= differ != 0u;
    r.w[0] = place_signs(r.w[0]);
    r.w[1] = place_signs(r.w[1]);
  } else {
    r.scale = 0;
    const float2 fl = make_float2(f * lo, f * lo), fh = make_float2(f * hi, f * hi);
    uint32_t differ = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = make_float2(v[4 * i], v[4 * i + 1]), y = make_float2(v[4 * i + 2], v[4 * i + 3]);
      if (NORM) {
        const float2 xl = mul2(x, fl), yl = mul2(y, fl), xh = mul2(x, fh), yh = mul2(y, fh);
        r.w[i] = e4m3x2(xl.x, xl.y) | (e4m3x2(yl.x, yl.y) << 16);
        differ |= r.w[i] ^ (e4m3x2(xh.x, xh.y) | (e4m3x2(yh.x, yh.y) << 16));
      } else {
        r.w[i] = e4m3x2(x.x * f, x.y * f) | (e4m3x2(y.x * f, y.y * f) << 16);
      }
    }
    if (NORM) off |= differ != 0u;
  }
  if (NORM) *near = off;
  return r;
}

// The same row with every value in two floats, 2^-44 of it off: x the inputs, w the weights.  (fp64 itself took 8 us for
// 64 rows, some of which always come here.)  A row whose squares are too small for fp32 is taken 2^80 times as large, which
// leaves c as it is.
template <bool FP4>
__device__ __noinline__ Codes encode_close(const float (&in)[16], const float (&w)[16], float eps, bool tiny) {
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = in[i] * (tiny ? 0x1p80f : 1.f);
  if (tiny) eps = eps * 0x1p80f * 0x1p80f;
  Two ss{0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 16; ++i) ss = add(ss, Two{x[i] * x[i], 0.f});  // (a square of 8 bits is exact)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Two other{__shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o)};
    ss = add(ss, other);
  }
  const Two mean = add(Two{ss.hi * (1.f / kRank), ss.lo * (1.f / kRank)}, Two{eps, 0.f});
  // 1 / sqrt(mean) = y + y r / 2, r = 1 - mean y^2
  const float y = mean.hi > 0.f ? rsqrtf(mean.hi) : 0.f;
  const Two yy = two_prod(y, y), my = two_prod(mean.hi, yy.hi);
  const float r0 = (1.f - my.hi) - (my.lo + (mean.hi * yy.lo + mean.lo * yy.hi));
  const float dy = 0.5f * y * r0;
  float v[16], rest[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const Two wx = two_prod(w[i], x[i]), p = two_prod(wx.hi, y);
    v[i] = p.hi;
    rest[i] = p.lo + (wx.hi * dy + wx.lo * y);
  }
  float odd[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) odd[i] = to_odd(v[i], rest[i]);
  // exponent and scales from the values cut to odd: one just above a border stays above it
  Codes r;
  const float block = amax16<FP4>(odd), amax = warp_max(block);
  r.E = row_exponent<FP4>(amax);
  const float f = pow2f(-r.E);
  if (!FP4) {
    r.scale = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r.w[i] = e4m3x2(odd[4 * i] * f, odd[4 * i + 1] * f) | (e4m3x2(odd[4 * i + 2] * f, odd[4 * i + 3] * f) << 16);
    return r;
  }
  const float s = block_scale(block * f);
  r.scale = static_cast<int>(__float_as_uint(s) >> 20) - (122 << 3);
  r.w[0] = r.w[1] = r.w[2] = r.w[3] = 0u;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float t = v[i] * f, q = __fdiv_rn(t, s);
    odd[i] = to_odd(q, __fdiv_rn(__fmaf_rn(-q, s, t) + rest[i] * f, s));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) r.w[i >> 2] |= e2m1x2(odd[2 * i], odd[2 * i + 1]) << (8 * (i & 3));
  r.w[0] = place_signs(r.w[0]);
  r.w[1] = place_signs(r.w[1]);
  return r;
}

template <bool FP4, bool NORM, int TOK>
__global__ void __launch_bounds__(kWarps * 32) quant_append_kernel(const dsa_mla_quant_append_args a, unsigned* status) {
  constexpr int kRow = FP4 ? kRow4 : kRow8;
  const int lane = threadIdx.x & 31;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const long long t0 = (static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * TOK;
  const long long n_slots = static_cast<long long>(a.num_pages) * a.page_size;
  const __nv_bfloat16* c_in = static_cast<const __nv_bfloat16*>(a.c_kv);
  const __nv_bfloat16* r_in = static_cast<const __nv_bfloat16*>(a.k_rope);
  uint8_t* cache = static_cast<uint8_t*>(a.cache);
  long long slot[TOK];
  uint4 raw[TOK][2];
#pragma unroll
  for (int k = 0; k < TOK; ++k) {
    const long long t = t0 + k;
    slot[k] = t < a.n ? a.slot_mapping[t] : -1;
    raw[k][0] = raw[k][1] = make_uint4(0u, 0u, 0u, 0u);
    if (t < a.n) {
      const uint4* row = reinterpret_cast<const uint4*>(c_in + t * a.c_stride) + 2 * lane;
      raw[k][0] = __ldg(row);
      raw[k][1] = __ldg(row + 1);
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

  float w[16];
  if (NORM) {
    const float4* wp = reinterpret_cast<const float4*>(a.norm_weight) + 4 * lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 u = __ldg(wp + i);
      w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
    }
  }
  long long rslot = -1;
  int rE = 0;
#pragma unroll
  for (int k = 0; k < TOK; ++k) {
    if (slot[k] < 0) continue;  // the same in the whole warp
    float x[16];
    {
      float lo[8], hi[8];
      unpack_bf16(raw[k][0], lo);
      unpack_bf16(raw[k][1], hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = lo[i], x[8 + i] = hi[i];
    }
    Codes c;
    if (NORM) {
      float part[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) part[i] = x[i] * x[i];
#pragma unroll
      for (int i = 4; i < 16; ++i) part[i & 3] = fmaf(x[i], x[i], part[i & 3]);
      float ss = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float mean = ss * (1.f / kRank) + a.norm_eps;
      float inv = rsqrtf(mean);
      inv = inv < INFINITY ? fmaf(0.5f * inv, fmaf(-mean * inv, inv, 1.f), inv) : 0.f;  // (zeros without norm_eps stay zeros)
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = x[i] * (inv * w[i]);
      bool near;
      c = encode<FP4, true>(v, &near);
      const bool tiny = mean < 0x1p-90f;  // squares this small lose bits, or all
      if (__any_sync(0xffffffffu, near | tiny)) c = encode_close<FP4>(x, w, a.norm_eps, tiny);
    } else {
      c = encode<FP4, false>(x, nullptr);
    }
    uint8_t* row = cache + slot[k] * kRow;
    if (FP4) {
      reinterpret_cast<uint2*>(row)[lane] = make_uint2(c.w[0], c.w[1]);
      const int hidden = lane < 8 ? (((c.E + 128) >> lane) & 1) << 7 : 0;
      row[kScale4 + lane] = static_cast<uint8_t>(c.scale | hidden);
    } else {
      reinterpret_cast<uint4*>(row)[lane] = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
      if (lane == 0) *reinterpret_cast<uint4*>(row + kScale8) = make_uint4(__float_as_uint(pow2f(c.E)), 0u, 0u, 0u);
    }
    if (rk == k) {
      rslot = slot[k];
      rE = c.E;
    }
  }
  // RoPE: the lane's eight values are elements 8 ch .. 8 ch + 7 of its token's row
  uint4 other;  // the chunk that holds the other members of the pairs (i, i + 32)
  other.x = __shfl_xor_sync(0xffffffffu, rraw.x, 4);
  other.y = __shfl_xor_sync(0xffffffffu, rraw.y, 4);
  other.z = __shfl_xor_sync(0xffffffffu, rraw.z, 4);
  other.w = __shfl_xor_sync(0xffffffffu, rraw.w, 4);
  if (rslot < 0) return;
  float x[8], y[8], z[8];
  unpack_bf16(rraw, x);
  if (turn) {
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
      unpack_bf16(other, y);
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
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = x[i];
  }
  const float f = pow2f(-rE);  // before the rounding: a power of two, the rounded value is the same
  const uint4 res = make_uint4(pack_bf16(z[0] * f, z[1] * f), pack_bf16(z[2] * f, z[3] * f), pack_bf16(z[4] * f, z[5] * f),
                               pack_bf16(z[6] * f, z[7] * f));
  reinterpret_cast<uint4*>(cache + rslot * kRow + (FP4 ? kRope4 : kRope8))[ch] = res;
}

template <int TOK>
cudaError_t launch_append(const dsa_mla_quant_append_args& a, unsigned* status, cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(a.n) + kWarps * TOK - 1) / (kWarps * TOK));
  const bool fp4 = a.format == DSA_FP4_E2M1, norm = a.norm_weight != nullptr;
  auto* kern = fp4 ? (norm ? quant_append_kernel<true, true, TOK> : quant_append_kernel<true, false, TOK>)
                   : (norm ? quant_append_kernel<false, true, TOK> : quant_append_kernel<false, false, TOK>);
  return launch_pdl(kern, dim3(blocks), dim3(kWarps * 32), 0, s, a, status);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

int dsa_mla_quant_row_bytes(int format) { return quant::row_bytes(format); }

dsa_status dsa_mla_quant_append(const dsa_mla_quant_append_args* a, dsa_stream_t stream) {
  if (!a) return DSA_ERR_INVALID_ARGUMENT;
  if (a->n < 0 || a->page_size <= 0 || a->num_pages < 0 || a->kv_rank <= 0 || a->rope_dim < 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (a->kv_rank != quant::kRank || a->rope_dim != quant::kRope || quant::row_bytes(a->format) == 0)
    return DSA_ERR_UNSUPPORTED;
  if (a->n == 0) return DSA_OK;
  if (!a->c_kv || !a->k_rope || !a->slot_mapping || (!a->cache && a->num_pages > 0)) return DSA_ERR_INVALID_ARGUMENT;
  if ((a->rope_cos == nullptr) != (a->rope_sin == nullptr)) return DSA_ERR_INVALID_ARGUMENT;
  if (a->rope_cos && (a->rope_rows < 1 || (!a->positions && a->rope_rows < a->n))) return DSA_ERR_INVALID_ARGUMENT;
  if (a->norm_weight && !(a->norm_eps >= 0.f)) return DSA_ERR_INVALID_ARGUMENT;
  // (one token's strides lead nowhere)
  if (a->n > 1 && (a->c_stride < 0 || a->r_stride < 0 || a->c_stride % 8 != 0 || a->r_stride % 8 != 0))
    return DSA_ERR_INVALID_ARGUMENT;
  auto al = [](const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  if (!al(a->c_kv, 16) || !al(a->k_rope, 16) || !al(a->cache, 16) || !al(a->norm_weight, 16) ||
      !al(a->rope_cos, 16) || !al(a->rope_sin, 16) || !al(a->slot_mapping, 8) || !al(a->positions, 4))
    return DSA_ERR_INVALID_ARGUMENT;
  unsigned* status = device_status_ptr();
  if (!status) return DSA_ERR_CUDA;
  // Tokens a warp: more of them share the weights' loads, as long as the warps fill the SMs.  1, 2, 4 tokens a warp, us by itself:
  //   norm, 8 bits     64 rows 2.6, 3.1, 3.7    2048 5.2, 4.7, 5.2    8192 10.6, 9.8, 8.2    32768 29.7, 26.3, 22.6
  //   norm, 4 bits     64 rows 4.7, 5.2, 6.7    2048 6.8, 6.3, 7.2    8192 12.4, 10.7, 10.2  32768 32.0, 26.1, 23.7
  //   without, 8 bits  2048 2.6, 2.7, 3.1       4096 3.7, 3.1, 3.6    16384 7.2, 5.7, 5.7    32768 12.3, 9.8, 8.8
  //   without, 4 bits  2048 3.6, 3.9, 5.1       4096 4.7, 4.7, 5.7    16384 10.3, 9.7, 9.3   32768 18.4, 16.0, 16.4
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int two = a->norm_weight ? 2048 : 4096, four = a->norm_weight ? 8192 : 16384;
  const cudaError_t e = a->n >= four ? launch_append<4>(*a, status, s) : a->n >= two ? launch_append<2>(*a, status, s) : launch_append<1>(*a, status, s);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
