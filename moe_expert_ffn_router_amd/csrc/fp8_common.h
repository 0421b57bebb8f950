// Shared by the FP8 product kernels: quantisation of a 128-block to E4M3, the
// plain E4M3 MFMA, and the lookup of a row tile among the experts' segments.
// Also the debug-flag readers of the translation units outside the bf16 /
// FP4 layer path.
#pragma once

#include "moe_internal.h"

namespace moe {

typedef __attribute__((__vector_size__(8 * sizeof(int)))) int fp8x32;  // 32 E4M3 codes

constexpr int kFp8Block = 128;  // columns (and weight rows) of one scale

// D (16 x 16) = A (16 x 128) B (128 x 16) + C, E4M3 operands, unit scales.
// Lane (g, i) = (lane / 16, lane % 16) holds 32 codes of row i of A (column i
// of B); the instruction pairs equal byte positions of equal lane groups, so
// any split of the 128 codes over the groups works that is the same for both.
// C: lane (g, i) element r is C[4g + r][i].
__device__ __forceinline__ f32x4 mfma_e4m3(fp8x32 a, fp8x32 b, f32x4 c) {
  // scale operands that are the constant 0 select the instruction without scales
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// The same product on the bf16 MFMA, of codes decoded to bf16 (exact), which keeps what the
// E4M3 one drops: that adds 8 products at a time and cuts each to a multiple of 2^-13 of the
// largest.  Half its rate.  For sums that are rounded to E4M3 again: an error of 2^-13 moves
// one value in a few hundred to the next code, a step of up to 1/8 of it, and with few rows one
// such step shows in the result (120 FFNs of random sizes: largest error 1.4 times the fp32
// formula's, on the E4M3 MFMA 3.1 times; 8 tokens take 47 us both ways).
struct Decoded {
  bf16x8 v[4];
};
__device__ __forceinline__ Decoded decode_e4m3(const fp8x32& c) {
  Decoded d;
#pragma unroll
  for (int i = 0; i < 4; ++i) d.v[i] = fp8x8_to_bf16((uint32_t)c[2 * i], (uint32_t)c[2 * i + 1]);
  return d;
}
__device__ __forceinline__ f32x4 mfma_decoded(const Decoded& a, const Decoded& b, f32x4 c) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}

// Keeps a value at this point of the program: without it the compiler moves an MFMA
// down to the first use of its result, and the loop's order with it.
__device__ __forceinline__ void pin(f32x4& v) { asm volatile("" : "+v"(v)); }

// Scale of a block from the bits of its largest magnitude (an fp32 value):
// 448 = 1.75 * 2^8, so amax = 1.m * 2^q needs 2^(q-8) where 1.m <= 1.75, else
// 2^(q-7).  inv = 1 / scale (exact).  Non-finite blocks: NaN scale.
struct Fp8Scale {
  float scale, inv;
  bool finite;
};
__device__ __forceinline__ Fp8Scale fp8_block_scale(uint32_t amax_bits) {
  const int q = (int)(amax_bits >> 23);
  int b = q - ((amax_bits & 0x7fffffu) <= 0x600000u ? 8 : 7);  // biased exponent of the scale
  b = b < 1 ? 1 : b;
  b = amax_bits == 0 ? 127 : b;
  Fp8Scale s;
  s.finite = q != 255;
  s.scale = __uint_as_float(s.finite ? (uint32_t)b << 23 : 0x7fc00000u);
  s.inv = __uint_as_float((uint32_t)(254 - (s.finite ? b : 127)) << 23);
  return s;
}

// Four values of a block -> E4M3 codes in one dword.
__device__ __forceinline__ int fp8_pack4(float a, float b, float c, float d, const Fp8Scale& s) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * s.inv, b * s.inv, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c * s.inv, d * s.inv, w, true);
  return s.finite ? w : 0x7f7f7f7f;
}

// Two fp32 values -> packed bf16, nearest-even (NaN quiet): one instruction.
__device__ __forceinline__ uint32_t bf16_pack2(float a, float b) {
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// SiLU(g) * u = g * u / (1 + e^-g), with e^-g = 2^(-g log2(e)) on the hardware's 2^x and 1/x
// (one ulp each).  The exponent's rounding makes e^-g off by |g| 2^-24 relative: enough for
// a value that goes to 4 significant bits next (FFN of 4096 tokens, 8 of 64 experts of
// 2048 x 1024: 352 us, with expf and a division 374).
__device__ __forceinline__ float swiglu(float g, float u) {
  const float z = __builtin_amdgcn_exp2f(g * -1.44269504f);
  return g * __builtin_amdgcn_rcpf(1.0f + z) * u;
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Row tiles of BM rows over the experts' segments, experts in ascending order, looked up by
// one whole wave: lane l owns the experts [l * per, l * per + per) and loads their counts
// and offsets together.
struct RowTile {
  int e, row0, rows;
};
template <int BM>
struct RowTiles {
  int n[kMaxE / 64], o[kMaxE / 64], per, first, mine, upto;

  __device__ __forceinline__ int load(const int* __restrict__ counts,
                                      const int* __restrict__ offsets, int E, int lane) {
    per = (E + 63) >> 6;  // at most 16
    first = lane * per;
#pragma unroll
    for (int i = 0; i < kMaxE / 64; ++i) {
      const bool ok = i < per && first + i < E;
      n[i] = ok ? counts[first + i] : 0;
      o[i] = ok ? offsets[first + i] : 0;
    }
    mine = 0;
#pragma unroll
    for (int i = 0; i < kMaxE / 64; ++i) {
      n[i] = n[i] > 0 ? n[i] : 0;
      mine += (n[i] + BM - 1) / BM;
    }
    upto = wave_incl_scan(mine);
    return __builtin_amdgcn_readlane(upto, 63);  // tiles in all
  }

  // tile < load()'s result
  __device__ __forceinline__ RowTile at(int tile) const {
    const uint64_t owner = __ballot(tile >= upto - mine && tile < upto);
    const int ol = (int)__builtin_ctzll(owner);
    int left = tile - (upto - mine), e = first, rows = 0, row0 = 0;
#pragma unroll
    for (int i = 0; i < kMaxE / 64; ++i) {
      const int tiles = (n[i] + BM - 1) / BM;
      if (rows == 0 && left >= 0 && left < tiles) {
        e = first + i;
        rows = n[i] - left * BM;
        row0 = o[i] + left * BM;
      }
      left -= tiles;
    }
    RowTile t;
    t.e = __builtin_amdgcn_readlane(e, ol);
    const int r = __builtin_amdgcn_readlane(rows, ol);
    t.row0 = __builtin_amdgcn_readlane(row0, ol);
    t.rows = r < BM ? r : BM;
    return t;
  }
};

// Upper bound on the row tiles of A rows over E experts (host).
inline int64_t row_tiles_bound(int64_t A, int64_t E, int64_t BM) {
  const int64_t touched = A < E ? A : E;
  return (A + touched * (BM - 1)) / BM;
}

#ifdef MOE_DEBUG
uint32_t dbg_take_balance();
uint32_t dbg_take_fp8();
uint32_t dbg_take_train();
#endif

}  // namespace moe
