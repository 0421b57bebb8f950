// Products of E4M3 operands with a scale for each block of 128, and what
// feeds them: quantisation of bf16 rows, the dense / grouped product, and the
// expert FFN of FP8 records with E4M3 activations.
//
// The 16x16x128 MFMA sums one scale block (128 columns) of 16 weight rows and
// 16 activation rows; its fp32 result t enters the accumulators as
// acc += (a_scale * w_scale) * t.  The weights are the first operand, so a
// lane's four results are consecutive output columns of one activation row,
// whose scale it holds once, and the weight scale is the same for the whole
// 16-row subtile.
#include <algorithm>
#include <type_traits>

#include "fp8_common.h"
#include "lds_copy.h"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// bf16 (x) or fp32 (h) rows -> E4M3.  A thread holds 8 consecutive columns, 16 lanes
// (one DPP row) a 128-block; short blocks leave lanes without columns.
// ---------------------------------------------------------------------------
template <typename SRC>
__global__ __launch_bounds__(256) void fp8_quantize_kernel(const SRC* __restrict__ x, int T, int K,
                                                           uint8_t* __restrict__ codes,
                                                           float* __restrict__ scales) {
  const int kb = (K + kFp8Block - 1) / kFp8Block;
  const int64_t n = (int64_t)T * kb * 16;  // 8-column units, rows padded to whole blocks
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < n; u += (int64_t)gridDim.x * 256) {
    const int64_t block = u >> 4;
    const int64_t row = block / kb;
    const int b = (int)(block - row * kb);
    const int col = b * kFp8Block + (int)(u & 15) * 8;
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (col < K) {
      if constexpr (sizeof(SRC) == 2) {
        const uint4 v = *reinterpret_cast<const uint4*>(x + row * K + col);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f[2 * q] = __uint_as_float(w[q] << 16);
          f[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
        }
      } else {
        const float4* v = reinterpret_cast<const float4*>(x + row * K + col);
        const float4 lo = v[0], hi = v[1];
        f[0] = lo.x, f[1] = lo.y, f[2] = lo.z, f[3] = lo.w;
        f[4] = hi.x, f[5] = hi.y, f[6] = hi.z, f[7] = hi.w;
      }
    }
    uint32_t am = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) am = umax(am, __float_as_uint(f[q]) & 0x7fffffffu);
    am = umax(am, (uint32_t)dpp_i32<0xB1>((int)am, (int)am));
    am = umax(am, (uint32_t)dpp_i32<0x4E>((int)am, (int)am));
    am = umax(am, (uint32_t)dpp_i32<0x141>((int)am, (int)am));
    am = umax(am, (uint32_t)dpp_i32<0x140>((int)am, (int)am));
    const Fp8Scale s = fp8_block_scale(am);
    if (col < K) {
      const int w0 = fp8_pack4(f[0], f[1], f[2], f[3], s);
      const int w1 = fp8_pack4(f[4], f[5], f[6], f[7], s);
      *reinterpret_cast<uint2*>(codes + row * K + col) = uint2{(uint32_t)w0, (uint32_t)w1};
    }
    if ((u & 15) == 0) scales[block] = s.scale;
  }
}

template <typename SRC>
void launch_quantize(const SRC* x, int T, int K, uint8_t* codes, float* scales,
                     hipStream_t s) {
  const int64_t n = (int64_t)T * ((K + kFp8Block - 1) / kFp8Block) * 16;
  const int64_t blocks = (n + 255) / 256;
  fp8_quantize_kernel<<<(unsigned)(blocks < 65536 ? blocks : 65536), 256, 0, s>>>(x, T, K, codes,
                                                                                  scales);
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
struct Fp8Args {
  const uint8_t* a;      // codes [.][K]
  const float* a_scale;  // [.][kb]
  const int* row_of;     // GATED: sorted_idx (activation row of p = row_of[p] / k), else NULL
  int k;
  const uint8_t* w;  // expert record e: w + slot * w_stride
  int64_t w_stride;
  const uint8_t* ws;  // its scales: ws + slot * ws_stride
  int64_t ws_stride;
  const int* slot_of;
  const int* counts;  // NULL: dense, rows [0, M)
  const int* offsets;
  int E, M, N, K, I;  // N weight rows (gate/up: 2I)
  uint16_t* y;        // bf16 [M][N]
  float* h;           // gate/up, few rows: fp32 [M][I]
  uint8_t* hq;        // gate/up, tiles: E4M3 [M][I]
  float* hs;          // and its scales [M][I/128]
  int mt, nnb;        // tiles: row tiles (dense) and column blocks
};

// A grid has fewer than 2^32 threads.
bool grid_fits(int64_t blocks, int threads) { return blocks < ((int64_t)1 << 32) / threads; }

__device__ __forceinline__ const uint8_t* slot_base(const uint8_t* base, int64_t stride,
                                                    const Fp8Args& p, int e) {
  const int slot = p.slot_of ? dbg_clamp(p.slot_of[e], p.E, kDbgSlot) : e;
  return base + (size_t)slot * stride;
}

// Four consecutive outputs of a row, of which the first `left` exist; 8-byte aligned where
// `vec` (rows of a multiple of 4).
__device__ __forceinline__ void store4(uint16_t* dst, const f32x4& v, int left, bool vec) {
  const uint2 b = {bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3])};
  if (vec) {
    if (left > 0) *reinterpret_cast<uint2*>(dst) = b;
  } else {
    if (left > 0) dst[0] = (uint16_t)b.x;
    if (left > 1) dst[1] = (uint16_t)(b.x >> 16);
    if (left > 2) dst[2] = (uint16_t)b.y;
    if (left > 3) dst[3] = (uint16_t)(b.y >> 16);
  }
}

// Activations of the 16-row kernel: codes with their scales, or rows that it quantises as it
// reads them (bf16 x, fp32 h), which saves the quantising launch where few rows are read.
enum { kSrcCodes, kSrcBf16, kSrcF32 };

// A lane's 32 consecutive values [col, col + 32) of a row -> codes, and the scale of the
// row's 128-block, which the lanes i16, i16 + 16, i16 + 32, i16 + 48 hold together.
template <typename SRC>
struct RawRow {
  i32x4 v[sizeof(SRC) * 2];
};
template <typename SRC>
__device__ __forceinline__ void load_raw(const SRC* row, int col, int K, bool live, RawRow<SRC>& r) {
  constexpr int N = sizeof(SRC) * 2, PER = 16 / sizeof(SRC);  // 16-byte pieces, values of one
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const i32x4 zero = {0, 0, 0, 0};
    r.v[q] = live && col + q * PER < K ? *reinterpret_cast<const i32x4*>(row + col + q * PER) : zero;
  }
}
template <typename SRC>
__device__ __forceinline__ fp8x32 quantize_raw(const RawRow<SRC>& r, float& scale) {
  auto at = [&](int i) -> float {
    if constexpr (sizeof(SRC) == 2) {
      const uint32_t w = (uint32_t)r.v[i / 8][(i % 8) / 2];
      return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    } else {
      return __int_as_float(r.v[i / 4][i % 4]);
    }
  };
  uint32_t am = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) am = umax(am, __float_as_uint(at(i)) & 0x7fffffffu);
  am = umax(am, (uint32_t)__shfl_xor((int)am, 16, 64));
  am = umax(am, (uint32_t)__shfl_xor((int)am, 32, 64));
  const Fp8Scale s = fp8_block_scale(am);
  scale = s.scale;
  fp8x32 c;
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = fp8_pack4(at(4 * i), at(4 * i + 1), at(4 * i + 2), at(4 * i + 3), s);
  return c;
}

// Tiles of 16 rows, for few rows: bound by the weight bytes, which go from memory straight to
// registers, U blocks of K in flight per wave.  A wave takes NSUB subtiles of 16 weight rows
// (gate/up: half gate rows, half their up rows).  SPLIT = NW: the NW waves share the subtiles
// and split K (blocks w, w + NW, ...), their sums meet in LDS in wave order; SPLIT = 1: each
// has subtiles of its own over the whole K.
template <int SRC, bool GATED, int NSUB, int NW, int SPLIT, int U>
__global__ __launch_bounds__(64 * NW) void fp8_rows16_kernel(Fp8Args p) {
  constexpr int OUT = GATED ? NSUB / 2 : NSUB;          // output subtiles of a wave
  constexpr int COLS = OUT * 16 * (SPLIT == 1 ? NW : 1);  // output columns of a workgroup
  static_assert(SPLIT == 1 || (SPLIT == NW && NW >= OUT), "split");
  __shared__ f32x4 red[SPLIT == 1 ? 1 : NW][NSUB][64];
  const int nnb = p.nnb;
  const int tile = (int)blockIdx.x / nnb, nb = (int)blockIdx.x - tile * nnb;
  const int lane = threadIdx.x & 63, g = lane >> 4, i16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowTile t;
  if (p.counts) {
    RowTiles<16> tiles;
    if (tile >= tiles.load(p.counts, p.offsets, p.E, lane)) return;  // uniform per block
    t = tiles.at(tile);
    dbg_segment(t.row0, t.rows, p.M);
  } else {
    t.e = 0;
    t.row0 = tile * 16;
    t.rows = min(16, p.M - t.row0);
  }
  const int K = p.K, kb = (K + kFp8Block - 1) / kFp8Block;
  const uint8_t* w = slot_base(p.w, p.w_stride, p, t.e);
  const float* ws = reinterpret_cast<const float*>(slot_base(p.ws, p.ws_stride, p, t.e));
  const int n0 = nb * COLS + (SPLIT == 1 ? wave * OUT * 16 : 0);
  uint32_t wo[NSUB];
  int so[NSUB];
#pragma unroll
  for (int j = 0; j < NSUB; ++j) {
    const int base = GATED ? (j < OUT ? n0 : p.I + n0) + j % OUT * 16 : n0 + j * 16;
    wo[j] = (uint32_t)min(base + i16, p.N - 1) * (uint32_t)K;
    so[j] = min(base, p.N - 1) / kFp8Block * kb;
  }
  const bool have = i16 < t.rows;
  size_t arow = 0;
  if (have) {
    const int r = t.row0 + i16;
    arow = p.row_of ? (size_t)(dbg_clamp(p.row_of[r], p.M, kDbgSorted) / p.k) : (size_t)r;
  }
  using Raw = std::conditional_t<SRC == kSrcF32, float, uint16_t>;

  f32x4 acc[NSUB];
#pragma unroll
  for (int j = 0; j < NSUB; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const i32x4 zero = {0, 0, 0, 0};
  for (int c0 = SPLIT == 1 ? 0 : wave; c0 < kb; c0 += SPLIT * U) {
    i32x4 wf[U][NSUB][2];
    RawRow<uint8_t> af[U];
    RawRow<Raw> raw[U];
    float sa[U], sw[U][NSUB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + SPLIT * u;
      const int col = c * kFp8Block + 32 * g;  // K a multiple of 16: 16-byte units are whole
      const bool ok0 = c < kb && col < K, ok1 = c < kb && col + 16 < K;
#pragma unroll
      for (int j = 0; j < NSUB; ++j) {
        wf[u][j][0] = ok0 ? *reinterpret_cast<const i32x4*>(w + wo[j] + col) : zero;
        wf[u][j][1] = ok1 ? *reinterpret_cast<const i32x4*>(w + wo[j] + col + 16) : zero;
        sw[u][j] = c < kb ? ws[so[j] + c] : 0.0f;
      }
      if constexpr (SRC == kSrcCodes) {
        load_raw<uint8_t>(p.a + arow * K, col, K, have && c < kb, af[u]);
        sa[u] = c < kb && have ? p.a_scale[arow * kb + c] : 0.0f;
      } else {
        load_raw<Raw>(reinterpret_cast<const Raw*>(p.a) + arow * K, col, K, have && c < kb, raw[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      fp8x32 b;
      if constexpr (SRC == kSrcCodes) {
        const i32x4 x = af[u].v[0], y = af[u].v[1];
        b = fp8x32{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
      } else {
        b = quantize_raw<Raw>(raw[u], sa[u]);
      }
      Decoded bd;
      if constexpr (GATED) bd = decode_e4m3(b);
#pragma unroll
      for (int j = 0; j < NSUB; ++j) {
        const i32x4 x = wf[u][j][0], y = wf[u][j][1];
        const fp8x32 a = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
        f32x4 d = {0.f, 0.f, 0.f, 0.f};
        if constexpr (GATED) d = mfma_decoded(decode_e4m3(a), bd, d);
        else d = mfma_e4m3(a, b, d);
        const float s = sa[u] * sw[u][j];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][r] = fmaf(s, d[r], acc[j][r]);
      }
    }
  }
  // output subtile j (gate/up: from its gate and up sums) of row i16, columns 4g..4g+3
  auto put = [&](int j, const f32x4& v, const f32x4& u) {
    const int col = n0 + j * 16 + 4 * g;
    if (!have) return;
    if constexpr (GATED) {
      if (col < p.I)
        *reinterpret_cast<float4*>(p.h + (size_t)(t.row0 + i16) * p.I + col) =
            float4{swiglu(v[0], u[0]), swiglu(v[1], u[1]), swiglu(v[2], u[2]), swiglu(v[3], u[3])};
    } else {
      store4(p.y + (size_t)(t.row0 + i16) * p.N + col, v, p.N - col, p.N % 4 == 0);
    }
  };
  if constexpr (SPLIT == 1) {
#pragma unroll
    for (int j = 0; j < OUT; ++j) put(j, acc[j], acc[GATED ? j + OUT : j]);
  } else {
#pragma unroll
    for (int j = 0; j < NSUB; ++j) red[wave][j][lane] = acc[j];
    __syncthreads();
    if (wave >= OUT) return;
    auto total = [&](int j) {
      f32x4 v = red[0][j][lane];
#pragma unroll
      for (int q = 1; q < NW; ++q) {
        const f32x4 x = red[q][j][lane];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] += x[r];
      }
      return v;
    };
    const f32x4 v = total(wave);
    put(wave, v, GATED ? total(wave + OUT) : v);
  }
}

// ---------------------------------------------------------------------------
// Tiles of BM rows x BN weight rows on WM x WN waves, K in blocks of 128.
// Both operands are copied from memory straight into LDS, two blocks deep; the
// rows' scales likewise, four blocks at a time.  A wave owns MI x NJ subtiles of
// 16 x 16: it keeps the block's NJ weight fragments in registers and streams its
// MI activation fragments past them; each MFMA starts from zero and its result
// is folded into the accumulators two MFMAs later, so the fold's multiply-adds
// run under the MFMAs between.
//   The copies bound this kernel (a block's 64 KB take as long to arrive as to
// multiply), so they never stop: a stage is refilled piece by piece as it is
// read rather than as a whole at its end - the weights once every wave holds its
// fragments (row subtile 1), the first half of each wave's rows at subtile MI/2,
// the second at the last - and the waits leave the pieces issued since
// outstanding.  Every piece has at least one block's time to arrive.  A
// workgroup owns its compute unit (LDS, registers) and works through a list of
// tiles as one sequence of blocks: the next tile's first two blocks are copied
// during the last two of the current one, so its look-up, launch and first loads
// hide behind MFMAs and the epilogue.
// ---------------------------------------------------------------------------
template <int BM, int BN>
struct TileStage {
  uint8_t a[BM * 128];  // [row][128 codes], 16-byte unit u stored at u ^ a_swz(row)
  uint8_t b[BN * 128];  // weights, same layout
};

constexpr int kListTiles = 32;  // tiles of one workgroup at most
constexpr int kXcds = 8, kXcdCus = 32;

template <int BM, int BN, int WN, bool GATED>
struct TileLds {
  TileStage<BM, BN> st[2];
  __attribute__((aligned(16))) float sc[3][BM * 4];  // rows' scales: [group of 4 blocks % 3][row][4]
  float wsc[2][2][65536 / kFp8Block];  // [tile % 2]: its two rows of weight scales
  __attribute__((aligned(16))) int list[kListTiles][4];  // slot, first row, rows, column block
  int src[BM];  // gathered activation rows of the next tile
  float row_max[GATED ? WN : 1][GATED ? BM : 1];  // largest |h| per wave column
};

// m-tiles that consecutive workgroups of one XCD share weights over
constexpr int kPanel = 4;

// Tile v of mt x nnb: in panels of kPanel row tiles that go column block by column block.
__device__ __forceinline__ void panel_tile(int v, int mt, int nnb, int& tile, int& nb) {
  const int panel = v / (kPanel * nnb), r = v - panel * (kPanel * nnb);
  const int rows = min(kPanel, mt - panel * kPanel);
  nb = r / rows;
  tile = panel * kPanel + r - nb * rows;
}

// Waits for this wave's LDS accesses, then a barrier that no memory access moves across.
#define MOE_LDS_SYNC()                                                   \
  do {                                                                   \
    __builtin_amdgcn_s_waitcnt(::moe::waitcnt_vm_lgkm0(63));             \
    asm volatile("s_barrier" ::: "memory");                              \
  } while (0)

// Needs at least two blocks of K; QUAD: at least four.
template <int BM, int BN, int WM, int WN, bool GATED, bool QUAD>
__global__ __launch_bounds__(64 * WM * WN) void fp8_tile_kernel(Fp8Args p) {
  constexpr int NW = WM * WN, MI = BM / WM / 16, NJ = BN / WN / 16;
  constexpr int COLS = GATED ? BN / 2 : BN;    // output columns
  constexpr int CPA = BM / 8 / NW, CPB = BN / 8 / NW;  // 1 KB copies (8 rows) per wave
  constexpr int RW = BM / WM, HALF = RW / 2;           // rows of a wave row, and of half of one
  static_assert(NJ == 4 && BM % 64 == 0 && BM / 64 <= NW && MI > 2 && CPA / 2 <= NJ, "wave shape");
  static_assert(!GATED || COLS == kFp8Block, "gate/up: one scale block of h per tile");
  __shared__ TileLds<BM, BN, WN, GATED> lds;
  auto& st = lds.st;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int mh = wave / WN, nh = wave % WN;
  const int K = p.K, kb = (K + kFp8Block - 1) / kFp8Block;

  // This workgroup's tiles.  Hardware block b runs on XCD b % 8: the tiles are cut into
  // eight contiguous ranges (grouped products know their number here only; the host sized the
  // grid from a bound).  An XCD's workgroups take its range in rounds, first the tiles of over
  // BM / 2 rows, then the cheaper ones (of half the rows: about 2/3 of the time), every other round
  // in reverse order, so that the last round's work falls on those with least so far (16384 rows
  // over 64 experts of 2048 x 4096: 240 us, 249 with the range taken in order; the FFN of 32768
  // rows 338 against 349).
  int mine;
  {
    const int x = (int)blockIdx.x % kXcds, i0 = (int)blockIdx.x / kXcds;
    const int W = (int)gridDim.x / kXcds;
    // scratch in the stages, which hold nothing yet
    int* before = reinterpret_cast<int*>(&st);  // [E + 1]: row tiles before each expert
    int* rows_of = before + kMaxE + 1;          // [E]
    int* wave_big = rows_of + kMaxE;            // [NW], then the number of big tiles
    int* n_big = wave_big + NW;
    if (tid == 0) *n_big = 0;
    if (p.counts && wave == 0) {
      RowTiles<BM> t;
      const int total = t.load(p.counts, p.offsets, p.E, lane);
      int run = t.upto - t.mine;
#pragma unroll
      for (int i = 0; i < kMaxE / 64; ++i)
        if (i < t.per && t.first + i < p.E) {
          before[t.first + i] = run;
          rows_of[t.first + i] = t.n[i];
          run += (t.n[i] + BM - 1) / BM;
        }
      if (lane == 0) before[p.E] = total;
    }
    __syncthreads();
    const int mt = p.counts ? before[p.E] : p.mt;
    const int G = mt * p.nnb, per = (G + kXcds - 1) / kXcds;
    const int n = min(per, G - x * per);
    // round r of this workgroup is position r * W + (r even ? i0 : W - 1 - i0) of the range
    const int whole_rounds = n / W;
    mine = n <= 0 ? 0 : whole_rounds + ((whole_rounds & 1 ? W - 1 - i0 : i0) < n - whole_rounds * W);
    mine = __builtin_amdgcn_readfirstlane(min(mine, kListTiles));
    if (mine == 0) return;  // uniform
    // tile i of the range: expert, its tile and column block; rows in the tile
    auto look_up = [&](int i, int& e, int& sub, int& nb) {
      int tile;
      panel_tile(x * per + i, mt, p.nnb, tile, nb);
      if (!p.counts) {
        e = 0;
        sub = tile;
        return min(BM, p.M - tile * BM);
      }
      int lo = 0, hi = p.E - 1;  // the last expert with before[e] <= tile
      while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (before[m] <= tile) lo = m;
        else hi = m - 1;
      }
      e = lo;
      sub = tile - before[e];
      return min(BM, rows_of[e] - sub * BM);
    };
    for (int i = tid; i < n; i += 64 * NW) {
      int e, sub, nb;
      if (look_up(i, e, sub, nb) > BM / 2) atomicAdd(n_big, 1);
    }
    __syncthreads();
    const int big = *n_big;
    int seen = 0;  // big tiles before this turn
    for (int i1 = 0; i1 < n; i1 += 64 * NW) {
      const int i = i1 + tid;
      int e = 0, sub = 0, nb = 0, rows = 0;
      if (i < n) rows = look_up(i, e, sub, nb);
      const uint64_t b = __ballot(rows > BM / 2);
      if (lane == 0) wave_big[wave] = __popcll(b);
      __syncthreads();
      int at = seen + (int)__popcll(b & ((1ull << lane) - 1));
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        at += w < wave ? wave_big[w] : 0;
        seen += wave_big[w];
      }
      if (i < n) {
        const int q = rows > BM / 2 ? at : big + i - at;  // position in the order of the rounds
        const int r = q / W, c = q - r * W;
        if ((r & 1 ? W - 1 - c : c) == i0 && r < kListTiles) {
          int row0 = p.counts ? p.offsets[e] + sub * BM : sub * BM;
          dbg_segment(row0, rows, p.M);
          const int slot = p.slot_of ? dbg_clamp(p.slot_of[e], p.E, kDbgSlot) : e;
          *reinterpret_cast<i32x4*>(lds.list[r]) = i32x4{slot, row0, rows, nb};
        }
      }
      __syncthreads();
    }
  }
  auto entry = [&](int q, int f) { return __builtin_amdgcn_readfirstlane(lds.list[q][f]); };

  // -- copies -----------------------------------------------------------------------
  // Cursor: tile cr, block cc, with the tile's addresses.
  int cr = 0, cc = 0, cgrp = 0;  // cgrp: scale group counter % 3
  const uint8_t *ab, *sb, *wb;
  uint32_t ao[CPA], wo[CPB], so = 0;
  // The lane's part of the addresses is recomputed per tile: hoisted out of the loop it would
  // cost registers that the accumulators need.
  auto fresh_lane = [&]() {
    int l = lane;
    asm volatile("" : "+v"(l));
    return l;
  };
  // local row that copy q of this wave starts at: the first CPA / 2 cover the first halves of
  // the waves' row groups, the others the second halves
  auto a_row = [&](int q) {
    const int x = (wave * (CPA / 2) + q % (CPA / 2)) * 8;
    return x / HALF * RW + x % HALF + (q < CPA / 2 ? 0 : HALF);
  };
  // the activation rows of tile q, gathered ones through LDS (issue_src)
  auto issue_src = [&](int q) {
    if (wave < BM / 64) {
      const int r = min(wave * 64 + lane, max(entry(q, 2), 1) - 1);
      dma4(reinterpret_cast<const uint8_t*>(p.row_of + entry(q, 1)), (uint32_t)r * 4u,
           lds.src + wave * 64);
    }
  };
  auto point_at = [&](int q) {
    const int slot = entry(q, 0), row0 = entry(q, 1), rows = entry(q, 2), nb = entry(q, 3);
    const int ln = fresh_lane();
    const uint32_t unit = (uint32_t)(ln & 7);
    // rows past the tile read its last one
    auto source = [&](int lr) -> uint32_t {
      if (p.row_of) return (uint32_t)(dbg_clamp(lds.src[lr], p.M, kDbgSorted) / p.k);
      return (uint32_t)min(lr, max(rows, 1) - 1);
    };
    ab = p.row_of ? p.a : p.a + (size_t)row0 * K;
    sb = reinterpret_cast<const uint8_t*>(p.row_of ? p.a_scale : p.a_scale + (size_t)row0 * kb);
    wb = p.w + (size_t)slot * p.w_stride + (GATED ? 0 : (size_t)nb * BN * K);
#pragma unroll
    for (int i = 0; i < CPA; ++i) {
      const int lr = a_row(i) + (ln >> 3);
      ao[i] = source(lr) * (uint32_t)K + ((unit ^ a_swz(lr)) * 16);
    }
#pragma unroll
    for (int i = 0; i < CPB; ++i) {
      const int lr = (wave * CPB + i) * 8 + (ln >> 3);
      int wr;
      if constexpr (GATED) {  // a wave's 64 weight rows: 32 gate rows, then their up rows
        const int col = nb * COLS + (lr >> 6) * 32 + (lr & 31);
        wr = (lr & 32) ? p.I + col : col;
      } else {
        wr = min(lr, p.N - 1 - nb * BN);
      }
      wo[i] = (uint32_t)wr * (uint32_t)K + ((unit ^ a_swz(lr)) * 16);
    }
    if (wave < BM / 64) so = source(wave * 64 + ln) * (uint32_t)kb * 4u;
    // the tile's two rows of weight scales (gate/up: the gate and the up block)
    const int last = (p.N - 1) / kFp8Block;
    const int b0 = GATED ? nb : min(nb * (BN / kFp8Block), last);
    const int b1 = GATED ? p.I / kFp8Block + nb : min(nb * (BN / kFp8Block) + 1, last);
    const uint8_t* ws = p.ws + (size_t)slot * p.ws_stride;
    for (int i = wave; i < 2 * ((kb + 63) >> 6); i += NW)
      dma4(ws + (size_t)(i & 1 ? b1 : b0) * kb * 4,
           (uint32_t)min((i >> 1) * 64 + ln, kb - 1) * 4u, &lds.wsc[q & 1][i & 1][(i >> 1) * 64]);
  };
  // a short last block: units past K re-read its first
  auto back = [&](int row) -> uint32_t {
    const int ln = fresh_lane();
    const uint32_t u = (uint32_t)((ln & 7) ^ a_swz(row + (ln >> 3))) * 16;
    return u < (uint32_t)(K % kFp8Block) ? 0u : u;
  };
  auto is_short = [&](int c) { return c + 1 == kb && K % kFp8Block != 0; };
  // copies [q0, q1) of the cursor's block into stage s
  auto issue_a = [&](int s, int q0, int q1) {
    const uint8_t* src = ab + (size_t)cc * kFp8Block;
    const bool cut = is_short(cc);
#pragma unroll
    for (int q = q0; q < q1; ++q)
      dma16(src, cut ? ao[q] - back(a_row(q)) : ao[q], st[s].a + a_row(q) * 128);
  };
  auto issue_b = [&](int s, int q0, int q1) {
    uint8_t* dst = st[s].b + wave * CPB * 1024;
    const uint8_t* src = wb + (size_t)cc * kFp8Block;
    const bool cut = is_short(cc);
#pragma unroll
    for (int q = q0; q < q1; ++q)
      dma16(src, cut ? wo[q] - back((wave * CPB + q) * 8) : wo[q], dst + q * 1024);
  };
  // The rows' scales in groups of four blocks, the last one ending with K (fewer than four
  // blocks in all: one by one).  Three groups may be in use at once, where the middle one is
  // a single block.
  constexpr int PER = QUAD ? 4 : 1;
  auto opens = [&](int c) { return !QUAD || (c & 3) == 0; };
  auto s_first = [&](int c) { return QUAD ? min(c & ~3, kb - 4) : c; };
  auto next3 = [](int v) { return v == 2 ? 0 : v + 1; };
  auto issue_s = [&]() {
    if (wave >= BM / 64) return;
    float* dst = lds.sc[cgrp] + wave * 64 * PER;
    const uint32_t off = so + (uint32_t)s_first(cc) * 4u;
    if (QUAD) dma16(sb, off, dst);
    else dma4(sb, off, dst);
  };
  // Moves the cursor on by one block; true where that opens a tile.  Behind the last tile it
  // stays: the loop's last two turns copy a block that nobody reads, rather than carry
  // branches through all the others.
  auto advance = [&]() {
    if (cc + 1 == kb && cr + 1 == mine) return false;
    const bool fresh = cc + 1 == kb;
    cc = fresh ? 0 : cc + 1;
    cr += fresh;
    if (opens(cc)) cgrp = next3(cgrp);
    return fresh;
  };

  // -- compute ----------------------------------------------------------------------
  // A row's swizzle depends on its low 4 bits only: one address per operand and unit, the
  // subtiles at constant offsets.
  auto frag = [&](const uint8_t* base, int o0, int o1) {
    const i32x4 x = *reinterpret_cast<const i32x4*>(base + o0);
    const i32x4 y = *reinterpret_cast<const i32x4*>(base + o1);
    return fp8x32{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
  };
  const int r0 = mh * RW + l16, rb = nh * (BN / WN) + l16;
  const int u0 = ((2 * g) ^ a_swz(l16)) * 16, u1 = ((2 * g + 1) ^ a_swz(l16)) * 16;
  auto frag_a = [&](int s, int i) {
    return frag(st[s].a + i * 2048, r0 * 128 + u0, r0 * 128 + u1);
  };
  auto frag_b = [&](int s, int j) {
    return frag(st[s].b + j * 2048, rb * 128 + u0, rb * 128 + u1);
  };
  auto scale_of = [&](int grp, int c, int i) {
    return *(lds.sc[grp] + (c - s_first(c)) + r0 * PER + i * 16 * PER);
  };
  // Zeros past K in a short last block: once its copies have landed, before it is read.
  auto whole = [&](int s, int c) {
    if (!is_short(c)) return;
    const int z0 = K % kFp8Block / 16, nz = 8 - z0;
    for (int i = tid; i < (BM + BN) * nz; i += 64 * NW) {
      const int r = i / nz, u = z0 + i - r * nz, lr = r < BM ? r : r - BM;
      *reinterpret_cast<i32x4*>((r < BM ? st[s].a : st[s].b) + lr * 128 + ((u ^ a_swz(lr)) * 16)) =
          i32x4{0, 0, 0, 0};
    }
    MOE_LDS_SYNC();
  };

  // The first two blocks.
  if (p.row_of) {
    issue_src(0);
    MOE_DMA_SYNC(0);
  }
  point_at(0);
  issue_s();
  issue_b(0, 0, CPB);
  issue_a(0, 0, CPA);
  advance();  // kb >= 2: the same tile
  if (opens(cc)) issue_s();
  issue_b(1, 0, CPB);
  issue_a(1, 0, CPA);
  MOE_DMA_SYNC(CPA + CPB);
  if (p.row_of && mine > 1) {
    issue_src(1);
    // Two blocks of K: the first turn opens tile 1 and reads its rows with no landed() before
    // that (of three and more, the first turn's covers this copy; of later tiles' copies, the
    // second turn's of the tile before).
    if (kb == 2) MOE_DMA_SYNC(0);
  }
  whole(0, 0);

  f32x4 acc[MI][NJ], d[2];  // d: the last two results, not folded in yet
  fp8x32 bf[NJ], af;
  float sa;
  const int wrow = GATED ? 0 : nh * (BN / WN) / kFp8Block;
  int s = 0, grp = 0;  // stage and scale group of the block being multiplied
  // its weight and first activation fragments
  auto first_frags = [&](int c) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) bf[j] = frag_b(s, j);
    af = frag_a(s, 0);
    sa = scale_of(grp, c, 0);
  };
  first_frags(0);
  // Every wave has read what the next copies overwrite (the waits on this wave's own LDS reads
  // come before its barrier): the weights' place, the first and the second halves of the rows.
  // At the second, the next block has landed; the one behind it may still be on its way.
  auto free_b = [&](bool fresh) {
    MOE_LDS_SYNC();
    if (fresh) point_at(cr);
    if (opens(cc)) issue_s();
  };
  auto free_a = [&](bool fresh) {
    MOE_LDS_SYNC();
    if (fresh && p.row_of && cr + 1 < mine) issue_src(cr + 1);
  };
  auto landed = [&](int cn) {
    MOE_DMA_SYNC(CPB + CPA / 2);
    whole(s ^ 1, cn);
  };
  for (int r = 0; r < mine; ++r) {
    const int rows = entry(r, 2), row0 = entry(r, 1), nb = entry(r, 3);
    if (mh * RW >= rows) {  // no rows for this wave: its share of the copies and the barriers
      for (int c = 0; c < kb; ++c) {
        const int cn = c + 1 == kb ? 0 : c + 1;
        const bool fresh = advance();
        free_b(fresh);
        issue_b(s, 0, CPB);
        free_a(fresh);
        issue_a(s, 0, CPA / 2);
        landed(cn);
        issue_a(s, CPA / 2, CPA);
        s ^= 1;
        if (opens(cn)) grp = next3(grp);
      }
      if (GATED) MOE_LDS_SYNC();  // the other waves' exchange of row maxima
      first_frags(0);
      continue;
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    d[0] = d[1] = f32x4{0.f, 0.f, 0.f, 0.f};
    float w0 = lds.wsc[r & 1][wrow][0], w1 = GATED ? lds.wsc[r & 1][1][0] : 0.f;
    float s1 = 0.f;  // scale of the previous row subtile's last two results
    for (int c = 0; c < kb; ++c) {
      const int cn = c + 1 == kb ? 0 : c + 1;
      const int gn = opens(cn) ? next3(grp) : grp;
      const float n0 = lds.wsc[r & 1][wrow][cn], n1 = GATED ? lds.wsc[r & 1][1][cn] : 0.f;
      const bool fresh = advance();
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const fp8x32 a = af;
        const float f0 = sa * w0, f1 = GATED ? sa * w1 : f0;
        if (i == 1) free_b(fresh);
        if (i == MI / 2) free_a(fresh);
        if (i + 1 < MI) {
          af = frag_a(s, i + 1);
          sa = scale_of(grp, c, i + 1);
        } else {
          landed(cn);
          af = frag_a(s ^ 1, 0);
          sa = scale_of(gn, cn, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          // the result of two MFMAs ago
          f32x4& o = j >= 2 ? acc[i][j - 2] : acc[i == 0 ? MI - 1 : i - 1][j + 2];
          const float f = j >= 2 ? f0 : s1;
#pragma unroll
          for (int q = 0; q < 4; ++q) o[q] = fmaf(f, d[j & 1][q], o[q]);
          pin(o);
          d[j & 1] = mfma_e4m3(bf[j], a, f32x4{0.f, 0.f, 0.f, 0.f});
          pin(d[j & 1]);
          if (i + 1 == MI) bf[j] = frag_b(s ^ 1, j);
          // the freed pieces' copies, spread over the MFMAs
          if (i == 1) issue_b(s, j * CPB / NJ, (j + 1) * CPB / NJ);
          if (i == MI / 2 && j < CPA / 2) issue_a(s, j, j + 1);
          if (i + 1 == MI && j < CPA / 2) issue_a(s, CPA / 2 + j, CPA / 2 + j + 1);
          __builtin_amdgcn_sched_barrier(0);
        }
        s1 = f1;
      }
      w0 = n0;
      w1 = n1;
      s ^= 1;
      grp = gn;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[MI - 1][j + 2][q] = fmaf(s1, d[j][q], acc[MI - 1][j + 2][q]);
    // acc[i][j][q]: row er + 16i, weight row nh*64 + 16j + 4eg + q of the tile
    const int el = fresh_lane(), eg = el >> 4, er = mh * RW + (el & 15);
    if constexpr (GATED) {
      // h in place of the gate sums; its largest magnitude per row over the waves' columns
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            acc[i][j][q] = swiglu(acc[i][j][q], acc[i][j + 2][q]);
            m = umax(m, __float_as_uint(acc[i][j][q]) & 0x7fffffffu);
          }
        m = umax(m, (uint32_t)__shfl_xor((int)m, 16, 64));
        m = umax(m, (uint32_t)__shfl_xor((int)m, 32, 64));
        if (eg == 0) lds.row_max[nh][er + i * 16] = __uint_as_float(m);
      }
      MOE_LDS_SYNC();
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < WN; ++q) m = umax(m, __float_as_uint(lds.row_max[q][er + i * 16]));
        const Fp8Scale sc = fp8_block_scale(m);
        if (er + i * 16 < rows) {
          const size_t row = (size_t)(row0 + er + i * 16);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            *reinterpret_cast<int*>(p.hq + row * p.I + nb * COLS + nh * 32 + j * 16 + 4 * eg) =
                fp8_pack4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3], sc);
          if (nh == 0 && eg == 0) p.hs[row * (p.I / kFp8Block) + nb] = sc.scale;
        }
      }
    } else {
      const int col0 = nb * BN + nh * (BN / WN) + 4 * eg;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if (er + i * 16 >= rows) continue;
        uint16_t* dst = p.y + (size_t)(row0 + er + i * 16) * p.N + col0;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          store4(dst + j * 16, acc[i][j], p.N - col0 - j * 16, p.N % 4 == 0);
      }
    }
  }
  MOE_DMA_SYNC(0);  // copies still on their way into this workgroup's LDS
}

template <int BM, int BN, int WM, int WN, bool GATED>
int launch_tiles(Fp8Args p, hipStream_t s, const char* who) {
  constexpr int COLS = GATED ? BN / 2 : BN;
  p.nnb = ((GATED ? p.I : p.N) + COLS - 1) / COLS;
  const int64_t mt = p.counts ? row_tiles_bound(p.M, p.E, BM) : ((int64_t)p.M + BM - 1) / BM;
  const int64_t per = (mt * p.nnb + kXcds - 1) / kXcds;  // tiles of an XCD
  // one workgroup per compute unit, more where its list would overflow
  int64_t W = per < kXcdCus ? per : kXcdCus;
  if (W * kListTiles < per) W = (per + kListTiles - 1) / kListTiles;
  if (mt * p.nnb > ((int64_t)1 << 31) - 1)
    return set_error(MOE_ERR_UNSUPPORTED, "%s: too many tiles", who);
  p.mt = (int)mt;
  const unsigned grid = (unsigned)(W * kXcds);
  if (p.K > 3 * kFp8Block)
    fp8_tile_kernel<BM, BN, WM, WN, GATED, true><<<grid, 64 * WM * WN, 0, s>>>(p);
  else
    fp8_tile_kernel<BM, BN, WM, WN, GATED, false><<<grid, 64 * WM * WN, 0, s>>>(p);
  return check_launch(who);
}

// ---------------------------------------------------------------------------
// Smaller tiles for products that cannot fill the chip with 256-row ones (few
// rows per expert, few tiles): BM x BN on WM x WN waves over a ring of stages
// of one K block each, S - 1 blocks in flight, one barrier per block.  Bound by
// the bytes it can keep in flight (weights of experts with few rows) or by the
// blocks' latency (small dense products).  Gate/up: on the bf16 MFMA, as few values of h share
// the cost of a rounding that moved (FFN of 64 experts of 2048 x 1024, 16 rows each: 105 us, on
// the E4M3 MFMA 99).
// ---------------------------------------------------------------------------
template <int BM, int BN, int WN, int S, bool GATED>
struct RingLds {
  TileStage<BM, BN> st[S];
  float sc[S][BM];  // the rows' scales
  float wsc[2][65536 / kFp8Block];
  float row_max[GATED ? WN : 1][GATED ? BM : 1];
};

template <int BM, int BN, int WM, int WN, int S, bool GATED>
__global__ __launch_bounds__(64 * WM * WN) void fp8_ring_kernel(Fp8Args p) {
  constexpr int NW = WM * WN, MI = BM / WM / 16, NJ = BN / WN / 16, RW = BM / WM, CW = BN / WN;
  constexpr int COLS = GATED ? BN / 2 : BN;
  constexpr int CPA = BM / 8 / NW, CPB = BN / 8 / NW;  // 1 KB copies (8 rows) per wave
  constexpr int COPIES = CPA + CPB + 1;                // per wave and block
  static_assert(BM == 64 && (NJ == 4 || !GATED) && S >= 3 && S <= 4, "ring shape");
  static_assert(!GATED || COLS == kFp8Block, "gate/up: one scale block of h per tile");
  __shared__ RingLds<BM, BN, WN, S, GATED> lds;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int mh = wave / WN, nh = wave % WN;
  const int K = p.K, kb = (K + kFp8Block - 1) / kFp8Block;

  // Hardware block b runs on XCD b % 8: the tiles are cut into eight contiguous ranges (grouped
  // products know their number here only; the grid was sized from a bound)
  RowTile t;
  int nb;
  {
    RowTiles<BM> tiles;
    const int mt = p.counts ? tiles.load(p.counts, p.offsets, p.E, lane) : p.mt;
    const int G = mt * p.nnb, per = (G + kXcds - 1) / kXcds;
    const int i = (int)blockIdx.x / kXcds, v = (int)blockIdx.x % kXcds * per + i;
    if (i >= per || v >= G) return;  // uniform per block
    int tile;
    panel_tile(v, mt, p.nnb, tile, nb);
    if (p.counts) {
      t = tiles.at(tile);
      dbg_segment(t.row0, t.rows, p.M);
      if (t.rows <= 0) return;
    } else {
      t.e = 0;
      t.row0 = tile * BM;
      t.rows = min(BM, p.M - t.row0);
    }
  }
  const int row0 = __builtin_amdgcn_readfirstlane(t.row0);
  const int rows = __builtin_amdgcn_readfirstlane(t.rows);
  const int e = __builtin_amdgcn_readfirstlane(t.e);
  const uint8_t* w = slot_base(p.w, p.w_stride, p, e);
  const float* ws = reinterpret_cast<const float*>(slot_base(p.ws, p.ws_stride, p, e));
  // rows past the tile read its last one
  auto source = [&](int lr) -> uint32_t {
    const int r = min(lr, rows - 1);
    if (p.row_of) return (uint32_t)(dbg_clamp(p.row_of[row0 + r], p.M, kDbgSorted) / p.k);
    return (uint32_t)r;
  };
  const uint8_t* ab = p.row_of ? p.a : p.a + (size_t)row0 * K;
  const uint8_t* sb = reinterpret_cast<const uint8_t*>(p.row_of ? p.a_scale
                                                                : p.a_scale + (size_t)row0 * kb);
  const uint8_t* wb = GATED ? w : w + (size_t)nb * BN * K;
  const uint32_t unit = (uint32_t)(lane & 7);
  uint32_t ao[CPA], wo[CPB];
#pragma unroll
  for (int q = 0; q < CPA; ++q) {
    const int lr = (wave * CPA + q) * 8 + (lane >> 3);
    ao[q] = source(lr) * (uint32_t)K + ((unit ^ a_swz(lr)) * 16);
  }
#pragma unroll
  for (int q = 0; q < CPB; ++q) {
    const int lr = (wave * CPB + q) * 8 + (lane >> 3);
    int wr;
    if constexpr (GATED) {  // a wave's 64 weight rows: 32 gate rows, then their up rows
      const int col = nb * COLS + (lr >> 6) * 32 + (lr & 31);
      wr = (lr & 32) ? p.I + col : col;
    } else {
      wr = min(lr, p.N - 1 - nb * BN);
    }
    wo[q] = (uint32_t)wr * (uint32_t)K + ((unit ^ a_swz(lr)) * 16);
  }
  const uint32_t so = source(lane) * (uint32_t)kb * 4u;
  {  // the tile's weight scales (gate/up: the gate and the up block)
    const int last = (p.N - 1) / kFp8Block;
    const int b0 = GATED ? nb : min(nb * BN / kFp8Block, last);
    const int b1 = GATED ? p.I / kFp8Block + nb : min(nb * BN / kFp8Block + 1, last);
    for (int i = tid; i < kb; i += 64 * NW) {
      lds.wsc[0][i] = ws[b0 * kb + i];
      lds.wsc[1][i] = ws[b1 * kb + i];
    }
    __syncthreads();
  }
  // a short last block: units past K re-read its first
  auto back = [&](int lr) -> uint32_t {
    const uint32_t u = (unit ^ a_swz(lr)) * 16;
    return u < (uint32_t)(K % kFp8Block) ? 0u : u;
  };
  auto issue = [&](int c, int s) {
    const bool cut = c + 1 == kb && K % kFp8Block != 0;
    const uint8_t* as = ab + (size_t)c * kFp8Block;
    const uint8_t* bs = wb + (size_t)c * kFp8Block;
#pragma unroll
    for (int q = 0; q < CPB; ++q) {
      const int n = wave * CPB + q;
      dma16(bs, cut ? wo[q] - back(n * 8 + (lane >> 3)) : wo[q], lds.st[s].b + n * 1024);
    }
#pragma unroll
    for (int q = 0; q < CPA; ++q) {
      const int n = wave * CPA + q;
      dma16(as, cut ? ao[q] - back(n * 8 + (lane >> 3)) : ao[q], lds.st[s].a + n * 1024);
    }
    dma4(sb, so + (uint32_t)c * 4u, lds.sc[s]);  // every wave the same 64: equal waits for all
  };

  const int r0 = mh * RW + l16, rb = nh * CW + l16;
  const int u0 = ((2 * g) ^ a_swz(l16)) * 16, u1 = ((2 * g + 1) ^ a_swz(l16)) * 16;
  auto frag = [&](const uint8_t* base, int r) {
    const i32x4 x = *reinterpret_cast<const i32x4*>(base + r * 128 + u0);
    const i32x4 y = *reinterpret_cast<const i32x4*>(base + r * 128 + u1);
    return fp8x32{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
  };
  const float* wsw = lds.wsc[GATED ? 0 : nh * CW / kFp8Block];
  f32x4 acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int c = 0; c < S - 1 && c < kb; ++c) issue(c, c);
  for (int c = 0, s = 0; c < kb; ++c, s = s + 1 == S ? 0 : s + 1) {
    // block c has landed, the blocks issued since may be on their way; every wave is done with
    // block c - 1, whose stage the next copies take
    const int behind = min(S - 2, kb - 1 - c);
    if (behind == 2) MOE_DMA_SYNC(2 * COPIES);
    else if (behind == 1) MOE_DMA_SYNC(COPIES);
    else MOE_DMA_SYNC(0);
    if (c + S - 1 < kb) issue(c + S - 1, s == 0 ? S - 1 : s - 1);
    TileStage<BM, BN>& T = lds.st[s];
    if (c + 1 == kb && K % kFp8Block) {  // zeros past K in the short last block
      const int z0 = K % kFp8Block / 16, nz = 8 - z0;
      for (int i = tid; i < (BM + BN) * nz; i += 64 * NW) {
        const int r = i / nz, u = z0 + i - r * nz, lr = r < BM ? r : r - BM;
        *reinterpret_cast<i32x4*>((r < BM ? T.a : T.b) + lr * 128 + ((u ^ a_swz(lr)) * 16)) =
            i32x4{0, 0, 0, 0};
      }
      MOE_LDS_SYNC();
    }
    const float w0 = wsw[c], w1 = GATED ? lds.wsc[1][c] : 0.f;
    using Frag = std::conditional_t<GATED, Decoded, fp8x32>;
    auto operand = [&](const uint8_t* base, int r) -> Frag {
      if constexpr (GATED) return decode_e4m3(frag(base, r));
      else return frag(base, r);
    };
    Frag bf[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) bf[j] = operand(T.b, rb + j * 16);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const Frag af = operand(T.a, r0 + i * 16);
      const float sa = lds.sc[s][r0 + i * 16];
      const float f0 = sa * w0, f1 = GATED ? sa * w1 : f0;
      f32x4 d[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        d[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (GATED) d[j] = mfma_decoded(bf[j], af, d[j]);
        else d[j] = mfma_e4m3(bf[j], af, d[j]);
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[i][j][q] = fmaf(GATED && j >= NJ / 2 ? f1 : f0, d[j][q], acc[i][j][q]);
    }
  }
  // acc[i][j][q]: row r0 + 16i, weight row nh*CW + 16j + 4g + q of the tile
  if constexpr (GATED) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          acc[i][j][q] = swiglu(acc[i][j][q], acc[i][j + 2][q]);
          m = umax(m, __float_as_uint(acc[i][j][q]) & 0x7fffffffu);
        }
      m = umax(m, (uint32_t)__shfl_xor((int)m, 16, 64));
      m = umax(m, (uint32_t)__shfl_xor((int)m, 32, 64));
      if (g == 0) lds.row_max[nh][r0 + i * 16] = __uint_as_float(m);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int q = 0; q < WN; ++q) m = umax(m, __float_as_uint(lds.row_max[q][r0 + i * 16]));
      const Fp8Scale sc = fp8_block_scale(m);
      if (r0 + i * 16 < rows) {
        const size_t row = (size_t)(row0 + r0 + i * 16);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<int*>(p.hq + row * p.I + nb * COLS + nh * 32 + j * 16 + 4 * g) =
              fp8_pack4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3], sc);
        if (nh == 0 && g == 0) p.hs[row * (p.I / kFp8Block) + nb] = sc.scale;
      }
    }
  } else {
    const int col0 = nh * CW + 4 * g, left = p.N - nb * BN;
    uint16_t* dst = p.y + (size_t)row0 * p.N + nb * BN;
    if (p.N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if (r0 + i * 16 >= rows) continue;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          store4(dst + (size_t)(r0 + i * 16) * p.N + col0 + j * 16, acc[i][j], left - col0 - j * 16,
                 true);
      }
    } else {  // rows that are not aligned: through LDS, so that a wave writes whole rows
      uint16_t(*out)[BN + 8] = reinterpret_cast<uint16_t(*)[BN + 8]>(lds.st);
      static_assert(sizeof(lds.st) >= BM * sizeof(out[0]), "output tile");
      __syncthreads();
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          store4(&out[r0 + i * 16][col0 + j * 16], acc[i][j], 4, true);
      __syncthreads();
      for (int r = wave; r < rows; r += NW)
        for (int c = lane; c < min(BN, left); c += 64) dst[(size_t)r * p.N + c] = out[r][c];
    }
  }
}

template <int BM, int BN, int WM, int WN, int S, bool GATED>
int launch_ring(Fp8Args p, hipStream_t s, const char* who) {
  constexpr int COLS = GATED ? BN / 2 : BN;
  p.nnb = ((GATED ? p.I : p.N) + COLS - 1) / COLS;
  const int64_t mt = p.counts ? row_tiles_bound(p.M, p.E, BM) : ((int64_t)p.M + BM - 1) / BM;
  const int64_t blocks = (mt * p.nnb + kXcds - 1) / kXcds * kXcds;
  if (!grid_fits(blocks, 64 * WM * WN))
    return set_error(MOE_ERR_UNSUPPORTED, "%s: too many tiles", who);
  p.mt = (int)mt;
  fp8_ring_kernel<BM, BN, WM, WN, S, GATED><<<(unsigned)blocks, 64 * WM * WN, 0, s>>>(p);
  return check_launch(who);
}

// ---------------------------------------------------------------------------
// Tiles of 16 MI rows x 16 NJ weight rows for products of a few dozen rows: the NW waves of a
// workgroup split K (blocks w, w + NW, ...), operands go from memory straight to registers, one
// block ahead, and the waves' sums of the whole tile meet in LDS in wave order.  Gate/up: half of
// the weight rows are gate rows, half their up rows, on the bf16 MFMA.  Bound by what
// a compute unit takes in, 31 bytes per ns whatever is in flight (two to four blocks ahead or 16
// waves change nothing): so the smallest tile that still needs no second round of workgroups
// (M = 64, N = 4096, K = 7168: 18.1 us on 32 x 32 tiles, 24.7 on 32 x 64, 54 on 64 x 64).
// ---------------------------------------------------------------------------
template <int MI, int NJ, int NW, bool GATED>
__global__ __launch_bounds__(64 * NW) void fp8_split_kernel(Fp8Args p) {
  constexpr int BM = 16 * MI, OUT = GATED ? NJ / 2 : NJ, COLS = 16 * OUT, U = 2;
  static_assert(MI * OUT <= NW && kFp8Block % COLS == 0, "one subtile per wave, one scale per tile");
  __shared__ f32x4 red[NW][MI * NJ][64];
  const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowTile t;
  int nb;
  {
    RowTiles<BM> tiles;
    const int mt = p.counts ? tiles.load(p.counts, p.offsets, p.E, lane) : p.mt;
    const int G = mt * p.nnb, per = (G + kXcds - 1) / kXcds;
    const int i = (int)blockIdx.x / kXcds, v = (int)blockIdx.x % kXcds * per + i;
    if (i >= per || v >= G) return;  // uniform per block
    int tile;
    panel_tile(v, mt, p.nnb, tile, nb);
    if (p.counts) {
      t = tiles.at(tile);
      dbg_segment(t.row0, t.rows, p.M);
      if (t.rows <= 0) return;
    } else {
      t.e = 0;
      t.row0 = tile * BM;
      t.rows = min(BM, p.M - t.row0);
    }
  }
  const int K = p.K, kb = (K + kFp8Block - 1) / kFp8Block;
  const int n0 = nb * COLS, up = GATED ? p.I : 0;  // up rows lie behind the gate rows
  const uint8_t* w = slot_base(p.w, p.w_stride, p, t.e) + (size_t)n0 * K;
  const float* ws = reinterpret_cast<const float*>(slot_base(p.ws, p.ws_stride, p, t.e)) +
                    n0 / kFp8Block * kb;
  const uint8_t* a = GATED ? p.a : p.a + (size_t)t.row0 * K;
  const float* as = GATED ? p.a_scale : p.a_scale + (size_t)t.row0 * kb;
  // lane group g: codes 16 g.. and 64 + 16 g.. of a block
  uint32_t wo[NJ], ao[MI], so[MI];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int row = min(16 * (j % OUT) + l16, p.N - 1 - n0) + (j < OUT ? 0 : up);
    wo[j] = (uint32_t)row * (uint32_t)K + 16u * g;
  }
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    int r = min(16 * i + l16, t.rows - 1);
    if constexpr (GATED) r = dbg_clamp(p.row_of[t.row0 + r], p.M, kDbgSorted) / p.k;
    ao[i] = (uint32_t)r * (uint32_t)K + 16u * g;
    so[i] = (uint32_t)r * (uint32_t)kb;
  }
  struct Block {
    i32x4 w[NJ][2], a[MI][2];
    float sa[MI], sw[GATED ? 2 : 1];
  };
  auto load = [&](Block& b, int c) {
    const int c0 = c * kFp8Block;
    const uint8_t* wc = w + c0;
    const uint8_t* ac = a + c0;
    if (c0 + kFp8Block <= K) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        b.w[j][0] = *reinterpret_cast<const i32x4*>(wc + wo[j]);
        b.w[j][1] = *reinterpret_cast<const i32x4*>(wc + wo[j] + 64);
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        b.a[i][0] = *reinterpret_cast<const i32x4*>(ac + ao[i]);
        b.a[i][1] = *reinterpret_cast<const i32x4*>(ac + ao[i] + 64);
      }
    } else {
      const i32x4 zero = {0, 0, 0, 0};
      const bool ok0 = c0 + 16 * g < K, ok1 = c0 + 64 + 16 * g < K;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        b.w[j][0] = ok0 ? *reinterpret_cast<const i32x4*>(wc + wo[j]) : zero;
        b.w[j][1] = ok1 ? *reinterpret_cast<const i32x4*>(wc + wo[j] + 64) : zero;
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        b.a[i][0] = ok0 ? *reinterpret_cast<const i32x4*>(ac + ao[i]) : zero;
        b.a[i][1] = ok1 ? *reinterpret_cast<const i32x4*>(ac + ao[i] + 64) : zero;
      }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) b.sa[i] = as[so[i] + c];
    b.sw[0] = ws[c];
    if constexpr (GATED) b.sw[1] = ws[up / kFp8Block * kb + c];
  };
  f32x4 acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto join = [](const i32x4 (&v)[2]) {
    return fp8x32{v[0][0], v[0][1], v[0][2], v[0][3], v[1][0], v[1][1], v[1][2], v[1][3]};
  };
  using Frag = std::conditional_t<GATED, Decoded, fp8x32>;
  auto operand = [&](const i32x4 (&v)[2]) -> Frag {
    if constexpr (GATED) return decode_e4m3(join(v));
    else return join(v);
  };
  auto take = [&](const Block& b) {
    Frag af[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) af[i] = operand(b.a[i]);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const Frag wf = operand(b.w[j]);
      f32x4 d[MI];
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        d[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (GATED) d[i] = mfma_decoded(wf, af[i], d[i]);
        else d[i] = mfma_e4m3(wf, af[i], d[i]);
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const float s = b.sa[i] * b.sw[j / OUT];
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = fmaf(s, d[i][q], acc[i][j][q]);
      }
    }
  };
  Block b[U];
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (wave + u * NW < kb) load(b[u], wave + u * NW);
  for (int c0 = wave; c0 < kb; c0 += U * NW) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * NW, ahead = c + (U - 1) * NW;
      if (c >= kb) break;
      if (ahead < kb) load(b[(u + U - 1) % U], ahead);
      __builtin_amdgcn_sched_barrier(0);
      take(b[u]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) red[wave][i * NJ + j][lane] = acc[i][j];
  __syncthreads();
  if (wave >= MI * OUT) return;
  auto total = [&](int n) {
    f32x4 v = red[0][n][lane];
#pragma unroll
    for (int x = 1; x < NW; ++x) {
      const f32x4 o = red[x][n][lane];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += o[r];
    }
    return v;
  };
  const int i = wave / OUT, j = wave % OUT;
  const int row = 16 * i + l16, col = n0 + 16 * j + 4 * g;
  const f32x4 v = total(i * NJ + j);
  if constexpr (GATED) {
    const f32x4 u = total(i * NJ + OUT + j);
    if (row < t.rows)
      *reinterpret_cast<float4*>(p.h + (size_t)(t.row0 + row) * p.I + col) =
          float4{swiglu(v[0], u[0]), swiglu(v[1], u[1]), swiglu(v[2], u[2]), swiglu(v[3], u[3])};
  } else if (row < t.rows) {
    store4(p.y + (size_t)(t.row0 + row) * p.N + col, v, p.N - col, p.N % 4 == 0);
  }
}

template <int MI, int NJ, int NW, bool GATED>
int launch_split(Fp8Args p, hipStream_t s, const char* who) {
  constexpr int COLS = GATED ? 8 * NJ : 16 * NJ;
  p.nnb = ((GATED ? p.I : p.N) + COLS - 1) / COLS;
  const int64_t mt = p.counts ? row_tiles_bound(p.M, p.E, 16 * MI)
                              : ((int64_t)p.M + 16 * MI - 1) / (16 * MI);
  const int64_t blocks = (mt * p.nnb + kXcds - 1) / kXcds * kXcds;
  if (!grid_fits(blocks, 64 * NW))
    return set_error(MOE_ERR_UNSUPPORTED, "%s: too many tiles", who);
  p.mt = (int)mt;
  fp8_split_kernel<MI, NJ, NW, GATED><<<(unsigned)blocks, 64 * NW, 0, s>>>(p);
  return check_launch(who);
}

template <int SRC, bool GATED, int NSUB, int NW, int SPLIT, int U>
int launch_rows16_as(Fp8Args p, int64_t tiles, hipStream_t s, const char* who) {
  const int cols = (GATED ? NSUB / 2 : NSUB) * 16 * (SPLIT == 1 ? NW : 1);
  p.nnb = ((GATED ? p.I : p.N) + cols - 1) / cols;
  if (!grid_fits(p.nnb * tiles, 64 * NW))
    return set_error(MOE_ERR_UNSUPPORTED, "%s: too many tiles", who);
  fp8_rows16_kernel<SRC, GATED, NSUB, NW, SPLIT, U>
      <<<(unsigned)(p.nnb * tiles), 64 * NW, 0, s>>>(p);
  return check_launch(who);
}

// FFN of 8 tokens, 256 experts of 2048 x 512: 46.8 us with one block of K in flight per wave, 49.5
// with two, 54.4 with four (registers); the down product's K of 4 blocks split over the waves 55.7.
// Fewer than two workgroups per compute unit take single subtiles and 8 waves along K
// (1 x 7168 x 2048: 5.9 against 8.0 us).
template <int SRC, bool GATED>
int launch_rows16(const Fp8Args& p, hipStream_t s, const char* who) {
  const int64_t tiles = p.counts ? row_tiles_bound(p.M, p.E, 16) : ((int64_t)p.M + 15) / 16;
  const int kb = (p.K + kFp8Block - 1) / kFp8Block;
  const int wide = GATED ? 32 : 64, n = GATED ? p.I : p.N;
  if (tiles * ((n + wide - 1) / wide) < 2 * kXcds * kXcdCus)
    return launch_rows16_as<SRC, GATED, GATED ? 2 : 1, 8, 8, 2>(p, tiles, s, who);
  if (kb <= 8) return launch_rows16_as<SRC, GATED, 4, 4, 1, 1>(p, tiles, s, who);
  return launch_rows16_as<SRC, GATED, 4, 4, 4, 1>(p, tiles, s, who);
}

// ---------------------------------------------------------------------------
// Which kernel: by what fills the chip and how often weights are read again (times in us, E4M3
// weights resident in HBM; R = rows per expert, M / E).
//  * 16-row tiles read an expert's weights once per 16 rows: up to 4 rows per expert on average,
//    or 32 rows in all (M = 32, N = 4096, K = 7168: 21.3 against 27.2 on 64 x 64 tiles; FFN of 512 experts of 4096 x 1024: R = 1 1192 against 1189 on 64 x 256
//    tiles, R = 16 1754 against 1324; of 64 experts of 2048 x 1024: R = 8 87 against 92).
// Products of codes:
//  * 32 x 16, 32 x 32 or 32 x 64 tiles while at most one of them falls on a compute unit, smallest
//    first, for more than 16 rows (N = 4096, K = 7168: M = 32 15.1 against 17.8 on 16-row tiles,
//    M = 64 18.1 and M = 128 24.6 against 27.4 and 27.8 on 64 x 64 tiles; N = 600, K = 4096: M = 64
//    9.4 against 17.1, M = 384 11.8 against 17.0), but up to 32 rows 16-row tiles if those need
//    no second round either (M = 32, N = 600, K = 4096: 7.9 against 9.3).
//  * 64 x 64 tiles while at most two of them fall on a compute unit (N = 4096, K = 7168: M = 512
//    36 against 47 on 64 x 256 tiles, M = 777 67 against 48).
//  * 64 x 256 tiles while at most two of them fall on a compute unit (N = 4096, K = 7168: M = 1024
//    51 against 95 on 256 x 256 tiles, M = 2048 95 against 96), or for up to 64 rows per expert
//    (both products of 64 experts of 2048 x 1024: R = 32 101 against 106, R = 64 113 against 113,
//    R = 96 154 against 117; of 256 experts of 7168 x 2048: R = 64 2359 against 2741, R = 128 3577
//    against 2723).
//  * 256 x 256 tiles otherwise (two K blocks at least).
// Gate/up products, whose tiles of 32 and 64 rows run on the bf16 MFMA (FFN times):
//  * 32-row tiles where gateup_split_cols says so.
//  * 64 x 256 tiles while at most one of them falls on a compute unit where the rows spread evenly
//    over the experts (8 experts of 4096 x 1024: R = 256 86 against 98, R = 400 132 against 101;
//    32 of 2048 x 768: R = 64 47 against 50, R = 128 77 against 57), or two for up to 32 rows per
//    expert (64 of 2048 x 1024: R = 32 111 against 122, R = 48 117 against 115).
//  * 256 x 256 tiles otherwise (512 experts of 4096 x 1024: R = 16 1345 against 1421, R = 64 1558
//    against 1759; 256 of 7168 x 2048: R = 16 2173 against 2184, R = 64 2406 against 2520).
// All but the 16-row tiles address gathered activation rows with 32-bit offsets.
// ---------------------------------------------------------------------------
constexpr int64_t kCus = kXcds * kXcdCus, kTwoPerCu = 2 * kCus;

bool few_rows(int64_t M, int64_t E) { return M <= 4 * E || M <= 32; }

int launch_product(const Fp8Args& p, hipStream_t s, const char* who) {
  const int64_t M = p.M, E = p.E;
  const int64_t rt = row_tiles_bound(M, E, 64);
  const int64_t rt16 = row_tiles_bound(M, E, 16), rt32 = row_tiles_bound(M, E, 32);
  if (M > 16 && M > 4 * E && (M > 32 || rt16 * ((p.N + 15) / 16) > kCus)) {
    if (rt32 * ((p.N + 15) / 16) <= kCus) return launch_split<2, 1, 8, false>(p, s, who);
    if (rt32 * ((p.N + 31) / 32) <= kCus) return launch_split<2, 2, 8, false>(p, s, who);
    if (rt32 * ((p.N + 63) / 64) <= kCus) return launch_split<2, 4, 8, false>(p, s, who);
  }
  if (few_rows(M, E)) return launch_rows16<kSrcCodes, false>(p, s, who);
  if (rt * ((p.N + 63) / 64) <= kTwoPerCu) return launch_ring<64, 64, 2, 2, 4, false>(p, s, who);
  if (rt * ((p.N + 255) / 256) <= kTwoPerCu || M <= 64 * E || p.K <= kFp8Block)
    return launch_ring<64, 256, 2, 4, 3, false>(p, s, who);
  return launch_tiles<256, 256, 2, 4, false>(p, s, who);
}

// gate/up into hq and hs, from rows that fit 32-bit offsets
int launch_gateup(const Fp8Args& p, hipStream_t s, const char* who) {
  const int64_t M = p.M, E = p.E;
  const int64_t tiles = (M < E ? M : E) * ((M + 64 * E - 1) / (64 * E)) * (p.I / kFp8Block);
  if (tiles <= (M <= 32 * E ? kTwoPerCu : kCus) || p.K <= kFp8Block)
    return launch_ring<64, 256, 2, 4, 3, true>(p, s, who);
  return launch_tiles<256, 256, 2, 4, true>(p, s, who);
}

// Output columns of the gate/up tiles of 32 rows whose waves split K (h leaves them in fp32 and
// takes a launch of its own to be quantised): 16 or 32 where at most one tile falls on a
// compute unit with the rows spread evenly, 0 where they are not taken.  FFN of 8 experts of
// 4096 x 1024, 16 rows each: 34 us, on 64 x 256 tiles 56; 4 of 2048 x 512, 128 rows each: 25 and 35;
// up to two tiles per unit: 32 of 1408 x 512, 16 rows each 32.3 against 30.7.  A K of less than one
// block per wave does not pay for the launch (4 of 256 x 256, 10 rows each: 19 against 17).
int gateup_split_cols(int64_t A, int64_t E, int64_t H, int64_t I) {
  const int64_t rt = std::min(A, E) * ((A + 32 * E - 1) / (32 * E));
  if (H < 8 * kFp8Block) return 0;
  return rt * (I / 16) <= kCus ? 16 : rt * (I / 32) <= kCus ? 32 : 0;
}

// FFN workspace: h (fp32) on the 16-row path; xq, its scales, hq and its scales on the others,
// and h behind them where gate/up tiles do not hold whole scale blocks.  The size covers all.
struct Fp8FfnWs {
  size_t h, xq, xs, hq, hs, h_behind, total;
};
Fp8FfnWs fp8_ffn_ws(int64_t T, int64_t k, int64_t H, int64_t I) {
  auto up = [](int64_t v) { return (size_t)((v + 255) / 256 * 256); };
  const int64_t A = T * k;
  Fp8FfnWs w;
  w.h = 0;
  w.xq = 0;
  w.xs = w.xq + up(T * H);
  w.hq = w.xs + up(T * (H / kFp8Block) * 4);
  w.hs = w.hq + up(A * I);
  w.h_behind = w.hs + up(A * (I / kFp8Block) * 4);
  // tiles of 32 x 32 on every compute unit at most; never less for more tokens
  w.total = w.h_behind + up(std::min(A * I, 32 * 32 * kCus) * 4);
  if (w.total < up(A * I * 4)) w.total = up(A * I * 4);
  return w;
}

}  // namespace

#ifdef MOE_DEBUG
uint32_t dbg_take_fp8() { return dbg_take_unit(); }
#endif

}  // namespace moe

using namespace moe;

extern "C" int moe_fp8_quantize(const uint16_t* x, int32_t T, int32_t K, uint8_t* codes,
                                float* scales, moe_stream_t stream) {
  const char* who = "moe_fp8_quantize";
  if (T < 0 || K < 8 || K % 8 || K > 65536)
    return set_error(MOE_ERR_INVALID_ARG, "%s: need T>=0, K a multiple of 8 in [8, 65536] "
                     "(T=%d K=%d)", who, T, K);
  if (T == 0) return MOE_OK;
  if (!x || !codes || !scales) return set_error(MOE_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales))
    return set_error(MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  launch_quantize(x, T, K, codes, scales, reinterpret_cast<hipStream_t>(stream));
  return check_launch(who);
}

extern "C" size_t moe_fp8_matmul_workspace(int32_t M, int32_t N, int32_t K, int32_t E) {
  (void)M; (void)N; (void)K; (void)E;
  return 0;
}

extern "C" int moe_fp8_matmul(const uint8_t* a, const float* a_scale, int32_t M, const uint8_t* w,
                              const float* w_scale, int32_t N, int32_t K, const int32_t* counts,
                              const int32_t* offsets, int32_t E, uint16_t* y, void* ws,
                              size_t ws_bytes, moe_stream_t stream) {
  const char* who = "moe_fp8_matmul";
  if (M < 0 || N < 1 || K < 16 || K % 16 || N > 65536 || K > 65536 || E < 1 || E > kMaxE)
    return set_error(MOE_ERR_INVALID_ARG, "%s: need M>=0, 1<=N<=65536, K a multiple of 16 in "
                     "[16, 65536], 1<=E<=%d (M=%d N=%d K=%d E=%d)", who, kMaxE, M, N, K, E);
  if (!counts != !offsets || (!counts && E != 1))
    return set_error(MOE_ERR_INVALID_ARG, "%s: counts and offsets go together (both NULL: E = 1)",
                     who);
  if (M > (1 << 27) || (int64_t)N * K >= ((int64_t)1 << 32))
    return set_error(MOE_ERR_UNSUPPORTED, "%s: M=%d N=%d K=%d too large", who, M, N, K);
  if (M == 0) return MOE_OK;
  const size_t need = moe_fp8_matmul_workspace(M, N, K, E);
  if (!a || !a_scale || !w || !w_scale || !y || (need && !ws))
    return set_error(MOE_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned16(a) || !aligned16(a_scale) || !aligned16(w) || !aligned16(w_scale) ||
      !aligned16(counts) || !aligned16(offsets) || !aligned16(y) || !aligned16(ws))
    return set_error(MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  if (ws_bytes < need)
    return set_error(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", who, ws_bytes, need);
  const int64_t kb = (K + kFp8Block - 1) / kFp8Block, nb = (N + kFp8Block - 1) / kFp8Block;
  Fp8Args p{};
  p.a = a;
  p.a_scale = a_scale;
  p.k = 1;
  p.w = w;
  p.w_stride = (int64_t)N * K;
  p.ws = reinterpret_cast<const uint8_t*>(w_scale);
  p.ws_stride = nb * kb * 4;
  p.counts = counts;
  p.offsets = offsets;
  p.E = E; p.M = M; p.N = N; p.K = K;
  p.y = y;
  return launch_product(p, reinterpret_cast<hipStream_t>(stream), who);
}

extern "C" size_t moe_expert_ffn_fp8_workspace(const moe_experts* W, int32_t T, int32_t k) {
  if (!W || T < 0 || k < 1 || W->H < 1 || W->I < 1) return 0;
  return fp8_ffn_ws(T, k, W->H, W->I).total;
}

extern "C" int moe_expert_ffn_fp8(const moe_experts* W, const int32_t* slot_of_expert,
                                  const uint16_t* x, int32_t T, int32_t k, const int32_t* counts,
                                  const int32_t* offsets, const int32_t* sorted_idx,
                                  uint16_t* y_perm, void* ws, size_t ws_bytes,
                                  moe_stream_t stream) {
  const char* who = "moe_expert_ffn_fp8";
  if (!W) return set_error(MOE_ERR_INVALID_ARG, "%s: W is NULL", who);
  if (W->E < 1 || W->E > kMaxE) return set_error(MOE_ERR_INVALID_ARG, "%s: E=%d", who, W->E);
  Layout L;
  if (W->fmt != MOE_W_FP8_B128 || !layout_of(W->fmt, W->H, W->I, &L))
    return set_error(MOE_ERR_UNSUPPORTED, "%s: needs FP8 block-scaled weights (fmt=%d H=%d I=%d)",
                     who, W->fmt, W->H, W->I);
  if (!W->base || !aligned16(W->base)) return set_error(MOE_ERR_INVALID_ARG, "%s: base", who);
  if (W->stride < L.stride || W->stride % 256)
    return set_error(MOE_ERR_INVALID_ARG, "%s: stride %lld (need >= %lld, multiple of 256)", who,
                     (long long)W->stride, (long long)L.stride);
  if (T < 0 || k < 1 || k > W->E || k > kMaxK)
    return set_error(MOE_ERR_INVALID_ARG, "%s: need T>=0, 1<=k<=min(E,%d)", who, kMaxK);
  const int64_t A = (int64_t)T * k;
  if (A > (1 << 27)) return set_error(MOE_ERR_UNSUPPORTED, "%s: T*k too large", who);
  if (T == 0) return MOE_OK;
  if (!x || !counts || !offsets || !sorted_idx || !y_perm || !ws)
    return set_error(MOE_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned16(x) || !aligned16(counts) || !aligned16(offsets) || !aligned16(sorted_idx) ||
      !aligned16(y_perm) || !aligned16(ws) || !aligned16(slot_of_expert))
    return set_error(MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  const int H = W->H, I = W->I;
  const Fp8FfnWs B = fp8_ffn_ws(T, k, H, I);
  if (ws_bytes < B.total)
    return set_error(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", who, ws_bytes, B.total);
  uint8_t* wb = static_cast<uint8_t*>(ws);
  const uint8_t* rec = static_cast<const uint8_t*>(W->base);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  Fp8Args p{};
  p.row_of = sorted_idx;
  p.k = k;
  p.w = rec + L.w13;
  p.ws = rec + L.w13s;
  p.w_stride = p.ws_stride = W->stride;
  p.slot_of = slot_of_expert;
  p.counts = counts;
  p.offsets = offsets;
  p.E = W->E; p.M = (int)A; p.N = 2 * I; p.K = H; p.I = I;
  Fp8Args d = p;  // down
  d.row_of = nullptr;
  d.w = rec + L.w2;
  d.ws = rec + L.w2s;
  d.N = H; d.K = I;
  d.y = y_perm;
  if (few_rows(A, W->E) || (int64_t)T * H >= ((int64_t)1 << 32)) {
    // two launches, which quantise x and h as they read them
    p.a = reinterpret_cast<const uint8_t*>(x);
    p.h = reinterpret_cast<float*>(wb + B.h);
    const int st = launch_rows16<kSrcBf16, true>(p, s, who);
    if (st) return st;
    d.a = wb + B.h;
    return launch_rows16<kSrcF32, false>(d, s, who);
  }
  launch_quantize(x, T, H, wb + B.xq, reinterpret_cast<float*>(wb + B.xs), s);
  p.a = wb + B.xq;
  p.a_scale = reinterpret_cast<const float*>(wb + B.xs);
  p.hq = wb + B.hq;
  p.hs = reinterpret_cast<float*>(wb + B.hs);
  const int cols = gateup_split_cols(A, W->E, H, I);
  if (cols) p.h = reinterpret_cast<float*>(wb + B.h_behind);
  const int st = cols == 16   ? launch_split<2, 2, 8, true>(p, s, who)
                 : cols == 32 ? launch_split<2, 4, 8, true>(p, s, who)
                              : launch_gateup(p, s, who);
  if (st) return st;
  if (cols) launch_quantize(p.h, (int)A, I, p.hq, p.hs, s);
  d.a = p.hq;
  d.a_scale = p.hs;
  return launch_product(d, s, who);
}
