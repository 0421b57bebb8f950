// Training of the experts (BF16 records): the SwiGLU FFN that keeps its gate and up products, and
// its gradient.  Rows p in expert order, expert e = that of the row:
//   forward   g = Wg x, u = Wu x (kept as bf16); h = silu(g) u;  y = Wd h
//   backward  dh = Wd^T dy, s = 1 / (1 + e^-g):  du = dh g s,  dg = dh u s (1 + g (1 - s)),
//             dx = W13^T (dg; du),  dW13 = sum_p (dg; du) x^T,  dWd = sum_p dy h^T
// Six grouped products on the 32x32x16 bf16 MFMA with fp32 accumulation, of two kinds:
//   rows     out[p][n] = sum_k A[p][k] B[n][k]: the forward's two (weights as stored, K contiguous)
//            and dh, dx (the weights' other index is summed over: K strided);
//   weights  out[e][m][n] = sum_(p of e) A[p][m] B[p][n]: both operands K strided.
// Roundings: h and (dg; du) go to bf16 once, as the operands of the next product (small batches: to
// two bf16 parts); the forward's h comes from the fp32 gate and up sums, the gradient's from the kept
// bf16 ones.  Why: the bf16 MFMA takes them, and a rounded operand is off by as much as the result's own
// rounding, so a result is off by 0.0023 to 0.0024 of its norm instead of 0.0017; two parts for all batches
// would leave 0.0017 but take 1.33 times the operations of the forward and 1.83 times the gradient's,
// which the MFMAs bound.
//
// Tiles of 256 x 256 outputs on 4 waves, one per SIMD, 128 x 128 outputs each (all of a wave's
// 256 accumulation registers): a K step of 16 then reads 8 KB of operands per wave from LDS for 16
// MFMAs.  The LDS delivers about 117 bytes a clock (measured; 97 through its transposing loads)
// and takes the copies besides, so 8 waves of 128 x 64 would need it for longer than the MFMAs.
// K goes in blocks of 64, both operands copied from memory straight into LDS, two stages.  An
// operand whose K is strided is read back through the transposing loads.
//   A wave keeps a block's fragments of the columns' operand (16 of 4 registers) and passes its
// four row subtiles over them, 16 MFMAs each.  So a block's columns are in registers when its
// first subtile ends, and its rows are read subtile by subtile: their places are refilled with the
// block after the next at two barriers per block, long before the stage is done, and a copy has
// 1.2 blocks' time to arrive.  They are spread over the MFMAs: the compute unit takes 64 bytes a
// clock, and a wave that issues them faster stands still (one per MFMA: 500 of 2050 clocks lost
// per block).
//   A workgroup owns its compute unit and works through a list of tiles as one sequence of blocks:
// the next tile's first blocks are copied under the current one's last and its epilogue.
//   Measured (averages of a kernel trace), 16384 tokens over 8 of 64 experts of 4096 x 1024: dh 1155 us
// (0.95 PFLOP/s, its epilogue moves 655 KB a tile), dx 2021 (1.09), dW13 2199 (1.00), dWd 958 (1.15);
// library products of these layouts reach 1.06 to 1.23.  A block takes 2630 clocks (weights: 2880), 2048 of
// them MFMAs, 2200 without its copies, at 1.6 to 1.75 GHz (the power limit).  4096 tokens over 8 of 64 of
// 2048 x 1024: gate/up 380 us, down 196, a quarter of it rows past the experts' last, the MFMAs busy for
// 63 and 61 % of the clocks; library products of as many MFMAs, both operands K-contiguous like these,
// take 251 and 135 us (78 and 67 %; 92 % at 8192^3), so it is the loop and not the power limit that is short.
#include <type_traits>

#include "fp8_common.h"
#include "lds_copy.h"
#include "moe_internal.h"

namespace moe {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((__vector_size__(4 * sizeof(short)))) short i16x4;
typedef __attribute__((__vector_size__(8 * sizeof(short)))) short i16x8;

constexpr int kBK = 64;            // K of a block
constexpr int kTile = 256;         // rows and columns of a tile
constexpr int kNW = 4;             // waves: 2 along the rows x 2 along the columns
constexpr int kXcds = 8, kXcdCus = 32;
constexpr int kPanel = 4;          // row tiles that share weights in an XCD's L2
constexpr int kSortE = 64 * kNW;   // experts that a workgroup sorts by rows (one per thread); with more, their
                                   // rows average out and the sort would cost more than a tile
constexpr int kListTiles = 64;     // tiles of one workgroup at most
constexpr int kOperandB = kTile * kBK * 2;          // bytes of an operand's block
constexpr int kCopies = kOperandB / 1024 / kNW;     // 1 KB copies of it per wave
constexpr int kEpiB = 4096;        // per wave: 32 rows of 128 bytes on their way out

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// One operand's block in LDS, 256 rows (or columns) x 64 K, copied in 32 pieces of 1 KB.
//   kRows: K contiguous, [256 rows][64 K], 16-byte units XORed by row; piece n: rows 8 n to 8 n + 7.
//   kByCols: K strided, [4 x 64 columns][64 K][64 columns], the 64-byte halves of a line exchanged
//     where K & 2; piece n: K 8 (n % 8) to + 7 of columns 64 (n / 8).
//   kByK: K strided, [64 K][256 columns], the 64-byte quarters of each 256 bytes XORed with K % 4;
//     piece n: K 2 n and 2 n + 1.  Whole rows of memory, but no part is done before the whole.
// The exchanges let a transposing load's 4 K x 32 columns meet distinct banks.
enum Staging { kRows, kByCols, kByK };
template <Staging L>
struct Operand {
  static constexpr int kAddrs = L == kRows ? 1 : L == kByCols ? 2 : 4;  // subtiles with addresses of their own
  // Of the lane's 16 bytes of piece n: the operand's row (column of a strided one) and K.
  static __device__ __forceinline__ int row_of(int n, int lane) {
    const int line = n * 8 + (lane >> 3);
    if constexpr (L == kRows) return line;
    else if constexpr (L == kByCols) return (n >> 3) * 64 + ((lane & 7) ^ ((line & 2) << 1)) * 8;
    else return ((lane & 31) ^ ((k_of(n, lane) & 3) << 2)) * 8;
  }
  static __device__ __forceinline__ int k_of(int n, int lane) {
    if constexpr (L == kRows) return ((lane & 7) ^ a_swz(n * 8 + (lane >> 3))) * 8;
    else if constexpr (L == kByCols) return (n * 8 + (lane >> 3)) & 63;
    else return n * 2 + (lane >> 5);
  }
  // This lane's address of subtile i (of 4, 32 rows each) of half `half` at K step 0, up to what
  // frag adds.
  static __device__ __forceinline__ int addr(int half, int i, int lane) {
    const int l = lane & 15, k = 8 * (lane >> 5) + (l >> 2), in = ((lane >> 4) & 1) * 32 + (l & 3) * 8;
    if constexpr (L == kRows) {
      const int r = half * 128 + (lane & 31);
      return r * 128 + (((lane >> 5) ^ a_swz(r)) << 4);
    } else if constexpr (L == kByCols) {
      return (half * 2 * 64 + k) * 128 + (((i & 1) ^ ((k >> 1) & 1)) << 6) + in;
    } else {
      return k * 512 + half * 256 + ((i ^ (k & 3)) << 6) + in;
    }
  }
  // The 8 values at K = 16 s + 8 (lane / 32) of subtile i's row (column) lane % 32.
  static __device__ __forceinline__ bf16x8 frag(const uint8_t* block, int addr, int i, int s) {
    if constexpr (L == kRows) {
      return *reinterpret_cast<const bf16x8*>(block + (addr ^ (s * 32)) + i * 32 * 128);
    } else {
      constexpr int kLine = L == kByCols ? 128 : 512;
      using lds_t = __attribute__((address_space(3))) i16x4;
      const uint8_t* p = block + addr + s * 16 * kLine + (L == kByCols ? (i >> 1) * 64 * 128 : 0);
      const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)p);
      const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)(p + 4 * kLine));
      const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      return __builtin_bit_cast(bf16x8, v);
    }
  }
};

// v-th tile of mt row tiles x nnb column blocks: panels of kPanel row tiles, column by column
__device__ __forceinline__ void panel_tile(int v, int mt, int nnb, int& tile, int& nb) {
  const int panel = v / (kPanel * nnb), r = v - panel * (kPanel * nnb);
  const int rows = min(kPanel, mt - panel * kPanel);
  nb = r / rows;
  tile = panel * kPanel + r - nb * rows;
}

enum Kind { kDown, kGateUp, kDh, kDx, kWeights };

// h and the gradients of g and u from dh and the kept g and u (bf16 pairs), four of them.  The
// sigmoid is on the hardware's 2^x and 1/x (one ulp each); all three are rounded to bf16 next.
struct GradSwiglu {
  float h[4], dg[4], du[4];
};
__device__ __forceinline__ GradSwiglu grad_swiglu(const f32x4& dh, const uint2& gb, const uint2& ub) {
  const uint32_t gw[2] = {gb.x, gb.y}, uw[2] = {ub.x, ub.y};
  GradSwiglu r;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const float g = __uint_as_float(v & 1 ? gw[v / 2] & 0xffff0000u : gw[v / 2] << 16);
    const float u = __uint_as_float(v & 1 ? uw[v / 2] & 0xffff0000u : uw[v / 2] << 16);
    const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(g * -1.44269504f));
    r.h[v] = g * s * u;
    r.du[v] = dh[v] * (g * s);
    r.dg[v] = dh[v] * u * (s * fmaf(g, 1.f - s, 1.f));
  }
  return r;
}

struct TrainArgs {
  int E, I, k, A;
  const int* counts;
  const int* offsets;
  const int* sorted_idx;   // rows of the gathered operand (a; weights: b), NULL: in expert order
  const uint8_t* a;        // bf16 [rows][K]; weights: [rows][M]
  const uint8_t* b;        // weights of expert 0; kWeights: bf16 [rows][N]
  int64_t stride;          // bytes between experts
  int M, N, K;             // M: kWeights' output rows; N: output columns (kGateUp: I); K: summed over
  int mt, nnb;             // kWeights: row tiles of an expert; column blocks
  void* out;               // [A][N]; kGateUp, kDh: h [A][I]; kWeights: [E][M][N]
  uint16_t* out2;          // kGateUp: gate_up; kDh: (dg; du)
  const uint16_t* gu;      // kDh: gate_up
  // Small batches: what rounding the products between (h, dg and du) to bf16 takes off, itself in bf16,
  // behind them by so many bytes (0: not kept): as operands (a, b), as results (h: out, dg and du: out2)
  int64_t a_rest, b_rest, out_rest, out2_rest;
  uint32_t k_magic;        // floor(2^32 / k) + 1: a / k for k > 1 and a < 2^27 as a 64-bit product's high word
};

__device__ __forceinline__ uint32_t token_of(uint32_t a, const TrainArgs& p) {
  return p.k == 1 ? a : __umulhi(a, p.k_magic);
}

struct TrainLds {
  uint8_t a[2][kOperandB];
  uint8_t b[2][kOperandB];
  uint8_t epi[kNW][kEpiB];
  __attribute__((aligned(16))) int list[kListTiles][4];
  int src[4][kTile];  // gathered rows: of a tile ([tile % 2]); weights: of a block ([block % 4][64])
};
static_assert(sizeof(TrainLds) <= 160 * 1024, "LDS");

// 32 x 32 fp32 or 32 x 64 bf16 values from the MFMA's layout to rows: 8 lanes per row, 16 bytes
// each, rows lane / 8 + 8 r.  A wave's own 4 KB of LDS, whose accesses stay in order.
__device__ __forceinline__ int epi_at(int row, int unit) {
  return row * 128 + ((unit ^ ((row >> 1) & 7)) << 4);
}
__device__ __forceinline__ void epi_put16(uint8_t* e, int lane, int unit, uint4 v) {
  *reinterpret_cast<uint4*>(e + epi_at(lane & 31, unit)) = v;
}
__device__ __forceinline__ void epi_put8(uint8_t* e, int lane, int unit, uint2 v) {
  *reinterpret_cast<uint2*>(e + epi_at(lane & 31, unit) + (lane >> 5) * 8) = v;
}
__device__ __forceinline__ uint4 epi_get(const uint8_t* e, int lane, int r) {
  return *reinterpret_cast<const uint4*>(e + epi_at((lane >> 3) + 8 * r, lane & 7));
}

// Keeps accumulators in their registers up to here: without it the compiler moves all 256 to
// others as the loop ends, and spills.
__device__ __forceinline__ void keep(f32x16& v) { asm volatile("" : "+a"(v)); }

// Value 4q + r of acc[i][j] is output row 32 i + lane % 32, column 32 j + 8q + 4 (lane / 32) + r of
// the wave's 128 x 128.
__device__ __forceinline__ uint2 pack4(const f32x16& v, int q) {
  return uint2{bf16_pack2(v[4 * q], v[4 * q + 1]), bf16_pack2(v[4 * q + 2], v[4 * q + 3])};
}

// GATHER: the rows of a (weights: of b) are tokens', through sorted_idx.
template <Kind KIND, bool F32, bool GATHER>
__global__ __launch_bounds__(64 * kNW, 1) void train_gemm_kernel(TrainArgs p, int accumulate) {
  constexpr bool W = KIND == kWeights;
  constexpr bool BT = W || KIND == kDh || KIND == kDx;
  constexpr int COLS = KIND == kGateUp ? kTile / 2 : kTile;
  using OA = Operand<W ? kByCols : kRows>;
  using OB = Operand<BT ? kByK : kRows>;
  __shared__ TrainLds lds;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int mh = wave >> 1, nh = wave & 1;

  // -- this workgroup's tiles: (expert, first row, rows, column block | row block << 16) -----------
  int mine;
  {
    const int x = (int)blockIdx.x % kXcds, i0 = (int)blockIdx.x / kXcds;
    const int NWG = (int)gridDim.x / kXcds;
    int* before = reinterpret_cast<int*>(lds.a);  // [E + 1]: row tiles before each expert
    int mt = 0;
    if constexpr (!W) {
      if (wave == 0) {
        RowTiles<kTile> t;
        const int total = t.load(p.counts, p.offsets, p.E, lane);
        int run = t.upto - t.mine;
#pragma unroll
        for (int i = 0; i < kMaxE / 64; ++i)
          if (i < t.per && t.first + i < p.E) {
            before[t.first + i] = run;
            run += (t.n[i] + kTile - 1) / kTile;
          }
        if (lane == 0) before[p.E] = total;
      }
      __syncthreads();
      mt = before[p.E];
    }
    // rows: an XCD takes a contiguous range.  weights: groups of 32 tiles, one for each of an XCD's
    // compute units, dealt to the XCDs back and forth from the expert with most rows to the one
    // with fewest.
    const int per_e = p.mt * p.nnb;
    const int G = W ? p.E * per_e : mt * p.nnb;
    const int per = (G + kXcds - 1) / kXcds;
    auto tile_of = [&](int i) {
      const int round = i / kXcdCus;
      return (round * kXcds + (round & 1 ? kXcds - 1 - x : x)) * kXcdCus + i % kXcdCus;
    };
    int* by_rows = before + kMaxE;  // [E]: experts, most rows first
    mine = 0;
    if constexpr (W) {
      const int rounds = (G + kXcdCus * kXcds - 1) / (kXcdCus * kXcds);
      const int n = rounds * kXcdCus;
      mine = i0 < n ? (n - i0 + NWG - 1) / NWG : 0;
      while (mine > 0 && tile_of(i0 + (mine - 1) * NWG) >= G) --mine;  // the last round may be short
      for (int e = tid; e < p.E; e += 64 * kNW) {
        before[e] = p.counts[e];
        by_rows[e] = e;
      }
      __syncthreads();
      if (p.E <= kSortE && tid < p.E) {
        const int n_e = before[tid];
        int rank = 0;
        for (int f = 0; f < p.E; ++f) rank += before[f] > n_e || (before[f] == n_e && f < tid);
        by_rows[rank] = tid;
      }
      __syncthreads();
    } else {
      const int n = min(per, G - x * per);
      mine = i0 < n ? (n - i0 + NWG - 1) / NWG : 0;
    }
    mine = __builtin_amdgcn_readfirstlane(min(mine, kListTiles));
    if (mine == 0) return;  // uniform
    if (tid < mine) {
      const int i = i0 + tid * NWG;
      int e, row0, rows, place;
      if constexpr (W) {
        const int v = tile_of(i);
        const int at = v / per_e;
        e = by_rows[at];
        int mb, nb;
        panel_tile(v - at * per_e, p.mt, p.nnb, mb, nb);
        place = nb | mb << 16;
        rows = max(p.counts[e], 0);
        row0 = p.offsets[e];
        dbg_segment(row0, rows, p.A);
      } else {
        int tile, nb;
        panel_tile(x * per + i, mt, p.nnb, tile, nb);
        int lo = 0, hi = p.E - 1;  // the last expert with before[e] <= tile
        while (lo < hi) {
          const int m = (lo + hi + 1) >> 1;
          if (before[m] <= tile) lo = m;
          else hi = m - 1;
        }
        e = lo;
        const int sub = tile - before[e];
        rows = min(kTile, p.counts[e] - sub * kTile);
        row0 = p.offsets[e] + sub * kTile;
        dbg_segment(row0, rows, p.A);
        place = nb;
      }
      *reinterpret_cast<i32x4*>(lds.list[tid]) = i32x4{e, row0, rows, place};
    }
    __syncthreads();
  }
  auto entry = [&](int r, int f) { return __builtin_amdgcn_readfirstlane(lds.list[r][f]); };
  // blocks of a tile (weights: at least one, of zeros where the expert has no rows)
  auto blocks_of = [&](int r) { return W ? max((entry(r, 2) + kBK - 1) / kBK, 1) : p.K / kBK; };

  // -- copies -------------------------------------------------------------------------------------
  // The block being copied: tile cr, cleft blocks left of it (this one included), from asrc and
  // bsrc at the lane's offsets.  Behind the last block the copies repeat it, into places that
  // nobody reads: no branches around them.
  //   A wave's pieces: of a, 4 of the waves' first two row subtiles (q < 4) and 4 of the others; of
  // b, 8 in a row.
  auto a_piece = [&](int q) { return (wave >> 1) * 16 + (q >> 2) * 8 + (wave & 1) * 4 + (q & 3); };
  auto b_piece = [&](int q) { return wave * kCopies + q; };
  int cr = 0, cleft = blocks_of(0);
  const uint8_t *asrc, *bsrc;
  uint32_t ao[kCopies], bo[kCopies];
  uint32_t bcol[2];  // weights, gathered: the lane's columns in even and odd pieces
  const size_t astep = W ? (size_t)kBK * p.M * 2 : (size_t)kBK * 2;
  const size_t bstep = GATHER && W ? 0 : BT ? (size_t)kBK * p.N * 2 : (size_t)kBK * 2;
  // Gathered rows of a block of weights come by the ring lds.src, two blocks ahead of the copies:
  // cursor of the block whose rows are next, tile sr, first of its rows sp of sn.  An expert without
  // rows owns no entry of the index, and its offset may name one that holds anything: token 0.
  int sr = 0, sp = 0, sn = 0, srow = 0, sq = 0;
  auto issue_ring = [&]() {
    if (wave == 0) {
      if (sp == 0) {
        srow = entry(sr, 1);
        sn = entry(sr, 2);
      }
      if (sn > 0) {  // rows past the segment: its last one
        dma4(reinterpret_cast<const uint8_t*>(p.sorted_idx + srow + sp), (uint32_t)min(lane, sn - 1 - sp) * 4u,
             lds.src[sq & 3]);
      } else {
        lds.src[sq & 3][lane] = 0;
      }
      ++sq;
      if (sp + kBK < sn) {
        sp += kBK;
      } else if (sr + 1 < mine) {
        ++sr;
        sp = 0;
      }
    }
  };
  int rq = 0;             // blocks whose rows have been read from the ring
  uint32_t rows_next[GATHER && W ? kCopies : 1];
  auto read_ring = [&](int q) {
    rows_next[q] = token_of((uint32_t)dbg_clamp(lds.src[rq & 3][OB::k_of(b_piece(q), lane)], p.A, kDbgSorted), p) *
                   (uint32_t)(p.N * 2);
  };
  // Gathered rows of tile r on their way into LDS.
  auto issue_src = [&](int r) {
    const int i = min(wave * 64 + lane, max(entry(r, 2), 1) - 1);
    dma4(reinterpret_cast<const uint8_t*>(p.sorted_idx + entry(r, 1)), (uint32_t)i * 4u,
         lds.src[r & 1] + wave * 64);
  };
  // The last block of an expert's rows may be short (weights): rows past the end read its last one,
  // and trim puts zeros in their place.
  auto shorten = [&](int left) {
    if (left >= kBK) return;
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      auto over = [&](int k) { return (uint32_t)max(k - max(left - 1, 0), 0); };
      ao[q] -= over(OA::k_of(a_piece(q), lane)) * (uint32_t)(p.M * 2);
      if (!GATHER) bo[q] -= over(OB::k_of(b_piece(q), lane)) * (uint32_t)(p.N * 2);
    }
  };
  // Zeros past the end in what has landed and is about to be read: the columns and the first rows
  // (all of them: also the second), or the second rows.
  enum { kFirst = 1, kSecond = 2 };
  auto trim = [&](int s, int left, int parts) {
    if constexpr (W) {
      if (left >= kBK) return;
      left = max(left, 0);
      const int n = (kBK - left) * 8;  // 16-byte units of a column piece
      for (int i = tid; i < 2 * n; i += 64 * kNW) {
        uint8_t* line = lds.a[s] + (i >= n ? 2 : 0) * 64 * 128 + left * 128 + (i >= n ? i - n : i) * 16;
        if (parts & kFirst) *reinterpret_cast<uint4*>(line) = uint4{0, 0, 0, 0};
        if (parts & kSecond) *reinterpret_cast<uint4*>(line + 64 * 128) = uint4{0, 0, 0, 0};
      }
      if (parts & kFirst)
        for (int i = tid; i < 4 * n; i += 64 * kNW)
          *reinterpret_cast<uint4*>(lds.b[s] + left * 512 + i * 16) = uint4{0, 0, 0, 0};
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(63));
      asm volatile("s_barrier" ::: "memory");
    }
  };
  auto point_at = [&](int r) {
    const int e = entry(r, 0), row0 = entry(r, 1), rows = entry(r, 2), place = entry(r, 3);
    const int nb = place & 0xffff;
    cleft = blocks_of(r);
    // the lane's part is recomputed per tile: hoisted out of the loop it would cost registers
    int ln = lane;
    asm volatile("" : "+v"(ln));
    if constexpr (W) {
      const int mb = place >> 16;
      const int first = min(max(row0, 0), p.A - 1);  // an expert without rows may start at A
      asrc = p.a + (size_t)first * p.M * 2;
      bsrc = GATHER ? p.b : p.b + (size_t)first * p.N * 2;
#pragma unroll
      for (int q = 0; q < kCopies; ++q) {
        const int na = a_piece(q), nb_ = b_piece(q);
        ao[q] = (uint32_t)OA::k_of(na, ln) * (uint32_t)(p.M * 2) +
                (uint32_t)min(mb * kTile + OA::row_of(na, ln), p.M - 8) * 2;
        const uint32_t c = (uint32_t)min(nb * kTile + OB::row_of(nb_, ln), p.N - 8) * 2;
        if (GATHER) bcol[q & 1] = c;
        else bo[q] = (uint32_t)OB::k_of(nb_, ln) * (uint32_t)(p.N * 2) + c;
      }
      if (cleft == 1) shorten(rows);
    } else {
      asrc = GATHER ? p.a : p.a + (size_t)row0 * p.K * 2;
      bsrc = p.b + (size_t)e * p.stride;
#pragma unroll
      for (int q = 0; q < kCopies; ++q) {
        const int lr = OA::row_of(a_piece(q), ln);
        const uint32_t row = GATHER ? token_of((uint32_t)dbg_clamp(lds.src[r & 1][lr], p.A, kDbgSorted), p)
                                    : (uint32_t)max(min(lr, rows - 1), 0);
        ao[q] = row * (uint32_t)(p.K * 2) + (uint32_t)OA::k_of(a_piece(q), ln) * 2;
      }
#pragma unroll
      for (int q = 0; q < kCopies; ++q) {
        const int lr = OB::row_of(b_piece(q), ln), k = OB::k_of(b_piece(q), ln);
        if constexpr (BT) {  // [K][N]
          bo[q] = (uint32_t)k * (uint32_t)(p.N * 2) + (uint32_t)min(nb * kTile + lr, p.N - 8) * 2;
        } else if constexpr (KIND == kGateUp) {  // a wave's 128 weight rows: 64 gate rows, their up rows
          const int col = min(nb * COLS + (lr >> 7) * 64 + (lr & 63), p.N - 1);
          bo[q] = (uint32_t)((lr & 64) ? p.I + col : col) * (uint32_t)(p.K * 2) + (uint32_t)k * 2;
        } else {
          bo[q] = (uint32_t)min(nb * kTile + lr, p.N - 1) * (uint32_t)(p.K * 2) + (uint32_t)k * 2;
        }
      }
    }
  };
  // On to the next block.
  auto advance = [&]() {
    if (cleft > 1) {
      --cleft;
      asrc += astep;
      bsrc += bstep;
      if (W && cleft == 1) shorten(entry(cr, 2) - (blocks_of(cr) - 1) * kBK);
    } else if (cr + 1 < mine) {
      ++cr;
      point_at(cr);
      if (!W && GATHER && cr + 1 < mine) issue_src(cr + 1);
    }
    if constexpr (W && GATHER) {
#pragma unroll
      for (int q = 0; q < kCopies; ++q) bo[q] = rows_next[q] + bcol[q & 1];
      ++rq;
      issue_ring();
    }
  };
  auto copy_a = [&](int s, int q) { dma16(asrc, ao[q], lds.a[s] + a_piece(q) * 1024); };
  auto copy_b = [&](int s, int q) { dma16(bsrc, bo[q], lds.b[s] + b_piece(q) * 1024); };

  // -- the first two blocks -----------------------------------------------------------------------
  if constexpr (GATHER) {
    if constexpr (W) {
      for (int i = 0; i < 3; ++i) issue_ring();
    } else {
      issue_src(0);
      if (mine > 1) issue_src(1);
    }
    MOE_DMA_SYNC(0);
  }
  point_at(0);
  if constexpr (W && GATHER) {
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      read_ring(q);
      bo[q] = rows_next[q] + bcol[q & 1];
    }
    ++rq;
#pragma unroll
    for (int q = 0; q < kCopies; ++q) read_ring(q);
  }
#pragma unroll
  for (int q = 0; q < kCopies; ++q) {
    copy_a(0, q);
    copy_b(0, q);
  }
  advance();
#pragma unroll
  for (int q = 0; q < kCopies; ++q) {
    copy_a(1, q);
    copy_b(1, q);
  }
  MOE_DMA_SYNC(0);

  // -- compute ------------------------------------------------------------------------------------
  int aa[OA::kAddrs], ba[OB::kAddrs];
#pragma unroll
  for (int i = 0; i < OA::kAddrs; ++i) aa[i] = OA::addr(mh, i, lane);
#pragma unroll
  for (int j = 0; j < OB::kAddrs; ++j) ba[j] = OB::addr(nh, j, lane);
  f32x16 acc[4][4];
  bf16x8 af[2][4], bf[4][4];  // of a: two subtiles' four K steps; of b: [K step][subtile]
  auto get_a = [&](int s, int i, int step) {
    af[i & 1][step] = OA::frag(lds.a[s], aa[i % OA::kAddrs], i, step);
  };
  auto get_b = [&](int s, int n) {  // in the order of their use
    bf[n >> 2][n & 3] = OB::frag(lds.b[s], ba[(n & 3) % OB::kAddrs], n & 3, n >> 2);
  };
  int s = 0;  // stage of the block being multiplied
  trim(0, entry(0, 2), kFirst | kSecond);
#pragma unroll
  for (int n = 0; n < 4; ++n) get_a(s, 0, n);
#pragma unroll
  for (int n = 0; n < 16; ++n) get_b(s, n);
  for (int r = 0; r < mine; ++r) {
    const int rows = entry(r, 2), row0 = entry(r, 1), place = entry(r, 3), nb = place & 0xffff;
    const int nblk = blocks_of(r);
    const int rows_after = W && r + 1 < mine ? entry(r + 1, 2) : kBK;  // weights: the next tile's
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
    for (int c = 0; c < nblk; ++c) {
      // 64 MFMAs: subtile i = n / 16, K step (n / 4) % 4, column subtile n % 4
      auto mfmas = [&](auto first, auto last) {
#pragma unroll
        for (int n = first; n < last; ++n) {
          const int i = n >> 4, step = (n >> 2) & 3, j = n & 3;
          acc[i][j] = mfma32(bf[step][j], af[i & 1][step], acc[i][j]);
          // The next block's columns replace this one's behind their last use, two in three MFMAs
          // (faster than the LDS could keep up with otherwise): the first ten under the last
          // subtile, the others under the next block's first, where they are used last.
          if (n >= 50 && (n - 50) % 3 != 2) get_b(s ^ 1, (n - 50) / 3 * 2 + (n - 50) % 3);
          if (n < 10 && (n + 14) % 3 != 2 && (n + 14) / 3 * 2 + (n + 14) % 3 < 16)
            get_b(s, (n + 14) / 3 * 2 + (n + 14) % 3);
          // the next subtile's rows, of the next block behind the last
          if (n >= 10 && n < 14) get_a(s, 1, n - 10);
          if (n >= 18 && n < 22) get_a(s, 2, n - 18);
          if (n >= 34 && n < 38) get_a(s, 3, n - 34);
          if (n >= 49 && n < 61 && (n - 49) % 3 == 0) get_a(s ^ 1, 0, (n - 49) / 3);
          if constexpr (W && GATHER)
            if (n >= 2 && n < 10) read_ring(n - 2);
          if (n >= 18 && n < 34 && n % 2 == 0) copy_b(s, (n - 18) / 2);
          if (n >= 34 && n < 42 && n % 2 == 0) copy_a(s, (n - 34) / 2);
          if (n >= 50 && n < 62 && n % 3 == 2) copy_a(s, 4 + (n - 50) / 3);
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      using std::integral_constant;
      mfmas(integral_constant<int, 0>{}, integral_constant<int, 17>{});
      // Every wave has this block's columns and its rows 0 to 63 of 128 in registers: their places
      // are free.  Landed: this block's other rows (16 copies were issued since).
      MOE_DMA_SYNC(16);
      if constexpr (W) trim(s, rows - c * kBK, kSecond);
      advance();
      mfmas(integral_constant<int, 17>{}, integral_constant<int, 33>{});
      mfmas(integral_constant<int, 33>{}, integral_constant<int, 49>{});
      // ... and its other rows.  Landed: the next block's columns and first rows (likewise).
      MOE_DMA_SYNC(16);
      if constexpr (W) trim(s ^ 1, c + 1 < nblk ? rows - (c + 1) * kBK : rows_after, kFirst);
      mfmas(integral_constant<int, 49>{}, integral_constant<int, 64>{});
      s ^= 1;
    }

    // -- epilogue -----------------------------------------------------------------------------------
    uint8_t* ep = lds.epi[wave];
    const int er = lane >> 3, eu = lane & 7;
    // kDh: gate_up of the next pieces (32 x 32) is loaded that many of them ahead
    constexpr int kGuAhead = 3;
    uint2 gbuf[KIND == kDh ? kGuAhead + 1 : 1][4], ubuf[KIND == kDh ? kGuAhead + 1 : 1][4];
    auto load_gu = [&](int piece) {
      const int col = min(nb * kTile + nh * 128 + (piece & 3) * 32 + eu * 4, p.I - 4);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int row = row0 + max(min(mh * 128 + (piece >> 2) * 32 + er + 8 * t, rows - 1), 0);
        const uint16_t* src = p.gu + (size_t)row * 2 * p.I + col;
        gbuf[piece % (kGuAhead + 1)][t] = *reinterpret_cast<const uint2*>(src);
        ubuf[piece % (kGuAhead + 1)][t] = *reinterpret_cast<const uint2*>(src + p.I);
      }
    };
    if constexpr (KIND == kDh) {
#pragma unroll
      for (int i = 0; i < kGuAhead; ++i) load_gu(i);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int lr = mh * 128 + i * 32;  // first of these 32 rows in the tile
      if constexpr (W) {
        const int m0 = (place >> 16) * kTile + lr;
        if (m0 >= p.M) continue;  // M is a multiple of 32: all rows or none
        const size_t out0 = (size_t)entry(r, 0) * p.M * p.N;
        if constexpr (F32) {
          if (accumulate && rows <= 0) continue;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            keep(acc[i][j]);
            const int col = nb * kTile + nh * 128 + j * 32 + eu * 4;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              epi_put16(ep, lane, 2 * q + (lane >> 5),
                        __builtin_bit_cast(uint4, f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                                        acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]}));
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint4 v = epi_get(ep, lane, t);
              if (col >= p.N) continue;
              f32x4* dst = reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + out0 +
                                                    (size_t)(m0 + er + 8 * t) * p.N + col);
              f32x4 w = __builtin_bit_cast(f32x4, v);
              if (accumulate) w += *dst;
              *dst = w;
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            keep(acc[i][j]);
            keep(acc[i][j + 1]);
            const int col = nb * kTile + nh * 128 + j * 32 + eu * 8;
#pragma unroll
            for (int jj = 0; jj < 2; ++jj)
#pragma unroll
              for (int q = 0; q < 4; ++q) epi_put8(ep, lane, jj * 4 + q, pack4(acc[i][j + jj], q));
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint4 v = epi_get(ep, lane, t);
              if (col < p.N)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + out0 +
                                          (size_t)(m0 + er + 8 * t) * p.N + col) = v;
            }
          }
        }
      } else if constexpr (KIND == kDown || KIND == kDx) {
        if (lr >= rows) continue;
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          keep(acc[i][j]);
          keep(acc[i][j + 1]);
          const int col = nb * kTile + nh * 128 + j * 32 + eu * 8;
#pragma unroll
          for (int jj = 0; jj < 2; ++jj)
#pragma unroll
            for (int q = 0; q < 4; ++q) epi_put8(ep, lane, jj * 4 + q, pack4(acc[i][j + jj], q));
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint4 v = epi_get(ep, lane, t);
            if (col < p.N && lr + er + 8 * t < rows)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) +
                                        (size_t)(row0 + lr + er + 8 * t) * p.N + col) = v;
          }
        }
      } else if constexpr (KIND == kGateUp) {
        if (lr >= rows) continue;
        const int col = nb * COLS + nh * 64 + eu * 8;
#pragma unroll
        for (int part = 0; part < 3; ++part) {  // gate, up, h
#pragma unroll
          for (int j = 0; j < 4; ++j) keep(acc[i][j]);
#pragma unroll
          for (int jj = 0; jj < 2; ++jj)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint2 v;
              if (part < 2) {
                v = pack4(acc[i][2 * part + jj], q);
              } else {
                float h[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) h[t] = swiglu(acc[i][jj][4 * q + t], acc[i][2 + jj][4 * q + t]);
                v = uint2{bf16_pack2(h[0], h[1]), bf16_pack2(h[2], h[3])};
              }
              epi_put8(ep, lane, jj * 4 + q, v);
            }
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint4 v = epi_get(ep, lane, t);
            if (col >= p.N || lr + er + 8 * t >= rows) continue;
            const size_t row = (size_t)(row0 + lr + er + 8 * t);
            uint16_t* dst = part == 2 ? static_cast<uint16_t*>(p.out) + row * p.I + col
                                      : p.out2 + row * 2 * p.I + part * p.I + col;
            *reinterpret_cast<uint4*>(dst) = v;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (i * 4 + j + kGuAhead < 16) load_gu(i * 4 + j + kGuAhead);
          if (lr >= rows) continue;
          keep(acc[i][j]);
          const int col = nb * kTile + nh * 128 + j * 32 + eu * 4;
          const uint2(&gw)[4] = gbuf[(i * 4 + j) % (kGuAhead + 1)];
          const uint2(&uw)[4] = ubuf[(i * 4 + j) % (kGuAhead + 1)];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            epi_put16(ep, lane, 2 * q + (lane >> 5),
                      __builtin_bit_cast(uint4, f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                                      acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]}));
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const f32x4 dh = __builtin_bit_cast(f32x4, epi_get(ep, lane, t));
            if (col >= p.N || lr + er + 8 * t >= rows) continue;
            const GradSwiglu d = grad_swiglu(dh, gw[t], uw[t]);
            const size_t row = (size_t)(row0 + lr + er + 8 * t);
            auto put = [](uint16_t* d, const float* f) {
              *reinterpret_cast<uint2*>(d) = uint2{bf16_pack2(f[0], f[1]), bf16_pack2(f[2], f[3])};
            };
            put(static_cast<uint16_t*>(p.out) + row * p.I + col, d.h);
            put(p.out2 + row * 2 * p.I + col, d.dg);
            put(p.out2 + row * 2 * p.I + p.I + col, d.du);
          }
        }
      }
    }
  }
  MOE_DMA_SYNC(0);  // nothing on its way into this workgroup's LDS any more
}

// ---------------------------------------------------------------------------
// The same products in tiles of 64 x 64 or 128 x 128 on 4 waves of 32 x 32 or 64 x 64, K in blocks
// of 64 through a ring of stages: for few rows or small layers, where 256 x 256 tiles would leave
// most compute units idle and run through their K blocks one after another.  Two workgroups
// share a compute unit, with four stages of 16 KB or two of 32 KB each; a block is read for a
// quarter or half of the MFMAs that the large tiles make of it, so latency and the LDS bound them.
//   Measured (averages of a kernel trace): FFN of 64 tokens over 2 of 8 experts of 256 x 128 6.9 + 4.3 us;
// gradient of 777 tokens over 3 of 13 of 1024 x 384 13.9 us (dh) + 32.6 (the rest), 76 MB and 11 GFLOP: 16 us
// at a copy's rate.  (Without the trace a call takes 41 to 45 us, back to back.)
// ---------------------------------------------------------------------------
constexpr int kIds = 16;  // blocks of gathered rows in LDS

template <int S>
struct Small {
  // 64 KB for two workgroups on a compute unit: one (three stages of 32 KB) measured slower where
  // there are many (weight gradients of 1024 tokens, 2 of 8 experts of 2048 x 1024: 68 against 85 us)
  static constexpr int kRing = S == 64 ? 4 : 2;
  static constexpr int kB = S * kBK * 2;             // bytes of an operand's block
  static constexpr int kPieces = kB / 1024 / kNW;    // 1 KB copies of it per wave
  static constexpr int kSub = S / 64;                // 32 x 32 subtiles of a wave along each side
};

template <int S>
struct SmallLds {
  uint8_t a[Small<S>::kRing][Small<S>::kB];  // behind the loop: 4 KB per wave for the results
  uint8_t b[Small<S>::kRing][Small<S>::kB];
  int ids[kIds][kBK];  // weights, gathered: the rows of K
};

// Tile `block` of a product (rows: of those on XCD block % 8).
template <int S, Kind KIND, bool F32, bool GATHER, bool TWO>
__device__ __forceinline__ void small_tile(const TrainArgs& p, int accumulate, unsigned block,
                                           SmallLds<S>& lds) {
  constexpr int kSmall = S, kRing = Small<S>::kRing, kSmallCopies = Small<S>::kPieces, SUB = Small<S>::kSub;
  constexpr bool W = KIND == kWeights;
  constexpr bool BT = W || KIND == kDh || KIND == kDx;
  constexpr int COLS = KIND == kGateUp ? kSmall / 2 : kSmall;
  using OA = Operand<W ? kByCols : kRows>;
  using OB = Operand<BT ? kByCols : kRows>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int mh = wave >> 1, nh = wave & 1;
  int e, row0, rows, mb = 0, nb;
  if constexpr (W) {
    const unsigned per_e = (unsigned)p.mt * (unsigned)p.nnb;
    e = (int)(block / per_e);
    const int v = (int)(block % per_e);
    mb = v / p.nnb;
    nb = v - mb * p.nnb;
    rows = p.counts[e];
    row0 = p.offsets[e];
    dbg_segment(row0, rows, p.A);
    rows = __builtin_amdgcn_readfirstlane(max(rows, 0));
    row0 = __builtin_amdgcn_readfirstlane(row0);
    // without rows: zeros (gradient of 8 tokens over 22 experts of 2304 x 640, k = 1: 65.0 us a call, with the
    // epilogue of a tile of zeros 67.6).  M and N
    // are multiples of 128, so the tile is whole.
    if (rows == 0) {
      if (accumulate) return;
      constexpr int kUnits = S * (F32 ? 4 : 2) / 16;  // 16 bytes each, of a row
      uint8_t* out = static_cast<uint8_t*>(p.out) + (((size_t)e * p.M + mb * S) * p.N + nb * S) * (F32 ? 4 : 2);
      for (int i = tid; i < S * kUnits; i += 64 * kNW)
        *reinterpret_cast<uint4*>(out + (size_t)(i / kUnits) * p.N * (F32 ? 4 : 2) + i % kUnits * 16) = uint4{0, 0, 0, 0};
      return;
    }
  } else {
    RowTiles<kSmall> t;
    const int mt = t.load(p.counts, p.offsets, p.E, lane);
    const int G = mt * p.nnb, per = (G + kXcds - 1) / kXcds;
    const int x = (int)block % kXcds, i = (int)block / kXcds;
    if (i >= per || x * per + i >= G) return;
    int tile;
    panel_tile(x * per + i, mt, p.nnb, tile, nb);
    RowTile r = t.at(tile);
    e = r.e;
    row0 = r.row0;
    rows = r.rows;
    dbg_segment(row0, rows, p.A);
    if (rows <= 0) return;  // only where the debug check took them away
  }
  const int K = W ? rows : p.K, nk = (K + kBK - 1) / kBK;
  // TWO: one operand is in two parts, once over K with each
  const int nblk = TWO && KIND != kGateUp && KIND != kDh ? 2 * nk : nk;
  auto k_block = [&](int c) { return TWO && c >= nk ? c - nk : c; };

  // this wave's pieces: kSmallCopies of a and of b
  const uint8_t *asrc, *bsrc;
  uint32_t ao[kSmallCopies], bo[kSmallCopies];
  int ak[kSmallCopies], bk[kSmallCopies];  // weights: K of the lane's part
#pragma unroll
  for (int q = 0; q < kSmallCopies; ++q) {
    const int n = wave * kSmallCopies + q;
    ak[q] = OA::k_of(n, lane);
    bk[q] = OB::k_of(n, lane);
    if constexpr (W) {
      ao[q] = (uint32_t)min(mb * kSmall + OA::row_of(n, lane), p.M - 8) * 2;
      bo[q] = (uint32_t)min(nb * kSmall + OB::row_of(n, lane), p.N - 8) * 2;
    } else {
      const int r = min(OA::row_of(n, lane), rows - 1);
      const uint32_t row = GATHER
          ? token_of((uint32_t)dbg_clamp(p.sorted_idx[row0 + r], p.A, kDbgSorted), p) : (uint32_t)r;
      ao[q] = row * (uint32_t)(p.K * 2) + (uint32_t)ak[q] * 2;
      const int c = OB::row_of(n, lane);
      if constexpr (BT) {
        bo[q] = (uint32_t)bk[q] * (uint32_t)(p.N * 2) + (uint32_t)min(nb * kSmall + c, p.N - 8) * 2;
      } else if constexpr (KIND == kGateUp) {  // a wave's 32 weight rows: 16 gate rows, their up rows
        const int col = min(nb * COLS + (c >> 5) * 16 + (c & 15), p.N - 1);
        bo[q] = (uint32_t)((c & 16) ? p.I + col : col) * (uint32_t)(p.K * 2) + (uint32_t)bk[q] * 2;
      } else {
        bo[q] = (uint32_t)min(nb * kSmall + c, p.N - 1) * (uint32_t)(p.K * 2) + (uint32_t)bk[q] * 2;
      }
    }
  }
  if constexpr (W) {
    asrc = p.a + (size_t)row0 * p.M * 2;
    bsrc = GATHER ? p.b : p.b + (size_t)row0 * p.N * 2;
  } else {
    asrc = GATHER ? p.a : p.a + (size_t)row0 * p.K * 2;
    bsrc = p.b + (size_t)e * p.stride;
  }
  auto issue_ids = [&](int c) {
    if (wave == 0) {
      const int first = min(k_block(min(c, nblk - 1)) * kBK, rows - 1);  // behind the last block: not used
      dma4(reinterpret_cast<const uint8_t*>(p.sorted_idx + row0 + first),
           (uint32_t)min(lane, rows - 1 - first) * 4u, lds.ids[c % kIds]);
    }
  };
  // Block c into its stage; behind the last block the last one again (nobody reads it).
  auto issue = [&](int c) {
    const int st = c % kRing, at = min(c, nblk - 1), b = k_block(at);
    const uint8_t* a0 = asrc + (TWO && at >= nk ? p.a_rest : 0);
    const uint8_t* b0 = bsrc + (TWO && at >= nk ? p.b_rest : 0);
#pragma unroll
    for (int q = 0; q < kSmallCopies; ++q) {
      const int n = wave * kSmallCopies + q;
      if constexpr (W) {
        const int last = min(K - b * kBK, kBK) - 1;  // rows past the segment: its last one
        dma16(a0 + (size_t)b * kBK * p.M * 2, ao[q] + (uint32_t)min(ak[q], last) * (uint32_t)(p.M * 2),
              lds.a[st] + n * 1024);
        uint32_t row = (uint32_t)min(bk[q], last);
        if (GATHER) row = token_of((uint32_t)dbg_clamp(lds.ids[at % kIds][row], p.A, kDbgSorted), p);
        dma16(GATHER ? b0 : b0 + (size_t)b * kBK * p.N * 2, bo[q] + row * (uint32_t)(p.N * 2),
              lds.b[st] + n * 1024);
      } else {
        dma16(a0 + (size_t)b * kBK * 2, ao[q], lds.a[st] + n * 1024);
        dma16(b0 + (BT ? (size_t)b * kBK * p.N * 2 : (size_t)b * kBK * 2), bo[q], lds.b[st] + n * 1024);
      }
    }
  };

  f32x16 acc[SUB][SUB];
#pragma unroll
  for (int i = 0; i < SUB; ++i)
#pragma unroll
    for (int j = 0; j < SUB; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
  // subtile i of this wave is the tile's mh * SUB + i (columns: nh * SUB + j)
  int aa[SUB], ba[SUB];
#pragma unroll
  for (int i = 0; i < SUB; ++i) {
    aa[i] = OA::addr(0, mh * SUB + i, lane);
    ba[i] = OB::addr(0, nh * SUB + i, lane);
  }
  const int er = lane >> 3, eu = lane & 7;
  // first row and column of the results of subtile (i, j)
  auto row_at = [&](int i) { return (mh * SUB + i) * 32; };
  auto col_at = [&](int j) {
    return KIND == kGateUp ? nb * COLS + (nh * SUB + j) * 16 : nb * kSmall + (nh * SUB + j) * 32;
  };
  // kDh: gate_up of the wave's results, on its way while they are summed
  uint2 gw[KIND == kDh ? SUB : 1][SUB][4], uw[KIND == kDh ? SUB : 1][SUB][4];
  if constexpr (KIND == kDh) {
#pragma unroll
    for (int i = 0; i < SUB; ++i)
#pragma unroll
      for (int j = 0; j < SUB; ++j)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int r = row0 + min(row_at(i) + er + 8 * t, rows - 1);
          const uint16_t* src = p.gu + (size_t)r * 2 * p.I + min(col_at(j) + eu * 4, p.I - 4);
          gw[i][j][t] = *reinterpret_cast<const uint2*>(src);
          uw[i][j][t] = *reinterpret_cast<const uint2*>(src + p.I);
        }
  }
  if (nblk > 0) {
    if constexpr (W && GATHER) {
      for (int c = 0; c < 2 * kRing; ++c) issue_ids(c);
      MOE_DMA_SYNC(0);
    }
#pragma unroll
    for (int c = 0; c < kRing - 1; ++c) issue(c);
    for (int c = 0; c < nblk; ++c) {
      // block c has landed, every wave has read block c - 1
      MOE_DMA_SYNC((kRing - 2) * 2 * kSmallCopies);
      if constexpr (W && GATHER) issue_ids(c + 2 * kRing);
      issue(c + kRing - 1);
      uint8_t *sa = lds.a[c % kRing], *sb = lds.b[c % kRing];
      if constexpr (W) {
        const int left = K - k_block(c) * kBK;
        if (left < kBK) {  // zeros past the segment's end
          for (int i = tid; i < (kBK - left) * 8; i += 64 * kNW)
#pragma unroll
            for (int c64 = 0; c64 < SUB; ++c64) {
              *reinterpret_cast<uint4*>(sa + c64 * 8192 + left * 128 + i * 16) = uint4{0, 0, 0, 0};
              *reinterpret_cast<uint4*>(sb + c64 * 8192 + left * 128 + i * 16) = uint4{0, 0, 0, 0};
            }
          __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(63));
          asm volatile("s_barrier" ::: "memory");
        }
      }
      bf16x8 af[2][SUB], bf[2][SUB];
      auto get = [&](int step) {
        // a subtile's place is in the address (K strided: but the 64 columns) or added by frag
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
          af[step & 1][i] = OA::frag(sa, aa[i], mh * SUB + i, step);
          bf[step & 1][i] = OB::frag(sb, ba[i], nh * SUB + i, step);
        }
      };
      get(0);
#pragma unroll
      for (int step = 0; step < 4; ++step) {
        if (step < 3) get(step + 1);
#pragma unroll
        for (int i = 0; i < SUB; ++i)
#pragma unroll
          for (int j = 0; j < SUB; ++j) acc[i][j] = mfma32(bf[step & 1][j], af[step & 1][i], acc[i][j]);
      }
    }
    MOE_DMA_SYNC(0);  // nothing on its way any more, every wave is done reading: the stages are free
  }

  // -- epilogue: the wave's 32 x 32 results as rows ---------------------------------------------------
  uint8_t* ep = lds.a[0] + wave * kEpiB;
  static_assert(kRing * Small<S>::kB >= kNW * kEpiB, "room for the results");
  // put: four bf16 values; put2: TWO: in two parts, `rest` bytes apart.  The first is cut, so that the second
  // has its sign (or stands for nothing at 2^-20 of it): an infinity that meets them stays one.
  auto put = [](uint16_t* d, const float* f) {
    *reinterpret_cast<uint2*>(d) = uint2{bf16_pack2(f[0], f[1]), bf16_pack2(f[2], f[3])};
  };
  auto put2 = [&](uint16_t* d, const float* f, int64_t rest) {
    if constexpr (!TWO) {
      put(d, f);
      return;
    }
    uint32_t hi[4];
    float lo[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      hi[x] = __float_as_uint(f[x]) & 0xffff0000u;
      const float h = __uint_as_float(hi[x]), r = f[x] - h;
      lo[x] = fabsf(r) > 0.f ? r : h * 0x1p-20f;  // also of infinities (r is NaN)
      if (f[x] != f[x]) hi[x] |= 0x00400000u;     // a NaN whose cut bits alone said so
    }
    *reinterpret_cast<uint2*>(d) = uint2{hi[0] >> 16 | hi[1], hi[2] >> 16 | hi[3]};
    *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(d) + rest) =
        uint2{bf16_pack2(lo[0], lo[1]), bf16_pack2(lo[2], lo[3])};
  };
  // bf16 rows of 64 columns at 16 bytes a lane (8 bytes of 32 columns, as below: a call for the gradient of 777
  // tokens, 3 of 13 experts of 1024 x 384, 46.7 instead of 44.9 us)
  if constexpr (SUB == 2 && !F32 && (W || KIND == kDown || KIND == kDx)) {
#pragma unroll
    for (int i = 0; i < SUB; ++i) {
#pragma unroll
      for (int j = 0; j < SUB; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) epi_put8(ep, lane, j * 4 + q, pack4(acc[i][j], q));
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint4 v = epi_get(ep, lane, t);
        const int lr = row_at(i) + er + 8 * t, col = col_at(0) + eu * 8;
        if (W ? mb * kSmall + lr >= p.M : lr >= rows) continue;
        if (col >= p.N) continue;
        const size_t row = W ? (size_t)e * p.M + mb * kSmall + lr : (size_t)(row0 + lr);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * p.N + col) = v;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < SUB; ++i)
#pragma unroll
    for (int j = 0; j < SUB; ++j) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        epi_put16(ep, lane, 2 * q + (lane >> 5),
                  __builtin_bit_cast(uint4, f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                                  acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]}));
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int lr = row_at(i) + er + 8 * t, col0 = col_at(j);
        f32x4 v = __builtin_bit_cast(f32x4, epi_get(ep, lane, t));
        if constexpr (W) {
          const int m = mb * kSmall + lr, col = col0 + eu * 4;
          if (m >= p.M || col >= p.N) continue;
          const size_t at = ((size_t)e * p.M + m) * p.N + col;
          if constexpr (F32) {
            f32x4* dst = reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + at);
            if (accumulate) v += *dst;
            *dst = v;
          } else {
            const float f[4] = {v[0], v[1], v[2], v[3]};
            put(static_cast<uint16_t*>(p.out) + at, f);
          }
        } else if constexpr (KIND == kGateUp) {
          // lanes 0..3 of a row hold 16 gate values, lanes 4..7 the up values of the same columns
          float u[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) u[x] = __shfl_xor(v[x], 4, 64);
          const int col = col0 + (eu & 3) * 4;
          if (lr >= rows || col >= p.N) continue;
          const size_t row = (size_t)(row0 + lr);
          const float f[4] = {v[0], v[1], v[2], v[3]};
          put(p.out2 + row * 2 * p.I + (eu & 4 ? p.I : 0) + col, f);
          if (eu & 4) continue;
          float h[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) h[x] = swiglu(v[x], u[x]);
          put2(static_cast<uint16_t*>(p.out) + row * p.I + col, h, p.out_rest);
        } else {
          const int col = col0 + eu * 4;
          if (lr >= rows || col >= p.N) continue;
          const size_t row = (size_t)(row0 + lr);
          if constexpr (KIND == kDh) {
            const GradSwiglu d = grad_swiglu(v, gw[i][j][t], uw[i][j][t]);
            put2(static_cast<uint16_t*>(p.out) + row * p.I + col, d.h, p.out_rest);
            put2(p.out2 + row * 2 * p.I + col, d.dg, p.out2_rest);
            put2(p.out2 + row * 2 * p.I + p.I + col, d.du, p.out2_rest);
          } else {
            const float f[4] = {v[0], v[1], v[2], v[3]};
            put(static_cast<uint16_t*>(p.out) + row * p.N + col, f);
          }
        }
      }
    }
}

template <int S, Kind KIND, bool GATHER, bool TWO>
__global__ __launch_bounds__(64 * kNW, 2) void train_small_kernel(TrainArgs p) {
  __shared__ SmallLds<S> lds;
  small_tile<S, KIND, false, GATHER, TWO>(p, 0, blockIdx.x, lds);
}

// The gradient's three products behind dh - dx, dW13, dWd - do not depend on each other: what
// takes small tiles of them runs as one launch, so that they fill the chip together (777 tokens
// over 13 experts of 1024 x 384: 45 us one after another, 33 in one; with dx, whose tiles have most
// blocks, last in the launch: 36).
struct SmallJob {
  TrainArgs p;
  unsigned blocks;  // 0: not in this launch
  int side;         // 64 or 128
};

// GATHER: the rows of dW13's x.
template <bool F32, bool GATHER, bool TWO>
__global__ __launch_bounds__(64 * kNW, 2) void train_rest_kernel(SmallJob dx, SmallJob w13, SmallJob w2,
                                                                 int accumulate) {
  __shared__ union {
    SmallLds<64> s64;
    SmallLds<128> s128;
  } lds;
  unsigned b = blockIdx.x;
  if (b < dx.blocks) {
    if (TWO || dx.side == 64) small_tile<64, kDx, false, false, TWO>(dx.p, 0, b, lds.s64);
    else small_tile<128, kDx, false, false, TWO>(dx.p, 0, b, lds.s128);
    return;
  }
  b -= dx.blocks;
  if (b < w13.blocks) {
    if (w13.side == 64) small_tile<64, kWeights, F32, GATHER, TWO>(w13.p, accumulate, b, lds.s64);
    else small_tile<128, kWeights, F32, GATHER, TWO>(w13.p, accumulate, b, lds.s128);
    return;
  }
  b -= w13.blocks;
  if (w2.side == 64) small_tile<64, kWeights, F32, false, TWO>(w2.p, accumulate, b, lds.s64);
  else small_tile<128, kWeights, F32, false, TWO>(w2.p, accumulate, b, lds.s128);
}

__global__ __launch_bounds__(256) void zero_kernel(uint4* out, size_t n) {
  for (size_t i = blockIdx.x * (size_t)256 + threadIdx.x; i < n; i += gridDim.x * (size_t)256)
    out[i] = uint4{0, 0, 0, 0};
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Workgroups for `tiles` tiles: one per compute unit, more where a list would overflow.
unsigned grid_of(int64_t tiles) {
  const int64_t per = (tiles + kXcds - 1) / kXcds;
  int64_t n = per < kXcdCus ? per : kXcdCus;
  if (n * kListTiles < per) n = (per + kListTiles - 1) / kListTiles;
  return (unsigned)(n * kXcds);
}

// Which tiles: those of 256 x 256 where there are enough to fill the chip, then those of 128 x 128,
// else those of 64 x 64.  Measured (us, 64 / 128 / 256; the row products' tiles are counted as
// as many as the rows fill and half a one per expert):
//   forward of 1024 tokens, 2 of 8 experts of 2048 x 1024 (96 tiles of 256 per product, 320 of 128):
//     68 / 55 / 77;  of 2048 (160, 576): 115 / 95 / 80;  of 8192, 2 of 8 of 512 x 256 (136, 528):
//     58 / 48 / 40;  of 777, 3 of 13 of 1024 x 384 (48 and 64, 150 and 200): 26 / 29 / 48
//   weight gradients of 1024 tokens, 2 of 8 of 2048 x 1024 (512 and 256 tiles of 256): 103 / 68 / 53;
//     of 777, 3 of 13 of 1024 x 384 (156 and 104, 624 and 312 of 128): 36 / 30 / 43;  of 8192, 2 of 8
//     of 512 x 256 (32 and 16, 128 and 64): 56 / 84 / 156
constexpr int64_t kRowTiles256 = 128, kRowTiles128 = 300, kWeightTiles256 = 200, kWeightTiles128 = 256;
// Experts of few rows: 256 rows would be mostly padding up to 64 rows an expert, where the weights'
// bytes bound the product (1024 tokens, 4 of 64 experts of 2048 x 1024: 245 / 232 / 252; at 128
// rows an expert, 2048 of them, 345 / - / 270), and 128 rows up to 16 (16 tokens, 8 of 256 of
// 2048 x 512: 118 / 135 / 150).
constexpr int64_t kRows256 = 64, kRows128 = 16;

// Small batches keep h, dg and du in two bf16 parts, up to this many rows and values of h: with few of them
// a handful carries a result's norm, and how their rounding falls shows in it.  Worst error of 24 batches
// each, over layers of 256 to 4096 x 128 to 1024, in errors of a result rounded once, one part / two: 4 rows
// 1.78 / 1.10, 16 rows 1.68, 32 rows 1.58, 48 rows 1.53, 64 to 96 rows 1.51, 112 and 128 rows 1.52, more 1.49; by
// values of h up to 8192 1.68, up to 16384 1.53, up to 32768 1.51, more 1.49 (1.42 in the mean at any size;
// two parts never above 1.05 from 16 rows on).  So the border stands where the worst batch comes down
// to within a tenth of the mean.  What two parts cost, the same layers: the forward 1.03 to 1.35 times,
// the gradient 0.87 to 1.6 times (below 1 where one part takes larger tiles).  us a call, one part / two:
// forward and gradient of 3 tokens over 2 experts of 256 x 512 11.9 14.2 / 13.0 18.1, of 8 over 22 of
// 2304 x 640 19.2 87 / 21.5 65.
constexpr int kTwoRows = 96, kTwoValues = 32768;

// Rows of a workspace for A rows that have second parts (smaller batches may run in it).
size_t two_part_rows(size_t A, int I) {
  const size_t most = kTwoValues / I < kTwoRows ? kTwoValues / I : kTwoRows;
  return A < most ? A : most;
}
bool in_two_parts(const TrainArgs& p) { return two_part_rows((size_t)p.A, p.I) == (size_t)p.A; }

// Tiles of a product: their side and how many workgroups.  Sets the arguments' counts of tiles.
struct Tiling {
  int side;
  unsigned grid;
};

template <Kind KIND>
Tiling tile_rows(TrainArgs& p) {
  constexpr int kShare = KIND == kGateUp ? 2 : 1;  // weight rows of an output column
  const int64_t touched = p.A < p.E ? p.A : p.E;
  auto columns = [&](int side) { return p.nnb = (p.N * kShare + side - 1) / side; };
  // as many row tiles as rows fill, and half a tile per expert
  auto about = [&](int side) { return (p.A / side + (touched + 1) / 2) * (int64_t)columns(side); };
  auto at_most = [&](int side) { return row_tiles_bound(p.A, p.E, side) * columns(side); };
  const bool two = in_two_parts(p);
  if (!two && about(kTile) >= kRowTiles256 && p.A > kRows256 * touched)
    return {kTile, grid_of(at_most(kTile))};
  const int side = !two && about(128) >= kRowTiles128 && p.A >= kRows128 * touched ? 128 : 64;
  return {side, (unsigned)((at_most(side) + kXcds - 1) / kXcds * kXcds)};
}

Tiling tile_weights(TrainArgs& p) {
  auto tiles = [&](int side) {
    p.mt = (p.M + side - 1) / side;
    p.nnb = (p.N + side - 1) / side;
    return (int64_t)p.E * p.mt * p.nnb;
  };
  const int64_t n = tiles(kTile);
  if (n >= kWeightTiles256 && !in_two_parts(p)) {
    // an XCD's tiles come in whole groups, and a workgroup's list holds one of each group or, of
    // more than fit there, of some
    const int64_t groups = (n + kXcdCus - 1) / kXcdCus;
    return {kTile, grid_of((groups + kXcds - 1) / kXcds * kXcds * kXcdCus)};
  }
  const int64_t mid = tiles(128);
  if (mid >= kWeightTiles128) return {128, (unsigned)mid};
  return {64, (unsigned)tiles(64)};
}

// The forward's products and dh.
template <Kind KIND>
int launch_rows(TrainArgs p, hipStream_t s, const char* who) {
  const Tiling t = tile_rows<KIND>(p);
  auto launch = [&](auto gather) {
    constexpr bool G = decltype(gather)::value;
    if (t.side == kTile) train_gemm_kernel<KIND, false, G><<<t.grid, 64 * kNW, 0, s>>>(p, 0);
    else if (t.side == 128) train_small_kernel<128, KIND, G, false><<<t.grid, 64 * kNW, 0, s>>>(p);
    else if (!in_two_parts(p)) train_small_kernel<64, KIND, G, false><<<t.grid, 64 * kNW, 0, s>>>(p);
    else train_small_kernel<64, KIND, G, true><<<t.grid, 64 * kNW, 0, s>>>(p);
    return check_launch(who);
  };
  if constexpr (KIND == kGateUp)
    if (p.sorted_idx) return launch(std::true_type{});
  return launch(std::false_type{});
}

// The gradient's products behind dh: those of large tiles by themselves, the others together.
struct Rest {
  SmallJob dx{}, w13{}, w2{};
};

int launch_rest(Rest& r, bool two, bool f32, int accumulate, hipStream_t s, const char* who) {
  bool any = false;
  auto large = [&](SmallJob& j, const Tiling& t) {
    j.side = t.side;
    j.blocks = t.side == kTile ? 0 : t.grid;
    any |= j.blocks != 0;
    return t.side == kTile;
  };
  if (r.dx.p.out) {
    const Tiling t = tile_rows<kDx>(r.dx.p);
    if (large(r.dx, t)) {
      train_gemm_kernel<kDx, false, false><<<t.grid, 64 * kNW, 0, s>>>(r.dx.p, 0);
      if (int st = check_launch(who)) return st;
    }
  }
  const std::true_type yes;
  const std::false_type no;
  // kernels by the type of the weights' gradients and whether rows are gathered
  auto pick = [&](const int32_t* gathered, auto f) {
    return f32 ? (gathered ? f(yes, yes) : f(yes, no)) : (gathered ? f(no, yes) : f(no, no));
  };
  for (SmallJob* j : {&r.w13, &r.w2}) {
    if (!j->p.out) continue;
    const Tiling t = tile_weights(j->p);
    if (!large(*j, t)) continue;
    const int st = pick(j->p.sorted_idx, [&](auto as_f32, auto gather) {
      train_gemm_kernel<kWeights, decltype(as_f32)::value, decltype(gather)::value>
          <<<t.grid, 64 * kNW, 0, s>>>(j->p, accumulate);
      return check_launch(who);
    });
    if (st) return st;
  }
  if (!any) return MOE_OK;
  return pick(r.w13.p.sorted_idx, [&](auto as_f32, auto gather) {
    auto launch = [&](auto kernel) {
      kernel<<<r.dx.blocks + r.w13.blocks + r.w2.blocks, 64 * kNW, 0, s>>>(r.dx, r.w13, r.w2, accumulate);
      return check_launch(who);
    };
    constexpr bool F = decltype(as_f32)::value, G = decltype(gather)::value;
    return two ? launch(train_rest_kernel<F, G, true>) : launch(train_rest_kernel<F, G, false>);
  });
}

int check_train(const char* who, const moe_experts* W, int32_t T, int32_t k, bool gathered, Layout* Lo) {
  if (!W) return set_error(MOE_ERR_INVALID_ARG, "%s: W is NULL", who);
  if (W->fmt != MOE_W_BF16 || !layout_of(W->fmt, W->H, W->I, Lo))
    return set_error(MOE_ERR_UNSUPPORTED, "%s: needs BF16 records, H and I multiples of 128 in "
                     "[128, 16384] (fmt=%d H=%d I=%d)", who, W->fmt, W->H, W->I);
  if (W->E < 1 || W->E > kMaxE || T < 0 || k < 1 || k > kMaxK)
    return set_error(MOE_ERR_INVALID_ARG, "%s: need 1<=E<=%d, T>=0, 1<=k<=%d (E=%d T=%d k=%d)", who,
                     kMaxE, kMaxK, W->E, T, k);
  if (W->stride != Lo->stride)
    return set_error(MOE_ERR_INVALID_ARG, "%s: stride %lld, expected %lld", who, (long long)W->stride,
                     (long long)Lo->stride);
  if ((int64_t)T * k > (int64_t)1 << 27)
    return set_error(MOE_ERR_UNSUPPORTED, "%s: T*k > 2^27", who);
  if (gathered && (int64_t)T * W->H * 2 >= (int64_t)1 << 32)
    return set_error(MOE_ERR_UNSUPPORTED, "%s: T*H >= 2^31 with sorted_idx (gather the rows with "
                     "moe_dispatch and pass NULL)", who);
  return MOE_OK;
}

bool bad(const void* p) { return !p || !aligned16(p); }

TrainArgs args_of(const moe_experts* W, int32_t T, int32_t k, const int32_t* counts,
                  const int32_t* offsets) {
  TrainArgs p{};
  p.E = W->E; p.I = W->I; p.k = k; p.A = T * k;
  p.counts = counts; p.offsets = offsets; p.stride = W->stride;
  p.k_magic = k > 1 ? (uint32_t)((1ull << 32) / k + 1) : 0;
  return p;
}

}  // namespace

#ifdef MOE_DEBUG
uint32_t dbg_take_train() { return dbg_take_unit(); }
#endif

}  // namespace moe

using namespace moe;

// Workspace: h bf16 [T*k][I], and the second parts of a small batch's.
extern "C" size_t moe_expert_ffn_train_workspace(const moe_experts* W, int32_t T, int32_t k) {
  if (!W || T < 0 || k < 1 || W->I < 1) return 0;
  const size_t A = (size_t)T * k;
  return align256(A * W->I * 2) + align256(two_part_rows(A, W->I) * W->I * 2);
}

extern "C" int moe_expert_ffn_train(const moe_experts* W, const uint16_t* x, int32_t T, int32_t k,
                                    const int32_t* counts, const int32_t* offsets,
                                    const int32_t* sorted_idx, uint16_t* gate_up, uint16_t* y_perm,
                                    void* ws, size_t ws_bytes, moe_stream_t stream) {
  const char* who = "moe_expert_ffn_train";
  Layout Lo;
  if (int st = check_train(who, W, T, k, sorted_idx != nullptr, &Lo)) return st;
  if (T == 0) return MOE_OK;
  if (bad(W->base) || bad(x) || bad(counts) || bad(offsets) || (sorted_idx && !aligned16(sorted_idx)) ||
      bad(gate_up) || bad(y_perm) || bad(ws))
    return set_error(MOE_ERR_INVALID_ARG, "%s: null or misaligned pointer", who);
  if (ws_bytes < moe_expert_ffn_train_workspace(W, T, k))
    return set_error(MOE_ERR_WORKSPACE, "%s: workspace %zu too small", who, ws_bytes);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  TrainArgs p = args_of(W, T, k, counts, offsets);
  p.sorted_idx = sorted_idx;
  p.b = static_cast<const uint8_t*>(W->base) + Lo.w13;
  p.a = reinterpret_cast<const uint8_t*>(x);
  p.K = W->H; p.N = W->I;
  p.out = ws; p.out2 = gate_up;
  const int64_t rest = in_two_parts(p) ? (int64_t)align256((size_t)p.A * W->I * 2) : 0;
  p.out_rest = rest;
  if (int st = launch_rows<kGateUp>(p, s, who)) return st;
  p.sorted_idx = nullptr;
  p.b = static_cast<const uint8_t*>(W->base) + Lo.w2;
  p.a = static_cast<const uint8_t*>(ws);
  p.K = W->I; p.N = W->H;
  p.out = y_perm; p.out2 = nullptr;
  p.a_rest = rest; p.out_rest = 0;
  return launch_rows<kDown>(p, s, who);
}

// Workspace: h bf16 [T*k][I], (dg; du) bf16 [T*k][2I], and their second parts.
extern "C" size_t moe_expert_ffn_backward_workspace(const moe_experts* W, int32_t T, int32_t k) {
  if (!W || T < 0 || k < 1 || W->I < 1) return 0;
  const size_t A = (size_t)T * k, two = two_part_rows(A, W->I);
  return align256(A * W->I * 2) + align256(A * W->I * 4) + align256(two * W->I * 2) + align256(two * W->I * 4);
}

extern "C" int moe_expert_ffn_backward(const moe_experts* W, const uint16_t* x, int32_t T, int32_t k,
                                       const int32_t* counts, const int32_t* offsets,
                                       const int32_t* sorted_idx, const uint16_t* gate_up,
                                       const uint16_t* d_y_perm, uint16_t* d_x_perm, void* d_w13,
                                       void* d_w2, int32_t d_w_type, int32_t accumulate, void* ws,
                                       size_t ws_bytes, moe_stream_t stream) {
  const char* who = "moe_expert_ffn_backward";
  Layout Lo;
  if (int st = check_train(who, W, T, k, sorted_idx != nullptr, &Lo)) return st;
  if (d_w_type != MOE_T_BF16 && d_w_type != MOE_T_F32)
    return set_error(MOE_ERR_UNSUPPORTED, "%s: weight gradients of type %d (bf16 or fp32)", who, d_w_type);
  if (accumulate && (d_w13 || d_w2) && d_w_type != MOE_T_F32)
    return set_error(MOE_ERR_UNSUPPORTED, "%s: only fp32 weight gradients accumulate", who);
  if ((d_w13 && !aligned16(d_w13)) || (d_w2 && !aligned16(d_w2)))
    return set_error(MOE_ERR_INVALID_ARG, "%s: misaligned pointer", who);
  if (T > 0) {
    if (bad(W->base) || bad(x) || bad(counts) || bad(offsets) || (sorted_idx && !aligned16(sorted_idx)) ||
        bad(gate_up) || bad(d_y_perm) || (d_x_perm && !aligned16(d_x_perm)) || bad(ws))
      return set_error(MOE_ERR_INVALID_ARG, "%s: null or misaligned pointer", who);
    if (ws_bytes < moe_expert_ffn_backward_workspace(W, T, k))
      return set_error(MOE_ERR_WORKSPACE, "%s: workspace %zu too small", who, ws_bytes);
  }
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int A = T * k, H = W->H, I = W->I;
  const size_t esize = d_w_type == MOE_T_F32 ? 4 : 2;
  if (T == 0) {
    auto zero = [&](void* out) {
      const size_t n = (size_t)W->E * (out == d_w13 ? 2 : 1) * I * H * esize / 16;
      zero_kernel<<<(unsigned)(n / 256 < 8192 ? n / 256 : 8192), 256, 0, s>>>(static_cast<uint4*>(out), n);
      return check_launch(who);
    };
    if (!accumulate && d_w13)
      if (int st = zero(d_w13)) return st;
    return !accumulate && d_w2 ? zero(d_w2) : MOE_OK;
  }
  if (!d_x_perm && !d_w13 && !d_w2) return MOE_OK;
  uint16_t* h = static_cast<uint16_t*>(ws);
  uint16_t* dgu = h + align256((size_t)A * I * 2) / 2;
  TrainArgs p = args_of(W, T, k, counts, offsets);
  p.b = static_cast<const uint8_t*>(W->base) + Lo.w2;
  p.a = reinterpret_cast<const uint8_t*>(d_y_perm);
  p.K = H; p.N = I;
  p.out = h; p.out2 = dgu; p.gu = gate_up;
  const bool two = in_two_parts(p);
  if (two) {  // the parts lie h, (dg; du), h's rest, (dg; du)'s rest
    const size_t hb = align256((size_t)A * I * 2), gb = align256((size_t)A * I * 4);
    p.out_rest = (int64_t)(hb + gb);
    p.out2_rest = (int64_t)(gb + hb);
  }
  const int64_t h_rest = p.out_rest, dgu_rest = p.out2_rest;
  if (int st = launch_rows<kDh>(p, s, who)) return st;
  Rest rest;
  p.out2 = nullptr; p.gu = nullptr;
  p.out_rest = p.out2_rest = 0;
  if (d_x_perm) {
    TrainArgs& q = rest.dx.p = p;
    q.b = static_cast<const uint8_t*>(W->base) + Lo.w13;
    q.a = reinterpret_cast<const uint8_t*>(dgu);
    q.K = 2 * I; q.N = H;
    q.out = d_x_perm;
    q.a_rest = dgu_rest;
  }
  if (d_w13) {
    TrainArgs& q = rest.w13.p = p;
    q.sorted_idx = sorted_idx;
    q.a = reinterpret_cast<const uint8_t*>(dgu);
    q.b = reinterpret_cast<const uint8_t*>(x);
    q.M = 2 * I; q.N = H; q.out = d_w13;
    q.a_rest = dgu_rest;
  }
  if (d_w2) {
    TrainArgs& q = rest.w2.p = p;
    q.a = reinterpret_cast<const uint8_t*>(d_y_perm);
    q.b = reinterpret_cast<const uint8_t*>(h);
    q.M = H; q.N = I; q.out = d_w2;
    q.b_rest = h_rest;
  }
  return launch_rest(rest, two, d_w_type == MOE_T_F32, accumulate, s, who);
}
