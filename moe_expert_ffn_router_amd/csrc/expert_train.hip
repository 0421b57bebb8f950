// Training of the experts (BF16 records): the SwiGLU FFN that keeps its gate and up products, and
// its gradient.  Rows p in expert order, expert e = that of the row:
//   forward   g = Wg x, u = Wu x (kept as bf16); h = silu(g) u;  y = Wd h
//   backward  dh = Wd^T dy, s = 1 / (1 + e^-g):  du = dh g s,  dg = dh u s (1 + g (1 - s)),
//             dx = W13^T (dg; du),  dW13 = sum_p (dg; du) x^T,  dWd = sum_p dy h^T
// Six grouped products on the 32x32x16 bf16 MFMA with fp32 accumulation, of two kinds:
//   rows     out[p][n] = sum_k A[p][k] B[n][k]: the forward's two (weights as stored, K contiguous)
//            and dh, dx (the weights' other index is summed over: K strided);
//   weights  out[e][m][n] = sum_(p of e) A[p][m] B[p][n]: both operands K strided.
// Roundings: h and (dg; du) go to bf16 once, as the operands of the next product; the forward's
// h comes from the fp32 gate and up sums, the gradient's from the kept bf16 ones.
//
// Tiles of BM x 256 outputs on 8 waves, 2 along the rows x 4 along the columns, K in blocks of
// 64, both operands copied from memory straight into LDS, two stages.  An operand with K
// contiguous lies as rows of 128 bytes, one with K strided as 64 rows of its tile's columns, read
// back through the transposing LDS loads.
#include "fp8_common.h"
#include "lds_copy.h"
#include "moe_internal.h"

namespace moe {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((__vector_size__(4 * sizeof(short)))) short i16x4;

constexpr int kBK = 64;   // K of a block
constexpr int kBN = 256;  // output columns of a tile
constexpr int kWM = 2, kWN = 4, kNW = kWM * kWN;
constexpr int kXcds = 8;
constexpr int kPanel = 4;  // row tiles that share weights in an XCD's L2

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// One operand of a tile in LDS: ROWS x 64 values.  STRIDED: [k][ROWS], 64-byte pieces of a row
// swizzled by k so that the transposing loads of 4 (k) x 32 values meet distinct banks;
// else [row][64], 16-byte units swizzled by row.
template <int ROWS, bool STRIDED>
struct Operand {
  static constexpr int kBytes = ROWS * kBK * 2;
  static constexpr int kCopies = kBytes / 1024 / kNW;  // 1 KB copies per wave
  static constexpr int kRowB = STRIDED ? ROWS * 2 : kBK * 2;
  static constexpr int kLanes = kRowB / 16;            // lanes (16-byte units) of a row
  static constexpr int kChunks = kRowB / 64;
  static_assert(kBytes % (1024 * kNW) == 0, "copies");

  // row of the stage that this lane's part of copy q fills
  static __device__ __forceinline__ int row_of(int wave, int q, int lane) {
    return (wave * kCopies + q) * (64 / kLanes) + lane / kLanes;
  }
  // which 16-byte unit of that row's source goes there
  static __device__ __forceinline__ int unit_of(int row, int lane) {
    const int u = lane % kLanes;
    if constexpr (STRIDED) return (((u >> 2) ^ swz(row)) << 2) | (u & 3);
    return u ^ a_swz(row);
  }
  static __device__ __forceinline__ int swz(int k) {
    return ((k & 3) ^ (((k >> 3) & 1) << 2)) & (kChunks - 1);
  }
  // the 8 values at K = 16 s + 8 (lane / 32) of row (column) block*32 + lane % 32
  static __device__ __forceinline__ bf16x8 frag(const uint8_t* st, int block, int s, int lane) {
    if constexpr (STRIDED) {
      const int i = lane & 15, hh = lane >> 5;
      const int k = 16 * s + 8 * hh + (i >> 2);
      const uint8_t* p = st + k * kRowB + ((block ^ swz(k)) << 6) + ((lane >> 4) & 1) * 32 + (i & 3) * 8;
      using lds_t = __attribute__((address_space(3))) i16x4;
      const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)p);
      const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)(p + 4 * kRowB));
      typedef __attribute__((__vector_size__(8 * sizeof(short)))) short i16x8;
      const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      return __builtin_bit_cast(bf16x8, v);
    } else {
      const int r = block * 32 + (lane & 31);
      return *reinterpret_cast<const bf16x8*>(st + r * kRowB + (((2 * s + (lane >> 5)) ^ a_swz(r)) << 4));
    }
  }
};

template <int BM, bool AT, bool BT>
struct Stage {
  uint8_t a[Operand<BM, AT>::kBytes];
  uint8_t b[Operand<kBN, BT>::kBytes];
};

// acc += the products of one block
template <int BM, bool AT, bool BT>
__device__ __forceinline__ void multiply(const Stage<BM, AT, BT>& st, int mh, int nh, int lane,
                                         f32x16 (&acc)[BM / 64][2]) {
  constexpr int MI = BM / 64;
  bf16x8 af[2][MI], bf[2][2];
  auto load = [&](int s) {
#pragma unroll
    for (int i = 0; i < MI; ++i) af[s & 1][i] = Operand<BM, AT>::frag(st.a, mh * MI + i, s, lane);
#pragma unroll
    for (int j = 0; j < 2; ++j) bf[s & 1][j] = Operand<kBN, BT>::frag(st.b, nh * 2 + j, s, lane);
  };
  load(0);
#pragma unroll
  for (int s = 0; s < kBK / 16; ++s) {
    if (s + 1 < kBK / 16) load(s + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma32(bf[s & 1][j], af[s & 1][i], acc[i][j]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Value 4q + r of acc[i][j] is output row 32 (mh MI + i) + lane % 32, column
// 32 (2 nh + j) + 8q + 4 (lane / 32) + r of the tile.
__device__ __forceinline__ void put4(uint16_t* p, const float* v) {
  *reinterpret_cast<uint2*>(p) = uint2{bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3])};
}

struct TrainArgs {
  int E, H, I, k, A;
  const int* counts;
  const int* offsets;
  const int* sorted_idx;  // rows of the gathered operand, NULL: in expert order
  const uint8_t* w;       // weights of expert 0
  int64_t stride;         // bytes between experts
  const uint8_t* a;       // bf16 [rows][K]
  int K, N;               // reduction length, output columns
  int nnb;                // column blocks
  uint16_t* out;          // rows: [A][N]; gated: h
  uint16_t* out2;         // gated: gate_up; dswiglu: (dg; du)
  const uint16_t* gu;     // dswiglu: gate_up
};

enum { kPlain, kGated, kDswiglu };

// v-th tile of mt row tiles x nnb column blocks: panels of kPanel row tiles, column by column
__device__ __forceinline__ void panel_tile(int v, int mt, int nnb, int& tile, int& nb) {
  const int panel = v / (kPanel * nnb), r = v - panel * (kPanel * nnb);
  const int rows = min(kPanel, mt - panel * kPanel);
  nb = r / rows;
  tile = panel * kPanel + r - nb * rows;
}

template <int BM, int MODE, bool BT>
__global__ __launch_bounds__(64 * kNW) void train_rows_kernel(TrainArgs p) {
  constexpr int MI = BM / 64;
  constexpr int COLS = MODE == kGated ? kBN / 2 : kBN;
  using OA = Operand<BM, false>;
  using OB = Operand<kBN, BT>;
  __shared__ Stage<BM, false, BT> st[2];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int mh = wave / kWN, nh = wave % kWN;
  RowTiles<BM> rt;
  const int mt = rt.load(p.counts, p.offsets, p.E, lane);
  const int G = mt * p.nnb, per = (G + kXcds - 1) / kXcds;
  const int x = (int)blockIdx.x % kXcds, i0 = (int)blockIdx.x / kXcds;
  const int v = x * per + i0;
  if (i0 >= per || v >= G) return;
  int tile, nb;
  panel_tile(v, mt, p.nnb, tile, nb);
  RowTile t = rt.at(tile);
  dbg_segment(t.row0, t.rows, p.A);
  if (t.rows <= 0) return;  // only where the debug check took the tile's rows away
  const int K = p.K, nblk = K / kBK;

  const uint8_t* ab = p.sorted_idx ? p.a : p.a + (size_t)t.row0 * K * 2;
  const uint8_t* wb = p.w + (size_t)t.e * p.stride;
  uint32_t ao[OA::kCopies], bo[OB::kCopies];
#pragma unroll
  for (int q = 0; q < OA::kCopies; ++q) {
    const int lr = OA::row_of(wave, q, lane), r = min(lr, t.rows - 1);
    const uint32_t src = p.sorted_idx
        ? (uint32_t)(dbg_clamp(p.sorted_idx[t.row0 + r], p.A, kDbgSorted) / p.k) : (uint32_t)r;
    ao[q] = src * (uint32_t)(K * 2) + (uint32_t)OA::unit_of(lr, lane) * 16;
  }
#pragma unroll
  for (int q = 0; q < OB::kCopies; ++q) {
    const int lr = OB::row_of(wave, q, lane), u = OB::unit_of(lr, lane);
    if constexpr (BT) {  // [K][N]: lr is k, the unit 8 columns
      bo[q] = (uint32_t)lr * (uint32_t)(p.N * 2) + (uint32_t)min(nb * kBN + u * 8, p.N - 8) * 2;
    } else if constexpr (MODE == kGated) {  // a wave's 64 weight rows: 32 gate rows, then their up rows
      const int col = min(nb * COLS + (lr >> 6) * 32 + (lr & 31), p.N - 1);
      bo[q] = (uint32_t)((lr & 32) ? p.I + col : col) * (uint32_t)(K * 2) + (uint32_t)u * 16;
    } else {
      bo[q] = (uint32_t)min(nb * kBN + lr, p.N - 1) * (uint32_t)(K * 2) + (uint32_t)u * 16;
    }
  }
  const size_t bstep = BT ? (size_t)kBK * p.N * 2 : (size_t)kBK * 2;
  auto issue = [&](int c) {
    Stage<BM, false, BT>& S = st[c & 1];
#pragma unroll
    for (int q = 0; q < OA::kCopies; ++q)
      dma16(ab + (size_t)c * kBK * 2, ao[q], S.a + (wave * OA::kCopies + q) * 1024);
#pragma unroll
    for (int q = 0; q < OB::kCopies; ++q)
      dma16(wb + c * bstep, bo[q], S.b + (wave * OB::kCopies + q) * 1024);
  };
  f32x16 acc[MI][2];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  issue(0);
  for (int c = 0; c < nblk; ++c) {
    MOE_DMA_SYNC(0);
    if (c + 1 < nblk) issue(c + 1);
    multiply<BM, false, BT>(st[c & 1], mh, nh, lane, acc);
  }

  const int l32 = lane & 31, hh = lane >> 5;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int lr = (mh * MI + i) * 32 + l32;
    if (lr >= t.rows) continue;
    const size_t row = (size_t)(t.row0 + lr);
    if constexpr (MODE == kGated) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = nb * COLS + nh * 32 + 8 * q + 4 * hh;
        if (col >= p.N) continue;
        float g[4], u[4], h[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          g[r] = acc[i][0][4 * q + r];
          u[r] = acc[i][1][4 * q + r];
          h[r] = swiglu(g[r], u[r]);
        }
        put4(p.out + row * p.I + col, h);
        put4(p.out2 + row * 2 * p.I + col, g);
        put4(p.out2 + row * 2 * p.I + p.I + col, u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = nb * kBN + (nh * 2 + j) * 32 + 8 * q + 4 * hh;
          if (col >= p.N) continue;
          if constexpr (MODE == kPlain) {
            float o[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = acc[i][j][4 * q + r];
            put4(p.out + row * p.N + col, o);
          } else {
            const uint2 gb = *reinterpret_cast<const uint2*>(p.gu + row * 2 * p.I + col);
            const uint2 ub = *reinterpret_cast<const uint2*>(p.gu + row * 2 * p.I + p.I + col);
            const uint32_t gw[2] = {gb.x, gb.y}, uw[2] = {ub.x, ub.y};
            float h[4], dg[4], du[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float g = __uint_as_float(r & 1 ? gw[r / 2] & 0xffff0000u : gw[r / 2] << 16);
              const float u = __uint_as_float(r & 1 ? uw[r / 2] & 0xffff0000u : uw[r / 2] << 16);
              const float dh = acc[i][j][4 * q + r];
              const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(g * -1.44269504f));
              h[r] = g * s * u;
              du[r] = dh * (g * s);
              dg[r] = dh * u * (s * fmaf(g, 1.f - s, 1.f));
            }
            put4(p.out + row * p.I + col, h);
            put4(p.out2 + row * 2 * p.I + col, dg);
            put4(p.out2 + row * 2 * p.I + p.I + col, du);
          }
        }
    }
  }
}

struct WgradArgs {
  int E, k, A;
  const int* counts;      // NULL: no expert has rows
  const int* offsets;
  const int* sorted_idx;  // rows of b, NULL: in expert order
  const uint8_t* a;       // bf16 [A][M]
  const uint8_t* b;       // bf16 [A][N], or gathered
  int M, N, mt, nt;
  void* out;              // [E][M][N]
};

// accumulate: out += (fp32 only)
template <bool F32>
__global__ __launch_bounds__(64 * kNW) void train_weights_kernel(WgradArgs p, int accumulate) {
  constexpr int BM = 256, MI = BM / 64;
  using OA = Operand<BM, true>;
  using OB = Operand<kBN, true>;
  __shared__ Stage<BM, true, true> st[2];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int mh = wave / kWN, nh = wave % kWN;
  const int per_e = p.mt * p.nt;
  const int e = (int)(blockIdx.x / (unsigned)per_e), v = (int)(blockIdx.x % (unsigned)per_e);
  const int mb = v / p.nt, nb = v % p.nt;
  int n = p.counts ? p.counts[e] : 0, row0 = p.counts ? p.offsets[e] : 0;
  dbg_segment(row0, n, p.A);
  n = __builtin_amdgcn_readfirstlane(n);
  row0 = __builtin_amdgcn_readfirstlane(row0);
  if (n <= 0 && accumulate) return;
  const int nblk = n > 0 ? (n + kBK - 1) / kBK : 0;

  int cola[OA::kCopies], colb[OB::kCopies];
#pragma unroll
  for (int q = 0; q < OA::kCopies; ++q)
    cola[q] = min(mb * BM + OA::unit_of(OA::row_of(wave, q, lane), lane) * 8, p.M - 8) * 2;
#pragma unroll
  for (int q = 0; q < OB::kCopies; ++q)
    colb[q] = min(nb * kBN + OB::unit_of(OB::row_of(wave, q, lane), lane) * 8, p.N - 8) * 2;
  auto issue = [&](int c) {
    Stage<BM, true, true>& S = st[c & 1];
    const int last = min(kBK, n - c * kBK) - 1;  // rows past the segment read its last one
    const uint8_t* ab = p.a + (size_t)(row0 + c * kBK) * p.M * 2;
    const uint8_t* bb = p.sorted_idx ? p.b : p.b + (size_t)(row0 + c * kBK) * p.N * 2;
#pragma unroll
    for (int q = 0; q < OA::kCopies; ++q)
      dma16(ab, (uint32_t)min(OA::row_of(wave, q, lane), last) * (uint32_t)(p.M * 2) + cola[q],
            S.a + (wave * OA::kCopies + q) * 1024);
#pragma unroll
    for (int q = 0; q < OB::kCopies; ++q) {
      const int r = min(OB::row_of(wave, q, lane), last);
      const uint32_t src = p.sorted_idx
          ? (uint32_t)(dbg_clamp(p.sorted_idx[row0 + c * kBK + r], p.A, kDbgSorted) / p.k) : (uint32_t)r;
      dma16(bb, src * (uint32_t)(p.N * 2) + colb[q], S.b + (wave * OB::kCopies + q) * 1024);
    }
  };
  f32x16 acc[MI][2];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  if (nblk) issue(0);
  for (int c = 0; c < nblk; ++c) {
    MOE_DMA_SYNC(0);
    const int left = n - c * kBK;
    if (left < kBK) {  // zeros past the segment's end (uniform; the last block)
      uint4* za = reinterpret_cast<uint4*>(st[c & 1].a + left * OA::kRowB);
      uint4* zb = reinterpret_cast<uint4*>(st[c & 1].b + left * OB::kRowB);
      for (int i = tid; i < (kBK - left) * OA::kRowB / 16; i += 64 * kNW) za[i] = uint4{0, 0, 0, 0};
      for (int i = tid; i < (kBK - left) * OB::kRowB / 16; i += 64 * kNW) zb[i] = uint4{0, 0, 0, 0};
      __syncthreads();
    }
    if (c + 1 < nblk) issue(c + 1);
    multiply<BM, true, true>(st[c & 1], mh, nh, lane, acc);
  }
  const int l32 = lane & 31, hh = lane >> 5;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = mb * BM + (mh * MI + i) * 32 + l32;
    if (m >= p.M) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = nb * kBN + (nh * 2 + j) * 32 + 8 * q + 4 * hh;
        if (col >= p.N) continue;
        const size_t at = ((size_t)e * p.M + m) * p.N + col;
        float o[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = acc[i][j][4 * q + r];
        if constexpr (F32) {
          f32x4* dst = reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + at);
          f32x4 w = {o[0], o[1], o[2], o[3]};
          if (accumulate) w += *dst;
          *dst = w;
        } else {
          put4(static_cast<uint16_t*>(p.out) + at, o);
        }
      }
  }
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

template <int MODE, bool BT>
int launch_rows(TrainArgs p, hipStream_t s, const char* who) {
  constexpr int BM = 256, COLS = MODE == kGated ? kBN / 2 : kBN;
  p.nnb = (p.N + COLS - 1) / COLS;
  const int64_t tiles = row_tiles_bound(p.A, p.E, BM) * p.nnb;
  const int64_t grid = (tiles + kXcds - 1) / kXcds * kXcds;
  if (grid * 64 * kNW >= (int64_t)1 << 32) return set_error(MOE_ERR_UNSUPPORTED, "%s: too many tiles", who);
  train_rows_kernel<BM, MODE, BT><<<(unsigned)grid, 64 * kNW, 0, s>>>(p);
  return check_launch(who);
}

int launch_weights(WgradArgs p, bool f32, int accumulate, hipStream_t s, const char* who) {
  p.mt = (p.M + 255) / 256;
  p.nt = (p.N + kBN - 1) / kBN;
  const int64_t grid = (int64_t)p.E * p.mt * p.nt;
  if (grid * 64 * kNW >= (int64_t)1 << 32) return set_error(MOE_ERR_UNSUPPORTED, "%s: too many tiles", who);
  if (f32) train_weights_kernel<true><<<(unsigned)grid, 64 * kNW, 0, s>>>(p, accumulate);
  else train_weights_kernel<false><<<(unsigned)grid, 64 * kNW, 0, s>>>(p, 0);
  return check_launch(who);
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

}  // namespace

#ifdef MOE_DEBUG
uint32_t dbg_take_train() { return dbg_take_unit(); }
#endif

}  // namespace moe

using namespace moe;

// Workspace: h bf16 [T*k][I].
extern "C" size_t moe_expert_ffn_train_workspace(const moe_experts* W, int32_t T, int32_t k) {
  if (!W || T < 0 || k < 1) return 0;
  return align256((size_t)T * k * W->I * 2);
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
  TrainArgs p{};
  p.E = W->E; p.H = W->H; p.I = W->I; p.k = k; p.A = T * k;
  p.counts = counts; p.offsets = offsets; p.sorted_idx = sorted_idx;
  p.w = static_cast<const uint8_t*>(W->base) + Lo.w13; p.stride = W->stride;
  p.a = reinterpret_cast<const uint8_t*>(x);
  p.K = W->H; p.N = W->I;
  p.out = static_cast<uint16_t*>(ws); p.out2 = gate_up;
  if (int st = launch_rows<kGated, false>(p, s, who)) return st;
  p.sorted_idx = nullptr;
  p.w = static_cast<const uint8_t*>(W->base) + Lo.w2;
  p.a = static_cast<const uint8_t*>(ws);
  p.K = W->I; p.N = W->H;
  p.out = y_perm; p.out2 = nullptr;
  return launch_rows<kPlain, false>(p, s, who);
}

// Workspace: h bf16 [T*k][I], (dg; du) bf16 [T*k][2I].
extern "C" size_t moe_expert_ffn_backward_workspace(const moe_experts* W, int32_t T, int32_t k) {
  if (!W || T < 0 || k < 1) return 0;
  return align256((size_t)T * k * W->I * 2) + align256((size_t)T * k * W->I * 4);
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
  if (accumulate && d_w_type != MOE_T_F32)
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
  uint16_t* h = static_cast<uint16_t*>(ws);
  uint16_t* dgu = h + align256((size_t)A * I * 2) / 2;
  if (T > 0 && (d_x_perm || d_w13 || d_w2)) {
    TrainArgs p{};
    p.E = W->E; p.H = H; p.I = I; p.k = k; p.A = A;
    p.counts = counts; p.offsets = offsets;
    p.stride = W->stride;
    p.w = static_cast<const uint8_t*>(W->base) + Lo.w2;
    p.a = reinterpret_cast<const uint8_t*>(d_y_perm);
    p.K = H; p.N = I;
    p.out = h; p.out2 = dgu; p.gu = gate_up;
    if (int st = launch_rows<kDswiglu, true>(p, s, who)) return st;
    if (d_x_perm) {
      p.w = static_cast<const uint8_t*>(W->base) + Lo.w13;
      p.a = reinterpret_cast<const uint8_t*>(dgu);
      p.K = 2 * I; p.N = H;
      p.out = d_x_perm; p.out2 = nullptr; p.gu = nullptr;
      if (int st = launch_rows<kPlain, true>(p, s, who)) return st;
    }
  }
  WgradArgs g{};
  g.E = W->E; g.k = k; g.A = A;
  g.counts = T > 0 ? counts : nullptr;
  g.offsets = offsets;
  if (d_w13 && !(T == 0 && accumulate)) {
    g.sorted_idx = sorted_idx;
    g.a = reinterpret_cast<const uint8_t*>(dgu);
    g.b = reinterpret_cast<const uint8_t*>(x);
    g.M = 2 * I; g.N = H; g.out = d_w13;
    if (int st = launch_weights(g, d_w_type == MOE_T_F32, accumulate, s, who)) return st;
  }
  if (d_w2 && !(T == 0 && accumulate)) {
    g.sorted_idx = nullptr;
    g.a = reinterpret_cast<const uint8_t*>(d_y_perm);
    g.b = reinterpret_cast<const uint8_t*>(h);
    g.M = H; g.N = I; g.out = d_w2;
    if (int st = launch_weights(g, d_w_type == MOE_T_F32, accumulate, s, who)) return st;
  }
  return MOE_OK;
}
