// Router training: load-balance loss with per-expert counts, and the gradient
// of the routing weights and of that loss with respect to the logits.
//
// Both passes are bound by one read of the logits (the backward also writes
// as much): a group of LPR lanes holds one row, LPR = 16 for E <= 64 (four
// rows per wave) and 64 above, with the row's softmax kept in registers.
//
// Forward.  The batch is cut into chunks of R rows, one workgroup each, which
// walks the pieces of sequences inside its chunk.  A piece (chunk c, sequence
// s) has the slot c + s of the partial arrays: going down the batch every
// piece raises c or s, so slots are unique and fewer than chunks + S.  Each
// lane sums the probabilities of its experts over its rows (fp32, at most
// R / 4 terms), the waves are added in LDS, and the ids are counted with
// integer LDS atomics (their order does not matter).  A second kernel
// adds a sequence's pieces in double in chunk order, a workgroup per sequence and
// 16 experts, and a third forms the loss.  A batch of one chunk in up to
// kOneKernelSeqs sequences is finished by the first kernel.
#include <algorithm>

#include "fp8_common.h"

namespace moe {
namespace {

struct BalArgs {
  const float* logits;
  const int* ids;
  const uint8_t* mask;
  const int* seq;  // NULL: one sequence [0, T)
  int T, E, k, S, R;
  float* part_p;  // [slots][E]
  int* part_c;    // [slots][E]
  int* part_n;    // [slots]
  double* part_d; // [S][slices of kSlice experts]
  int* n_tokens;
  int* counts;
  float* probs;
  float* loss;
};

struct RouteBwdArgs {
  const float* logits;
  const int* ids;
  const float* w;
  const float* dw;
  const uint8_t* mask;
  const int* seq;
  const int* n_tokens;
  const int* counts;
  const float* d_loss;
  float* d_logits;
  int T, E, k, S, R, renorm;
};

// Rows of sequence s, clamped into [0, T] (flagged in the checked build).
__device__ __forceinline__ void seq_rows(const int* seq, int s, int T, int& lo, int& hi) {
  lo = seq ? seq[s] : 0;
  hi = seq ? seq[s + 1] : T;
#ifdef MOE_DEBUG
  if (lo < 0 || hi < lo || hi > T) atomicOr(&g_dbg_flags, kDbgSegment);
#endif
  lo = lo < 0 ? 0 : lo > T ? T : lo;
  hi = hi < lo ? lo : hi > T ? T : hi;
}

// The first sequence that ends behind row t (S if none does), found by a whole wave: each
// step reads 64 evenly spaced offsets and keeps the interval between two of them (S <= 64:
// one step, so one memory latency).
__device__ __forceinline__ int first_seq(const int* seq, int S, int t, int lane) {
  if (!seq) return 0;
  int lo = 0, n = S;  // the answer lies in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 63) >> 6;
    const int i = lane * step;
    const bool past = i < n && seq[lo + min(i + step, n)] <= t;  // the lane's last sequence ends by t
    const int k = __popcll(__ballot(past));
    const int d = min(k * step, n);
    lo += d;
    n = step == 1 ? 0 : min(step, n - d);
  }
  return lo;
}

// The same by one lane alone.
__device__ __forceinline__ int seq_of_row(const int* seq, int S, int t) {
  int a = 0, b = seq ? S : 0;
  while (a < b) {
    const int m = (a + b) >> 1;
    if (seq[m + 1] > t) b = m;
    else a = m + 1;
  }
  return a;
}

// Maximum and sum over the LPR lanes of a group, in every lane of it.
template <int LPR>
__device__ __forceinline__ float group_max(float x) {
  int v = __float_as_int(x);
  auto mx = [](int a, int b) { return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b))); };
  v = mx(v, dpp_i32<0xB1>(v, v));
  v = mx(v, dpp_i32<0x4E>(v, v));
  v = mx(v, dpp_i32<0x141>(v, v));
  v = mx(v, dpp_i32<0x140>(v, v));
  if constexpr (LPR == 64) {
    v = mx(v, dpp_i32<0x142, 0xA>(v, v));
    v = mx(v, dpp_i32<0x143, 0xC>(v, v));
    v = __builtin_amdgcn_readlane(v, 63);
  }
  return __int_as_float(v);
}
template <int LPR>
__device__ __forceinline__ float group_sum(float x) {
  if constexpr (LPR == 64) return wave_sum_f32(x);
  int v = __float_as_int(x);
  auto add = [](int a, int b) { return __float_as_int(__int_as_float(a) + __int_as_float(b)); };
  v = add(v, dpp_i32<0xB1>(v, v));
  v = add(v, dpp_i32<0x4E>(v, v));
  v = add(v, dpp_i32<0x141>(v, v));
  v = add(v, dpp_i32<0x140>(v, v));
  return __int_as_float(v);
}

// Expert of value i of a lane (sub = lane within its group): VEC reads four
// consecutive experts with one 16-byte load (E a multiple of 4).
template <int LPR, bool VEC>
__device__ __forceinline__ int expert_of(int sub, int i) {
  return VEC ? 4 * (sub + LPR * (i >> 2)) + (i & 3) : sub + LPR * i;
}

template <int LPR, int VPL, bool VEC, typename V>
__device__ __forceinline__ void load_row(const V* __restrict__ row, int E, int sub, bool live,
                                         V fill, V (&x)[VPL]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4) {
      const int e = expert_of<LPR, VEC>(sub, i);
      uint4 q;
      const bool ok = live && e < E;
      if (ok) q = *reinterpret_cast<const uint4*>(row + e);
      x[i] = ok ? __builtin_bit_cast(V, q.x) : fill;
      x[i + 1] = ok ? __builtin_bit_cast(V, q.y) : fill;
      x[i + 2] = ok ? __builtin_bit_cast(V, q.z) : fill;
      x[i + 3] = ok ? __builtin_bit_cast(V, q.w) : fill;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = expert_of<LPR, VEC>(sub, i);
      x[i] = live && e < E ? row[e] : fill;
    }
  }
}

// e^d for d <= 0: 2^t with t = d log2(e), what t's rounding and the constant's lost (lo, under
// 2^-23 |t|) entered as 2^lo = 1 + lo ln 2: relative error (|d| + 3) 2^-24 with the rounding of
// d itself.  -inf gives 0 (lo is NaN there and clamped), NaN stays.
__device__ __forceinline__ float exp_neg(float d) {
  const float t = d * 1.44269504f;
  const float lo =
      __builtin_amdgcn_fmed3f(fmaf(d, 1.92596299e-8f, fmaf(d, 1.44269504f, -t)), -1.0f, 1.0f);
  const float z = __builtin_amdgcn_exp2f(t);
  return fmaf(z, lo * 0.69314718f, z);
}

// Logits of a row -> its softmax, over the group's lanes.  Experts past E and
// -inf logits get 0; a row of nothing but -inf gets zeros.
template <int LPR, int VPL>
__device__ __forceinline__ void row_softmax(float (&x)[VPL]) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) m = fmaxf(m, x[i]);
  m = group_max<LPR>(m);
  m = m == -INFINITY ? 0.0f : m;
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    x[i] = exp_neg(x[i] - m);
    z += x[i];
  }
  z = group_sum<LPR>(z);
  const float inv = z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
  for (int i = 0; i < VPL; ++i) x[i] *= inv;
}

constexpr int kMaxChunk = 128;  // rows of a chunk at most
// Sequences of one chunk that the first kernel finishes by itself, one after another; more leave
// the sums to the other two.  us a call, one kernel against three, E = 256 (E = 1024): T = 64, 1
// sequence 7.2 / 13.7, 2 10.6 / 14.6, 4 19.3 / 15.7, 8 36.7 / 23.5, 64 281 / 134; T = 128, 1 9.4 /
// 19.2 (18.6 / 33.4), 4 19.3 / 21.6 (25.4 / 37.1), 8 36.6 / 24.3 (32.5 / 42.6), 16 71 / 39 (62 / 54),
// 64 281 / 134 (235 / 181).
constexpr int kOneKernelSeqs = 4;

// U rows of a group, NG rows apart from row t on: loads in flight together, with the rows'
// mask bytes beside them (a masked row is read and dropped: waiting for its mask first
// would double the latency).
template <int NG, int U, int LPR, int VPL, bool VEC>
struct Rows {
  float x[U][VPL];
  bool live[U];
  __device__ __forceinline__ void load(const BalArgs& a, int t, int hi, int sub) {
    uint8_t m[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      live[u] = t + u * NG < hi;
      m[u] = a.mask && live[u] ? a.mask[t + u * NG] : 1;
      load_row<LPR, VPL, VEC>(a.logits + (size_t)(t + u * NG) * a.E, a.E, sub, live[u], -INFINITY,
                              x[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) live[u] = live[u] && m[u];
  }
};

// A thread's first assignments of the chunk (i = tid, tid + NT of its rows * k): row and id,
// -1 where the row is masked; and the mask of row tid.
template <int NT>
struct Ids {
  static constexpr int P = 2;
  int row[P], id[P];
  bool on;
  __device__ __forceinline__ void load(const BalArgs& a, int t0, int t1, int tid) {
    const int n = (t1 - t0) * a.k;
    uint8_t m[P];
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const int i = tid + q * NT;
      row[q] = i < n ? t0 + i / a.k : -1;
      id[q] = i < n ? a.ids[(size_t)t0 * a.k + i] : -1;
      m[q] = i < n && a.mask ? a.mask[row[q]] : 1;
    }
    on = t0 + tid < t1 && (!a.mask || a.mask[t0 + tid]);
#pragma unroll
    for (int q = 0; q < P; ++q) id[q] = m[q] ? id[q] : -1;
  }
};

// The rows [lo, hi) of a sequence inside the chunk [t0, t1): probability sums of the wave into
// its row of acc, counts into hist, counting rows into *nv (all LDS; finished by a barrier).
// `first` and `ids` hold what was loaded ahead: the chunk's first rows (this piece's if it
// starts the chunk) and its first assignments.
template <int NW, int U, int LPR, int VPL, bool VEC, typename R>
__device__ __forceinline__ void balance_piece(const BalArgs& a, int t0, int t1, int lo, int hi,
                                              const R& first, const Ids<64 * NW>& ids,
                                              float (*acc)[kMaxE], int* hist, int* nv) {
  constexpr int NT = 64 * NW, GPW = 64 / LPR, NG = NW * GPW;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int sub = lane % LPR, grp = wave * GPW + lane / LPR;
  const bool ahead = lo == t0;
  for (int i = tid; i < a.E; i += NT) hist[i] = 0;
  if (tid == 0) *nv = 0;
  __syncthreads();
  // counts, and the number of counting rows (a chunk has at most kMaxChunk <= NT rows)
#pragma unroll
  for (int q = 0; q < Ids<NT>::P; ++q)
    if ((unsigned)ids.id[q] < (unsigned)a.E && ids.row[q] >= lo && ids.row[q] < hi)
      atomicAdd(&hist[ids.id[q]], 1);
  for (int i = tid + Ids<NT>::P * NT; i < (t1 - t0) * a.k; i += NT) {
    const int t = t0 + i / a.k;
    const int id = a.ids[(size_t)t0 * a.k + i];
    if ((unsigned)id < (unsigned)a.E && t >= lo && t < hi && (!a.mask || a.mask[t]))
      atomicAdd(&hist[id], 1);
  }
  const uint64_t counting = __ballot(ids.on && t0 + tid >= lo && t0 + tid < hi);
  if (lane == 0 && counting) atomicAdd(nv, (int)__popcll(counting));
  float sum[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) sum[i] = 0.0f;
  auto take = [&](const R& r, int t) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = t + u * NG < hi && r.live[u];
      float p[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) p[i] = in ? r.x[u][i] : -INFINITY;
      row_softmax<LPR, VPL>(p);
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum[i] += p[i];
    }
  };
  int t = lo + grp;
  if (ahead) {
    take(first, t);
    t += NG * U;
  }
  for (; t - grp < hi; t += NG * U) {
    R r;
    r.load(a, t, hi, sub);
    take(r, t);
  }
  // the groups of a wave
  if constexpr (LPR == 16) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      sum[i] += __shfl_xor(sum[i], 16, 64);
      sum[i] += __shfl_xor(sum[i], 32, 64);
    }
  }
  if (lane < LPR) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = expert_of<LPR, VEC>(sub, i);
      if (e < a.E) acc[wave][e] = sum[i];
    }
  }
  __syncthreads();
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// loss of one sequence from its counts and sums.
__device__ __forceinline__ float loss_of(double dot, int E, int k, int n) {
  return n > 0 ? (float)(dot * (double)E / ((double)k * (double)n * (double)n)) : 0.0f;
}

template <int NW, int LPR, int VPL, bool VEC, bool FINAL>
__global__ __launch_bounds__(64 * NW) void balance_partial_kernel(BalArgs a) {
  __shared__ float acc[NW][kMaxE];
  __shared__ int hist[kMaxE];
  __shared__ double wdot[NW];
  __shared__ int nv;
  constexpr int NT = 64 * NW, NG = NW * 64 / LPR;
  constexpr int U = VPL == 4 ? 4 : VPL == 16 && NW == 16 ? 1 : 2;  // rows in flight per group
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = (int)blockIdx.x;
  const int t0 = c * a.R, t1 = FINAL ? a.T : min(a.T, t0 + a.R);
  Rows<NG, U, LPR, VPL, VEC> first;
  first.load(a, t0 + wave * (64 / LPR) + lane / LPR, t1, lane % LPR);
  Ids<NT> ids;
  ids.load(a, t0, t1, tid);
  for (int s = FINAL ? 0 : first_seq(a.seq, a.S, t0, lane); s < a.S; ++s) {
    int lo, hi;
    seq_rows(a.seq, s, a.T, lo, hi);
    if (!FINAL && lo >= t1) break;
    if (!FINAL && lo == hi) {  // a run of empty sequences: on to the one that holds row lo
      s = max(s, first_seq(a.seq, a.S, lo, lane) - 1);
      continue;
    }
    lo = max(lo, t0);
    hi = min(hi, t1);
    if (FINAL || hi > lo) {
      balance_piece<NW, U, LPR, VPL, VEC>(a, t0, t1, lo, hi, first, ids, acc, hist, &nv);
      const int n = nv;
      const size_t o = FINAL ? (size_t)s * a.E : (size_t)(c + s) * a.E;
      float* po = FINAL ? a.probs : a.part_p;
      int* co = FINAL ? a.counts : a.part_c;
      double dot = 0.0;
      for (int i = tid; i < a.E; i += NT) {  // the waves in order
        float p = acc[0][i];
#pragma unroll
        for (int w = 1; w < NW; ++w) p += acc[w][i];
        const int h = hist[i];
        po[o + i] = p;
        co[o + i] = h;
        if constexpr (FINAL) dot += (double)p * (double)h;
      }
      if (tid == 0) (FINAL ? a.n_tokens[s] : a.part_n[c + s]) = n;
      if constexpr (FINAL) {
        dot = wave_sum_f64(dot);
        if (lane == 0) wdot[wave] = dot;
        __syncthreads();
        if (tid == 0) {
          double d = 0.0;
#pragma unroll
          for (int w = 0; w < NW; ++w) d += wdot[w];
          a.loss[s] = loss_of(d, a.E, a.k, n);
        }
      }
      __syncthreads();  // acc, hist, wdot and nv are reused by the next piece
    }
  }
}

// The pieces of a sequence in chunk order, one workgroup per sequence and kSlice experts: thread
// = (expert, one of kRedLanes interleaved chunk lanes), U chunks in flight, the lanes then
// added in a fixed order.  Each slice leaves its share of the loss's sum.
constexpr int kSlice = 16, kRedLanes = 64;
__global__ __launch_bounds__(kSlice * kRedLanes) void balance_reduce_kernel(BalArgs a) {
  constexpr int NT = kSlice * kRedLanes, NW = NT / 64, U = 8;
  __shared__ double sp[NW][kSlice];
  __shared__ int sc[NW][kSlice], sn[NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nsl = (a.E + kSlice - 1) / kSlice;
  for (int b = (int)blockIdx.x; b < a.S * nsl; b += (int)gridDim.x) {
    const int s = b / nsl, sl = b - s * nsl;
    int lo, hi;
    seq_rows(a.seq, s, a.T, lo, hi);
    const int c0 = lo / a.R, c1 = hi > lo ? (hi - 1) / a.R + 1 : c0;
    const int e = sl * kSlice + tid % kSlice, cl = tid / kSlice;
    double p = 0.0;
    int c = 0;
    for (int i = c0 + cl; i < c1; i += kRedLanes * U) {
      float pv[U];
      int cv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool ok = i + u * kRedLanes < c1 && e < a.E;
        const size_t o = (size_t)(i + u * kRedLanes + s) * a.E + e;
        pv[u] = ok ? a.part_p[o] : 0.0f;
        cv[u] = ok ? a.part_c[o] : 0;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        p += (double)pv[u];
        c += cv[u];
      }
    }
    int n = 0;
    if (sl == 0)
      for (int i = c0 + tid; i < c1; i += NT) n += a.part_n[i + s];
#pragma unroll
    for (int o = 16; o < 64; o *= 2) {  // the wave's four chunk lanes
      p += __shfl_xor(p, o, 64);
      c += __shfl_xor(c, o, 64);
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) n += __shfl_xor(n, o, 64);
    if (lane < kSlice) {
      sp[wave][lane] = p;
      sc[wave][lane] = c;
    }
    if (lane == 0) sn[wave] = n;
    __syncthreads();
    if (wave == 0) {
      double dot = 0.0;
      if (lane < kSlice && e < a.E) {
#pragma unroll
        for (int w = 1; w < NW; ++w) {
          p += sp[w][lane];
          c += sc[w][lane];
        }
        a.probs[(size_t)s * a.E + e] = (float)p;
        a.counts[(size_t)s * a.E + e] = c;
        dot = p * (double)c;
      }
      dot = wave_sum_f64(dot);
      if (lane == 0) {
        a.part_d[(size_t)s * nsl + sl] = dot;
        if (sl == 0) {
#pragma unroll
          for (int w = 1; w < NW; ++w) n += sn[w];
          a.n_tokens[s] = n;
        }
      }
    }
    __syncthreads();  // sp, sc and sn are reused by the next slice
  }
}

// One wave per sequence: the slices' shares (at most 64) -> the loss.
__global__ __launch_bounds__(256) void balance_loss_kernel(BalArgs a) {
  const int lane = threadIdx.x & 63, s = (int)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (s >= a.S) return;
  const int nsl = (a.E + kSlice - 1) / kSlice;
  const double d = wave_sum_f64(lane < nsl ? a.part_d[(size_t)s * nsl + lane] : 0.0);
  if (lane == 0) a.loss[s] = loss_of(d, a.E, a.k, a.n_tokens[s]);
}

// Gradient: a group of LPR lanes per row, kBwdRows rows per workgroup of 4 waves (65536 x 512:
// 50.8 us with 16, 53.1 with 32, 59.3 with 64 rows).
constexpr int kBwdRows = 16;
template <int LPR, int VPL, bool VEC>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteBwdArgs a) {
  constexpr int GPW = 64 / LPR, NG = 4 * GPW;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int sub = lane % LPR, grp = wave * GPW + lane / LPR;
  __shared__ __attribute__((aligned(16))) float extra[NG][LPR * VPL];
  for (int i = tid; i < NG * LPR * VPL; i += 256) (&extra[0][0])[i] = 0.0f;
  __syncthreads();
  const int t0 = (int)blockIdx.x * a.R, t1 = min(a.T, t0 + a.R);
  int s = -1, lo = 0, hi = 0;
  float ac[VPL];  // a_s c_se of the current sequence
#pragma unroll
  for (int i = 0; i < VPL; ++i) ac[i] = 0.0f;
  // what a row needs is read whether or not it turns out to count (lane j < k of the group holds
  // assignment j)
  int s_next = first_seq(a.seq, a.S, t0, lane);
  for (int t = t0 + grp; t - grp < t1; t += NG) {
    const bool in = t < t1;
    const uint8_t m = a.mask && in ? a.mask[t] : 1;
    float p[VPL];
    load_row<LPR, VPL, VEC>(a.logits + (size_t)t * a.E, a.E, sub, in, -INFINITY, p);
    int id = -1;
    float w = 0.0f, wd = 0.0f;
    if (a.dw && in && sub < a.k) {
      const size_t o = (size_t)t * a.k + sub;
      id = a.ids[o];
      w = a.w[o];
      wd = a.dw[o];
    }
    // the row's sequence (per group; every lane of the group agrees): the next one, or, behind
    // empty ones, the one that a search finds
    for (int step = 0; s_next < a.S && t >= hi; ++step) {
      if (step == 1) s_next = max(s_next, seq_of_row(a.seq, a.S, t));
      if (s_next >= a.S) break;
      s = s_next++;
      seq_rows(a.seq, s, a.T, lo, hi);
      if (t < hi && a.d_loss) {
        const int n = a.n_tokens[s];
        const float as = n > 0 ? (float)((double)a.d_loss[s] * a.E / ((double)a.k * n * n)) : 0.0f;
        int c[VPL];
        load_row<LPR, VPL, VEC>(a.counts + (size_t)s * a.E, a.E, sub, true, 0, c);
#pragma unroll
        for (int i = 0; i < VPL; ++i) ac[i] = as * (float)c[i];
      }
    }
    const bool inside = in && s >= 0 && t >= lo && t < hi;
    const bool live = inside && m;
#pragma unroll
    for (int i = 0; i < VPL; ++i) p[i] = live ? p[i] : -INFINITY;
    if (!live || (unsigned)id >= (unsigned)a.E) id = -1;
    w = id < 0 ? 0.0f : w;
    wd = id < 0 ? 0.0f : w * wd;
    const float D = group_sum<LPR>(wd);
    const float add = a.renorm ? wd - w * D : wd;
    row_softmax<LPR, VPL>(p);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) dot += p[i] * ac[i];
    dot = group_sum<LPR>(dot) + (a.renorm ? 0.0f : D);
#pragma unroll
    for (int i = 0; i < VPL; ++i) p[i] *= ac[i] - dot;
    if (a.dw) {
      // the weights' share, through a row of LDS that is zero between rows: the first lane of
      // every id adds up that id's terms in order
      float mine = 0.0f;
      bool lead = id >= 0;
      for (int j = 0; j < a.k; ++j) {
        int idj;
        float v;
        if constexpr (LPR == 64) {
          idj = __builtin_amdgcn_readlane(id, j);
          v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(add), j));
        } else {
          idj = __shfl(id, (lane & ~15) + j, 64);
          v = __shfl(add, (lane & ~15) + j, 64);
        }
        if (id == idj) {
          mine += v;
          lead = lead && j >= sub;
        }
      }
      if (lead) extra[grp][id] = mine;
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < VPL; ++i) p[i] += extra[grp][expert_of<LPR, VEC>(sub, i)];
      __builtin_amdgcn_wave_barrier();
      if (lead) extra[grp][id] = 0.0f;
      __builtin_amdgcn_wave_barrier();
    }
    if (inside) {
      float* out = a.d_logits + (size_t)t * a.E;
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < VPL; i += 4) {
          const int e = expert_of<LPR, VEC>(sub, i);
          float4 q = {p[i], p[i + 1], p[i + 2], p[i + 3]};
          if (!live) q = float4{0.f, 0.f, 0.f, 0.f};
          if (e < a.E) *reinterpret_cast<float4*>(out + e) = q;
        }
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int e = expert_of<LPR, VEC>(sub, i);
          if (e < a.E) out[e] = live ? p[i] : 0.0f;
        }
      }
    }
  }
}

// Calls f with the row shape's constants: lanes per row, values per lane,
// 16-byte loads.
template <int L, int V, bool X>
struct RowShape {
  static constexpr int lpr = L, vpl = V;
  static constexpr bool vec = X;
};
template <typename F>
void with_row_shape(int E, F f) {
  if (E % 4 == 0) {
    if (E <= 64) f(RowShape<16, 4, true>{});
    else if (E <= 256) f(RowShape<64, 4, true>{});
    else if (E <= 512) f(RowShape<64, 8, true>{});
    else f(RowShape<64, 16, true>{});
  } else {
    if (E <= 64) f(RowShape<16, 4, false>{});
    else if (E <= 256) f(RowShape<64, 4, false>{});
    else if (E <= 512) f(RowShape<64, 8, false>{});
    else f(RowShape<64, 16, false>{});
  }
}

// Batches of at most kMaxChunk rows are one chunk; larger ones take chunks of
// 16 rows and up, so that 512 workgroups share the batch until chunks reach
// kMaxChunk rows.
int chunk_rows(int T) {
  const int64_t r = ((int64_t)T / 512 + 15) / 16 * 16;
  return (int)(T <= kMaxChunk || r > kMaxChunk ? kMaxChunk : r < 16 ? 16 : r);
}

struct BalWs {
  size_t p, c, n, d, total;
};
BalWs bal_ws(int T, int E, int S) {
  const size_t slots = (size_t)(T + chunk_rows(T) - 1) / chunk_rows(T) + (size_t)S;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  BalWs w;
  w.p = 0;
  w.c = up(slots * E * 4);
  w.n = w.c + up(slots * E * 4);
  w.d = w.n + up(slots * 4);
  w.total = w.d + up((size_t)S * ((E + kSlice - 1) / kSlice) * 8);
  return w;
}

int check_router_args(const char* who, int T, int E, int k, const int* seq, int S) {
  if (T < 0 || E < 1 || E > kMaxE || k < 1 || k > E || k > kMaxK)
    return set_error(MOE_ERR_INVALID_ARG, "%s: need T>=0, 1<=E<=%d, 1<=k<=min(E,%d) "
                     "(T=%d E=%d k=%d)", who, kMaxE, kMaxK, T, E, k);
  if (S < 1 || S > (1 << 20) || (!seq && S != 1))
    return set_error(MOE_ERR_INVALID_ARG, "%s: S=%d sequences (1..2^20; 1 without seq_offsets)",
                     who, S);
  if ((int64_t)T * k > (1 << 27))
    return set_error(MOE_ERR_UNSUPPORTED, "%s: T*k too large", who);
  if (!aligned16(seq)) return set_error(MOE_ERR_INVALID_ARG, "%s: seq_offsets misaligned", who);
  return MOE_OK;
}

}  // namespace

#ifdef MOE_DEBUG
uint32_t dbg_take_balance() { return dbg_take_unit(); }
#endif

}  // namespace moe

using namespace moe;

extern "C" size_t moe_balance_loss_workspace(int32_t T, int32_t E, int32_t S) {
  if (T < 0 || E < 1 || E > kMaxE || S < 1) return 0;
  return bal_ws(T, E, S).total;
}

extern "C" int moe_balance_loss(const float* logits, const int32_t* topk_ids, int32_t T, int32_t E,
                                int32_t k, const uint8_t* token_mask, const int32_t* seq_offsets,
                                int32_t S, int32_t* n_tokens, int32_t* counts, float* probs,
                                float* loss, void* ws, size_t ws_bytes, moe_stream_t stream) {
  const char* who = "moe_balance_loss";
  int st = check_router_args(who, T, E, k, seq_offsets, S);
  if (st) return st;
  if (!n_tokens || !counts || !probs || !loss || !ws || (T > 0 && (!logits || !topk_ids)))
    return set_error(MOE_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned16(logits) || !aligned16(topk_ids) || !aligned16(token_mask) ||
      !aligned16(n_tokens) || !aligned16(counts) || !aligned16(probs) || !aligned16(loss) ||
      !aligned16(ws))
    return set_error(MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  const BalWs L = bal_ws(T, E, S);
  if (ws_bytes < L.total)
    return set_error(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", who, ws_bytes, L.total);
  uint8_t* w = static_cast<uint8_t*>(ws);
  BalArgs a{};
  a.logits = logits;
  a.ids = topk_ids;
  a.mask = token_mask;
  a.seq = seq_offsets;
  a.T = T; a.E = E; a.k = k; a.S = S;
  a.R = chunk_rows(T);
  a.part_p = reinterpret_cast<float*>(w + L.p);
  a.part_c = reinterpret_cast<int*>(w + L.c);
  a.part_n = reinterpret_cast<int*>(w + L.n);
  a.part_d = reinterpret_cast<double*>(w + L.d);
  a.n_tokens = n_tokens;
  a.counts = counts;
  a.probs = probs;
  a.loss = loss;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (T <= kMaxChunk && S <= kOneKernelSeqs) {  // one chunk: finished by the first kernel
    with_row_shape(E, [&](auto r) {
      using Q = decltype(r);
      balance_partial_kernel<16, Q::lpr, Q::vpl, Q::vec, true><<<1, 1024, 0, s>>>(a);
    });
    return check_launch(who);
  }
  const unsigned chunks = (unsigned)((T + a.R - 1) / a.R);
  if (chunks) with_row_shape(E, [&](auto r) {
    using Q = decltype(r);
    balance_partial_kernel<4, Q::lpr, Q::vpl, Q::vec, false><<<chunks, 256, 0, s>>>(a);
  });
  const unsigned slices = (unsigned)((E + kSlice - 1) / kSlice);
  // a grid has fewer than 2^32 threads
  const unsigned blocks = std::min((unsigned)S * slices, 1u << 21);
  balance_reduce_kernel<<<blocks, kSlice * kRedLanes, 0, s>>>(a);
  balance_loss_kernel<<<((unsigned)S + 3) / 4, 256, 0, s>>>(a);
  return check_launch(who);
}

extern "C" int moe_route_backward(const float* logits, int32_t T, int32_t E, int32_t k,
                                  int32_t renorm, const int32_t* topk_ids, const float* topk_w,
                                  const float* d_topk_w, const uint8_t* token_mask,
                                  const int32_t* seq_offsets, int32_t S, const int32_t* n_tokens,
                                  const int32_t* counts, const float* d_loss, float* d_logits,
                                  moe_stream_t stream) {
  const char* who = "moe_route_backward";
  int st = check_router_args(who, T, E, k, seq_offsets, S);
  if (st) return st;
  if (!d_topk_w && !d_loss)
    return set_error(MOE_ERR_INVALID_ARG, "%s: needs d_topk_w or d_loss", who);
  if (T == 0) return MOE_OK;
  if (!logits || !d_logits || (d_topk_w && (!topk_ids || !topk_w)) ||
      (d_loss && (!n_tokens || !counts)))
    return set_error(MOE_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned16(logits) || !aligned16(d_logits) || !aligned16(topk_ids) || !aligned16(topk_w) ||
      !aligned16(d_topk_w) || !aligned16(token_mask) || !aligned16(n_tokens) ||
      !aligned16(counts) || !aligned16(d_loss))
    return set_error(MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  RouteBwdArgs a{};
  a.logits = logits;
  a.ids = topk_ids;
  a.w = topk_w;
  a.dw = d_topk_w;
  a.mask = token_mask;
  a.seq = seq_offsets;
  a.n_tokens = n_tokens;
  a.counts = counts;
  a.d_loss = d_loss;
  a.d_logits = d_logits;
  a.T = T; a.E = E; a.k = k; a.S = S; a.renorm = renorm;
  a.R = kBwdRows;
  const unsigned blocks = (unsigned)((T + a.R - 1) / a.R);
  with_row_shape(E, [&](auto r) {
    using Q = decltype(r);
    route_backward_kernel<Q::lpr, Q::vpl, Q::vec>
        <<<blocks, 256, 0, reinterpret_cast<hipStream_t>(stream)>>>(a);
  });
  return check_launch(who);
}
