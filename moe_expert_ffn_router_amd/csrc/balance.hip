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
// R / 4 terms), the groups are added in LDS, and the ids are counted with
// integer LDS atomics (their order does not matter).  A second kernel, one
// workgroup per sequence, adds a sequence's pieces in double in chunk order
// and forms the loss.  A batch of one chunk is finished by the first kernel.
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

// The first sequence that ends behind row t (S if none does).
__device__ __forceinline__ int first_seq(const int* seq, int S, int t) {
  if (!seq) return 0;
  int a = 0, b = S;
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
    x[i] = expf(x[i] - m);
    z += x[i];
  }
  z = group_sum<LPR>(z);
  const float inv = z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
  for (int i = 0; i < VPL; ++i) x[i] *= inv;
}

constexpr int kMaxChunk = 128;  // rows of a chunk at most

// The rows [lo, hi) of a sequence inside one chunk: probability sums into
// acc[0..E), counts into hist[0..E), counting rows into *nv (all LDS).
template <int NW, int LPR, int VPL, bool VEC>
__device__ __forceinline__ void balance_piece(const BalArgs& a, int lo, int hi, float* acc,
                                              int* hist, int* nv) {
  constexpr int NT = 64 * NW, GPW = 64 / LPR, NG = NW * GPW;
  constexpr int U = VPL >= 16 ? 2 : VPL == 8 ? 2 : 4;  // rows in flight per group
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int sub = lane % LPR, grp = wave * GPW + lane / LPR;
  for (int i = tid; i < a.E; i += NT) hist[i] = 0;
  if (tid == 0) *nv = 0;
  __syncthreads();
  float sum[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) sum[i] = 0.0f;
  for (int t0 = lo + grp; t0 - grp < hi; t0 += NG * U) {
    float x[U][VPL];
    bool live[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * NG;
      live[u] = t < hi && (!a.mask || a.mask[t]);
      load_row<LPR, VPL, VEC>(a.logits + (size_t)t * a.E, a.E, sub, live[u], -INFINITY, x[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      row_softmax<LPR, VPL>(x[u]);
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum[i] += x[u][i];
    }
  }
  // counts, and the number of counting rows
  const int rows = hi - lo;
  const int* ids = a.ids + (size_t)lo * a.k;
  for (int i = tid; i < rows * a.k; i += NT) {
    const int t = lo + i / a.k;
    const int id = ids[i];
    if ((unsigned)id < (unsigned)a.E && (!a.mask || a.mask[t])) atomicAdd(&hist[id], 1);
  }
  for (int i = tid; i < rows; i += NT)
    if (!a.mask || a.mask[lo + i]) atomicAdd(nv, 1);
  // the groups of a wave, then the waves in order
  if constexpr (LPR == 16) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      sum[i] += __shfl_xor(sum[i], 16, 64);
      sum[i] += __shfl_xor(sum[i], 32, 64);
    }
  }
  for (int w = 0; w < NW; ++w) {
    if (wave == w && lane < LPR) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = expert_of<LPR, VEC>(sub, i);
        if (e < a.E) acc[e] = w == 0 ? sum[i] : acc[e] + sum[i];
      }
    }
    __syncthreads();
  }
}

// loss of one sequence from its counts and sums (device layout), by one wave.
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

__device__ __forceinline__ float loss_of(double dot, int E, int k, int n) {
  return n > 0 ? (float)(dot * (double)E / ((double)k * (double)n * (double)n)) : 0.0f;
}

template <int NW, int LPR, int VPL, bool VEC, bool FINAL>
__global__ __launch_bounds__(64 * NW) void balance_partial_kernel(BalArgs a) {
  __shared__ float acc[kMaxE];
  __shared__ int hist[kMaxE];
  __shared__ int nv;
  constexpr int NT = 64 * NW;
  const int tid = threadIdx.x, lane = tid & 63;
  const int c = (int)blockIdx.x;
  const int t0 = c * a.R, t1 = FINAL ? a.T : min(a.T, t0 + a.R);
  for (int s = FINAL ? 0 : first_seq(a.seq, a.S, t0); s < a.S; ++s) {
    int lo, hi;
    seq_rows(a.seq, s, a.T, lo, hi);
    if (!FINAL && lo >= t1) break;
    lo = max(lo, t0);
    hi = min(hi, t1);
    if (FINAL || hi > lo) {
      balance_piece<NW, LPR, VPL, VEC>(a, lo, hi, acc, hist, &nv);
      const int n = nv;
      const size_t o = FINAL ? (size_t)s * a.E : (size_t)(c + s) * a.E;
      float* po = FINAL ? a.probs : a.part_p;
      int* co = FINAL ? a.counts : a.part_c;
      for (int i = tid; i < a.E; i += NT) {
        po[o + i] = acc[i];
        co[o + i] = hist[i];
      }
      if (tid == 0) (FINAL ? a.n_tokens[s] : a.part_n[c + s]) = n;
      if constexpr (FINAL) {
        if (tid < 64) {
          double dot = 0.0;
          for (int i = lane; i < a.E; i += 64) dot += (double)acc[i] * (double)hist[i];
          dot = wave_sum_f64(dot);
          if (lane == 0) a.loss[s] = loss_of(dot, a.E, a.k, n);
        }
      }
      __syncthreads();  // acc, hist and nv are reused by the next piece
    }
  }
}

// One workgroup per sequence: its pieces' sums in chunk order (thread =
// (expert, one of W interleaved chunk lanes), the lanes then added in order).
constexpr int kFinNT = 1024;
__global__ __launch_bounds__(kFinNT) void balance_final_kernel(BalArgs a) {
  __shared__ double sp[kFinNT];
  __shared__ int sc[kFinNT];
  __shared__ double wdot[kFinNT / 64];
  __shared__ int sn;
  const int tid = threadIdx.x, lane = tid & 63;
  const int s = (int)blockIdx.x;
  int lo, hi;
  seq_rows(a.seq, s, a.T, lo, hi);
  const int c0 = lo / a.R, c1 = hi > lo ? (hi - 1) / a.R + 1 : c0;
  const int W = kFinNT / a.E;  // E <= 1024
  const int e = tid % a.E, cl = tid / a.E;
  double p = 0.0;
  int c = 0;
  if (cl < W)
    for (int i = c0 + cl; i < c1; i += W) {
      const size_t o = (size_t)(i + s) * a.E + e;
      p += (double)a.part_p[o];
      c += a.part_c[o];
    }
  sp[tid] = p;
  sc[tid] = c;
  if (tid == 0) sn = 0;
  __syncthreads();
  int n = 0;
  for (int i = c0 + tid; i < c1; i += kFinNT) n += a.part_n[i + s];
  if (n) atomicAdd(&sn, n);
  double dot = 0.0;
  if (tid < a.E) {
    for (int w = 1; w < W; ++w) {
      p += sp[w * a.E + tid];
      c += sc[w * a.E + tid];
    }
    const float pf = (float)p;
    a.probs[(size_t)s * a.E + tid] = pf;
    a.counts[(size_t)s * a.E + tid] = c;
    dot = p * (double)c;
  }
  dot = wave_sum_f64(dot);
  if (lane == 0) wdot[tid >> 6] = dot;
  __syncthreads();
  if (tid == 0) {
    double d = 0.0;
#pragma unroll
    for (int w = 0; w < kFinNT / 64; ++w) d += wdot[w];
    a.n_tokens[s] = sn;
    a.loss[s] = loss_of(d, a.E, a.k, sn);
  }
}

// Gradient: a group of LPR lanes per row, R rows per workgroup of 4 waves.
template <int LPR, int VPL, bool VEC>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteBwdArgs a) {
  constexpr int GPW = 64 / LPR, NG = 4 * GPW;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int sub = lane % LPR, grp = wave * GPW + lane / LPR;
  const int t0 = (int)blockIdx.x * a.R, t1 = min(a.T, t0 + a.R);
  int s = -1, lo = 0, hi = 0;
  float ac[VPL];  // a_s c_se of the current sequence
#pragma unroll
  for (int i = 0; i < VPL; ++i) ac[i] = 0.0f;
  int s_next = first_seq(a.seq, a.S, t0);
  for (int t = t0 + grp; t - grp < t1; t += NG) {
    // the row's sequence (per group; every lane of the group agrees)
    while (s_next < a.S && t >= hi) {
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
    const bool inside = t < t1 && s >= 0 && t >= lo && t < hi;
    const bool live = inside && (!a.mask || a.mask[t]);
    float p[VPL];
    load_row<LPR, VPL, VEC>(a.logits + (size_t)t * a.E, a.E, sub, live, -INFINITY, p);
    // routing weights: lane j < k of the group holds assignment j
    int id = -1;
    float w = 0.0f, wd = 0.0f;
    if (a.dw && live && sub < a.k) {
      const size_t o = (size_t)t * a.k + sub;
      id = a.ids[o];
      if ((unsigned)id >= (unsigned)a.E) id = -1;
      w = id < 0 ? 0.0f : a.w[o];
      wd = id < 0 ? 0.0f : w * a.dw[o];
    }
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
#pragma unroll
        for (int i = 0; i < VPL; ++i) p[i] += expert_of<LPR, VEC>(sub, i) == idj ? v : 0.0f;
      }
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
  size_t p, c, n, total;
};
BalWs bal_ws(int T, int E, int S) {
  const size_t slots = (size_t)(T + chunk_rows(T) - 1) / chunk_rows(T) + (size_t)S;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  BalWs w;
  w.p = 0;
  w.c = up(slots * E * 4);
  w.n = w.c + up(slots * E * 4);
  w.total = w.n + up(slots * 4);
  return w;
}

int check_router_args(const char* who, int T, int E, int k, const int* seq, int S) {
  if (T < 0 || E < 1 || E > kMaxE || k < 1 || k > E || k > kMaxK)
    return set_error(MOE_ERR_INVALID_ARG, "%s: need T>=0, 1<=E<=%d, 1<=k<=min(E,%d) "
                     "(T=%d E=%d k=%d)", who, kMaxE, kMaxK, T, E, k);
  if (S < 1 || S > (1 << 20) || (!seq && S != 1))
    return set_error(MOE_ERR_INVALID_ARG, "%s: S=%d sequences (1..2^20; 1 without seq_offsets)",
                     who, S);
  if ((int64_t)T * k > (1 << 28))
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
  a.n_tokens = n_tokens;
  a.counts = counts;
  a.probs = probs;
  a.loss = loss;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (T <= kMaxChunk) {  // one chunk: finished by the first kernel
    with_row_shape(E, [&](auto r) {
      using Q = decltype(r);
      balance_partial_kernel<16, Q::lpr, Q::vpl, Q::vec, true><<<1, 1024, 0, s>>>(a);
    });
    return check_launch(who);
  }
  const unsigned chunks = (unsigned)((T + a.R - 1) / a.R);
  with_row_shape(E, [&](auto r) {
    using Q = decltype(r);
    balance_partial_kernel<4, Q::lpr, Q::vpl, Q::vec, false><<<chunks, 256, 0, s>>>(a);
  });
  balance_final_kernel<<<(unsigned)S, kFinNT, 0, s>>>(a);
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
  a.R = 32;
  const unsigned blocks = (unsigned)((T + a.R - 1) / a.R);
  with_row_shape(E, [&](auto r) {
    using Q = decltype(r);
    route_backward_kernel<Q::lpr, Q::vpl, Q::vec>
        <<<blocks, 256, 0, reinterpret_cast<hipStream_t>(stream)>>>(a);
  });
  return check_launch(who);
}
