// Tokens into expert order and back, with weights applied, and the gradients of both and of the
// combine (A = T*k assignments a = t*k + j, row inv[a] of the expert order, weight w[a]):
//   scatter:  out[inv[a]] = bf16(w[a] src[t])         dot[a] = <other[inv[a]], src[t]>
//   gather:   out[t] = bf16(sum_j w[a] src[inv[a]] (+ add[t]))   dot[a] = <src[inv[a]], x[t]>
// moe_dispatch and moe_combine_backward are scatters (y_perm as `other`), moe_dispatch_backward
// is the gather.  An inv[a] outside [0, R) is a dropped assignment: nothing is read or written
// for it and its dot is 0.
//   Both are bound by HBM.  A token's row is touched once and its k rows of the expert order once
// each: a wave owns 512 columns of a token (16 bytes per lane) and has the loads of all k rows in
// flight together.  Products and sums are fp32, one rounding to bf16; dots add a lane's products
// column by column, then the lanes and waves of a token in a fixed order.
//   The four waves of a workgroup share a token of more than 512 columns, so that all of its loads
// are issued at once, and take a token each of up to 512.  us, one wave a token / four (scatter,
// gather, scatter with dots; 8 rows a token, of the 512 columns 2): 64 tokens of 2048
// 4.7 5.1 7.6 / 2.9 2.9 4.4, 8192 of 2048 68 67 131 / 60 62 119, 65536 of 512 39 41 69 / 51 45 79.
//   Batches of more rows than the memory-side cache holds bypass it (NT).  us, through it / past it,
// the same: 8192 tokens of 2048 60 62 119 / 53 54 114, 16384 of 7168 422 425 803 / 421 390 794: 4.8 to
// 5.4 TB/s.  (The tokens' rows go by the cache in the plain scatter: 429 without.)  Smaller ones are
// left where the next call finds them.
#include "fp8_common.h"
#include "moe_internal.h"
#include "nontemporal.h"

namespace moe {
namespace {

struct RowArgs {
  const uint16_t* src;
  const uint16_t* other;  // scatter: rows of the dots; gather: x
  const uint16_t* add;
  const int* inv;
  const float* w;
  uint16_t* out;
  float* dot;
  int T, k, H, R;
};

struct F8 {
  float v[8];
};
__device__ __forceinline__ F8 unpack(const uint4& q) {
  F8 r;
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(w[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return r;
}
__device__ __forceinline__ uint4 pack(const F8& r) {
  return uint4{bf16_pack2(r.v[0], r.v[1]), bf16_pack2(r.v[2], r.v[3]), bf16_pack2(r.v[4], r.v[5]),
               bf16_pack2(r.v[6], r.v[7])};
}
__device__ __forceinline__ float dot8(const F8& a, const F8& b, float s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(a.v[i], b.v[i], s);
  return s;
}

// KM: assignments of a token in registers (k <= KM).  NW waves share a token's columns (and its
// dots, through LDS); a workgroup is 4 waves, so it holds 4 / NW tokens.
template <bool GATHER, bool DOT, int KM, int NW, bool NT>
__global__ __launch_bounds__(256) void rows_kernel(RowArgs p) {
  __shared__ float part[DOT ? 4 : 1][DOT ? KM : 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t = (int)blockIdx.x * (4 / NW) + wave / NW, sub = wave % NW;
  const bool live = t < p.T;
  float dots[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) dots[j] = 0.f;
  if (live) {
    int row[KM];
    float wt[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      const size_t a = (size_t)t * p.k + (j < p.k ? j : 0);
      const int r = p.inv[a];
      row[j] = j < p.k && r >= 0 && r < p.R ? r : -1;
      wt[j] = p.w ? p.w[a] : 1.f;
    }
    for (int c = (sub * 64 + lane) * 8; c < p.H; c += NW * 512) {
      const size_t at = (size_t)t * p.H + c;
      uint4 v[KM];
      if (GATHER || DOT) {
        const uint16_t* rows = GATHER ? p.src : p.other;
#pragma unroll
        for (int j = 0; j < KM; ++j)
          v[j] = row[j] >= 0 ? load16<NT>(rows + (size_t)row[j] * p.H + c) : uint4{0, 0, 0, 0};
      }
      if constexpr (GATHER) {
        F8 x, s;
        if (DOT) x = unpack(load16<NT>(p.other + at));
        uint4 q{0, 0, 0, 0};
        if (p.add) q = load16<NT>(p.add + at);
#pragma unroll
        for (int i = 0; i < 8; ++i) s.v[i] = 0.f;
#pragma unroll
        for (int j = 0; j < KM; ++j) {
          if (row[j] < 0) continue;  // uniform
          const F8 r = unpack(v[j]);
#pragma unroll
          for (int i = 0; i < 8; ++i) s.v[i] = fmaf(wt[j], r.v[i], s.v[i]);
          if (DOT) dots[j] = dot8(r, x, dots[j]);
        }
        if (p.add) {
          const F8 r = unpack(q);
#pragma unroll
          for (int i = 0; i < 8; ++i) s.v[i] += r.v[i];
        }
        store16<NT>(p.out + at, pack(s));
      } else {
        const uint4 q = load16<NT && DOT>(p.src + at);
        const F8 x = unpack(q);
        if (DOT) {
#pragma unroll
          for (int j = 0; j < KM; ++j)
            if (row[j] >= 0) dots[j] = dot8(unpack(v[j]), x, dots[j]);
        }
#pragma unroll
        for (int j = 0; j < KM; ++j) {
          if (row[j] < 0) continue;
          uint4 o = q;  // without weights a copy of the bits
          if (p.w) {
            F8 r;
#pragma unroll
            for (int i = 0; i < 8; ++i) r.v[i] = wt[j] * x.v[i];
            o = pack(r);
          }
          store16<NT>(p.out + (size_t)row[j] * p.H + c, o);
        }
      }
    }
  }
  if constexpr (DOT) {
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      const float s = wave_sum_f32(dots[j]);
      if (lane == 0) part[wave][j] = s;
    }
    __syncthreads();
    if (live && sub == 0 && lane < p.k) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) s += part[wave + i][lane];
      p.dot[(size_t)t * p.k + lane] = s;
    }
  }
}

// A grid has fewer than 2^32 threads: a batch goes in slices of 2^23 workgroups (of one token each or four).
template <bool GATHER, bool DOT, int KM>
int launch_k(RowArgs p, hipStream_t s, const char* who) {
  const bool nt = (int64_t)p.T * p.k * p.H * 2 >= kMemorySideCache;
  const int per = p.H > 512 ? 1 : 4;
  for (int left = p.T;;) {
    p.T = left < per << 23 ? left : per << 23;
    const unsigned grid = (unsigned)((p.T + per - 1) / per);
    auto launch = [&](auto kernel) { kernel<<<grid, 256, 0, s>>>(p); };
    if (per == 1) launch(nt ? rows_kernel<GATHER, DOT, KM, 4, true> : rows_kernel<GATHER, DOT, KM, 4, false>);
    else launch(nt ? rows_kernel<GATHER, DOT, KM, 1, true> : rows_kernel<GATHER, DOT, KM, 1, false>);
    if (int st = check_launch(who)) return st;
    left -= p.T;
    if (left == 0) return MOE_OK;
    // what goes by token; the rows in expert order are the whole batch's
    const size_t a = (size_t)p.T * p.k, rows = (size_t)p.T * p.H;
    p.inv += a;
    if (p.w) p.w += a;
    if (p.dot) p.dot += a;
    if (GATHER) {
      p.out += rows;
      if (p.add) p.add += rows;
      if (p.other) p.other += rows;
    } else {
      p.src += rows;
    }
  }
}

template <bool GATHER, bool DOT>
int launch(const RowArgs& p, hipStream_t s, const char* who) {
  if (p.k <= 2) return launch_k<GATHER, DOT, 2>(p, s, who);
  if (p.k <= 4) return launch_k<GATHER, DOT, 4>(p, s, who);
  if (p.k <= 8) return launch_k<GATHER, DOT, 8>(p, s, who);
  return launch_k<GATHER, DOT, 16>(p, s, who);
}

int check_rows(const char* who, int32_t T, int32_t k, int32_t H, int32_t R) {
  if (T < 0 || k < 1 || k > kMaxK || H < 8 || H % 8 || R < 0)
    return set_error(MOE_ERR_INVALID_ARG, "%s: need T>=0, 1<=k<=%d, H a multiple of 8, R>=0 "
                     "(T=%d k=%d H=%d R=%d)", who, kMaxK, T, k, H, R);
  if ((int64_t)T * k > (int64_t)1 << 27 || R > 1 << 27)
    return set_error(MOE_ERR_UNSUPPORTED, "%s: more than 2^27 assignments or rows", who);
  return MOE_OK;
}

bool bad(const void* p) { return !p || !aligned16(p); }
bool misaligned(const void* p) { return p && !aligned16(p); }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_dispatch(const uint16_t* x, const int32_t* inv_idx, const float* topk_w, int32_t T,
                            int32_t k, int32_t H, int32_t R, uint16_t* x_perm, moe_stream_t stream) {
  const char* who = "moe_dispatch";
  if (int st = check_rows(who, T, k, H, R)) return st;
  if (T == 0) return MOE_OK;
  if (bad(x) || bad(inv_idx) || misaligned(topk_w) || (R > 0 && bad(x_perm)))
    return set_error(MOE_ERR_INVALID_ARG, "%s: null or misaligned pointer", who);
  RowArgs p{};
  p.src = x; p.inv = inv_idx; p.w = topk_w; p.out = x_perm;
  p.T = T; p.k = k; p.H = H; p.R = R;
  return launch<false, false>(p, reinterpret_cast<hipStream_t>(stream), who);
}

extern "C" int moe_dispatch_backward(const uint16_t* d_x_perm, const int32_t* inv_idx,
                                     const float* topk_w, const uint16_t* x, int32_t T, int32_t k,
                                     int32_t H, int32_t R, const uint16_t* d_add, uint16_t* d_x,
                                     float* d_topk_w, moe_stream_t stream) {
  const char* who = "moe_dispatch_backward";
  if (int st = check_rows(who, T, k, H, R)) return st;
  if (T == 0) return MOE_OK;
  if ((R > 0 && bad(d_x_perm)) || bad(inv_idx) || misaligned(topk_w) || misaligned(d_add) ||
      bad(d_x) || misaligned(d_topk_w) || (d_topk_w && bad(x)))
    return set_error(MOE_ERR_INVALID_ARG, "%s: null or misaligned pointer", who);
  RowArgs p{};
  p.src = d_x_perm; p.other = x; p.add = d_add; p.inv = inv_idx; p.w = topk_w; p.out = d_x;
  p.dot = d_topk_w;
  p.T = T; p.k = k; p.H = H; p.R = R;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return d_topk_w ? launch<true, true>(p, s, who) : launch<true, false>(p, s, who);
}

extern "C" int moe_combine_backward(const uint16_t* d_y, const uint16_t* y_perm,
                                    const int32_t* inv_idx, const float* topk_w, int32_t T, int32_t k,
                                    int32_t H, int32_t R, uint16_t* d_y_perm, float* d_topk_w,
                                    moe_stream_t stream) {
  const char* who = "moe_combine_backward";
  if (int st = check_rows(who, T, k, H, R)) return st;
  if (T == 0) return MOE_OK;
  if (bad(d_y) || bad(inv_idx) || bad(topk_w) || (R > 0 && bad(d_y_perm)) || misaligned(d_topk_w) ||
      (d_topk_w && R > 0 && bad(y_perm)))
    return set_error(MOE_ERR_INVALID_ARG, "%s: null or misaligned pointer", who);
  RowArgs p{};
  p.src = d_y; p.other = y_perm; p.inv = inv_idx; p.w = topk_w; p.out = d_y_perm; p.dot = d_topk_w;
  p.T = T; p.k = k; p.H = H; p.R = R;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return d_topk_w ? launch<false, true>(p, s, who) : launch<false, false>(p, s, who);
}
