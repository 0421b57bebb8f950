// Clipping by the global norm: norm = sqrt(sum of the squares of every element of every
// gradient), scale = min(1, max_norm / (norm + 1e-6)), out_i = scale * grad_i.
//   Squares and sums are in 64 bits: the square of any bf16 or fp32 value is exact or rounded at
// 2^-53 and in range, so one huge or many tiny elements lose nothing (HBM bounds the pass all the
// same).  The order of the sums depends on the sizes alone.
//   The tensors travel as kernel arguments, kSet of them per launch: no table has to be copied to
// the device, so a captured graph replays the call as it was.  Every tensor is cut into chunks of
// kChunkUnits 16-byte units from the 16-byte boundary at or below its first element; the units
// across its ends are taken element by element, so any element-aligned view works and nothing
// outside it is read.
//   Norm pass: workgroups take the launch's chunks in strides and leave one partial sum each.
// Clip pass: every workgroup adds the partial sums itself (they are few and in the L2), which
// saves a launch between the passes; several launches of tensors: one finishing kernel.  In place
// with scale 1, the clip pass ends there.
//   Gradients of more bytes than the memory-side cache holds bypass it in both passes (NT): 1.6 GB
// clipped into other tensors 921 -> 850 us, 5.8 TB/s over the three times it moves them; bypassing
// the cache with the loads or the stores alone 925 and 893.  Fewer are in the cache for the
// second pass.  Outputs that lie otherwise in their 16 bytes than their gradients are written element by
// element (1.6 GB of bf16: 2407 us instead of 823).
#include <algorithm>
#include <new>
#include <utility>
#include <vector>

#include "fp8_common.h"
#include "moe_internal.h"
#include "nontemporal.h"

namespace moe {
namespace {

constexpr int kSet = 128;            // tensors per launch (kernel arguments are 4 KB at most)
constexpr int kChunkUnits = 2048;    // 16-byte units of a chunk: 32 KB, 8 loads per thread
constexpr int kMaxParts = 2048;      // partial sums of one launch

struct ClipSet {
  const uint8_t* src[kSet];
  uint8_t* dst[kSet];           // clip pass
  uint64_t numel[kSet];         // bit 63: fp32
  uint32_t first_chunk[kSet + 1];
  int n;
};
static_assert(sizeof(ClipSet) + 64 <= 4096, "kernel arguments");

struct Piece {
  const uint8_t* src;
  uint8_t* dst;
  uint64_t lo, hi;   // bytes of the tensor, from the 16-byte boundary at or below it
  uint64_t unit0;    // first unit of the chunk
  bool f32;
};

__device__ __forceinline__ Piece piece_of(const ClipSet& s, uint32_t chunk) {
  int lo = 0, hi = s.n - 1;  // the last tensor with first_chunk <= chunk
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (s.first_chunk[m] <= chunk) lo = m;
    else hi = m - 1;
  }
  Piece p;
  const uint64_t n = s.numel[lo];
  p.f32 = n >> 63;
  const uintptr_t a = (uintptr_t)s.src[lo];
  p.src = (const uint8_t*)(a & ~(uintptr_t)15);
  p.lo = a & 15;
  p.hi = p.lo + ((n & ~(1ull << 63)) << (p.f32 ? 2 : 1));
  p.dst = s.dst[lo] - p.lo;
  p.unit0 = (uint64_t)(chunk - s.first_chunk[lo]) * kChunkUnits;
  return p;
}

// Whether unit u lies within the tensor, and whether any of it does.
__device__ __forceinline__ bool whole(const Piece& p, uint64_t u) {
  return u * 16 >= p.lo && u * 16 + 16 <= p.hi;
}
__device__ __forceinline__ bool any(const Piece& p, uint64_t u) {
  return u * 16 + 16 > p.lo && u * 16 < p.hi;
}

__device__ __forceinline__ double square(float f, double s) {
  const double d = (double)f;
  return fma(d, d, s);
}
__device__ __forceinline__ double squares(uint4 q, bool f32, double s) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (f32) {
      s = square(__uint_as_float(w[i]), s);
    } else {
      s = square(__uint_as_float(w[i] << 16), s);
      s = square(__uint_as_float(w[i] & 0xffff0000u), s);
    }
  }
  return s;
}

// Sum over a workgroup of 256, in a fixed order, in every thread.
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

template <bool NT>
__global__ __launch_bounds__(256) void norm_kernel(ClipSet s, uint32_t chunks, double* parts) {
  __shared__ double lds[4];
  double sum = 0;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Piece p = piece_of(s, c);
    constexpr int U = kChunkUnits / 256;
    if (whole(p, p.unit0) && whole(p, p.unit0 + kChunkUnits - 1)) {
      uint4 q[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        q[i] = load16<NT>(p.src + (p.unit0 + i * 256 + threadIdx.x) * 16);
#pragma unroll
      for (int i = 0; i < U; ++i) sum = squares(q[i], p.f32, sum);
    } else {
      for (int i = 0; i < U; ++i) {
        const uint64_t u = p.unit0 + i * 256 + threadIdx.x;
        if (whole(p, u)) {
          sum = squares(*reinterpret_cast<const uint4*>(p.src + u * 16), p.f32, sum);
        } else if (any(p, u)) {
          const int step = p.f32 ? 4 : 2;
          for (int b = 0; b < 16; b += step) {
            const uint64_t at = u * 16 + b;
            if (at < p.lo || at >= p.hi) continue;
            sum = square(p.f32 ? *reinterpret_cast<const float*>(p.src + at)
                               : bf16_to_f32(*reinterpret_cast<const uint16_t*>(p.src + at)), sum);
          }
        }
      }
    }
  }
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) parts[blockIdx.x] = sum;
}

// The norm and the scale from the partial sums, by one workgroup of 256.
__device__ __forceinline__ float2 finish(const double* parts, int n, float max_norm, double* lds) {
  double sum = 0;
  for (int i = threadIdx.x; i < n; i += 256) sum += parts[i];
  const double norm = sqrt(block_sum(sum, lds));
  // a norm that is NaN gives a scale of NaN, an infinite one 0 (without a limit: 1)
  const double c = isinf(max_norm) && !isnan(norm) ? 1.0 : (double)max_norm / (norm + 1e-6);
  return float2{(float)norm, (float)(c >= 1.0 ? 1.0 : c)};
}

__global__ __launch_bounds__(256) void finish_kernel(const double* parts, int n, float max_norm,
                                                     float* norm_scale) {
  __shared__ double lds[4];
  const float2 r = finish(parts, n, max_norm, lds);
  if (threadIdx.x == 0) {
    norm_scale[0] = r.x;
    norm_scale[1] = r.y;
  }
}

__device__ __forceinline__ uint4 scaled(uint4 q, bool f32, float f) {
  uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = f32 ? __float_as_uint(__uint_as_float(w[i]) * f)
               : bf16_pack2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
  return uint4{w[0], w[1], w[2], w[3]};
}

// FINISH: the norm is formed here (parts of one launch); else it is read from norm_scale.
template <bool FINISH, bool NT>
__global__ __launch_bounds__(256) void clip_kernel(ClipSet s, uint32_t chunks, const double* parts,
                                                   int n_parts, float max_norm, float* norm_scale) {
  __shared__ double lds[4];
  float f;
  if constexpr (FINISH) {
    const float2 r = finish(parts, n_parts, max_norm, lds);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      norm_scale[0] = r.x;
      norm_scale[1] = r.y;
    }
    f = r.y;
  } else {
    f = norm_scale[1];
  }
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Piece p = piece_of(s, c);
    if (f == 1.f && p.src == p.dst) continue;  // in place and unclipped
    const bool same = (((uintptr_t)p.dst) & 15) == 0;  // both sides aligned alike
    constexpr int U = kChunkUnits / 256;
    if (same && whole(p, p.unit0) && whole(p, p.unit0 + kChunkUnits - 1)) {
      uint4 q[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        q[i] = load16<NT>(p.src + (p.unit0 + i * 256 + threadIdx.x) * 16);
#pragma unroll
      for (int i = 0; i < U; ++i)
        store16<NT>(p.dst + (p.unit0 + i * 256 + threadIdx.x) * 16, scaled(q[i], p.f32, f));
    } else {
      for (int i = 0; i < U; ++i) {
        const uint64_t u = p.unit0 + i * 256 + threadIdx.x;
        if (same && whole(p, u)) {
          *reinterpret_cast<uint4*>(p.dst + u * 16) =
              scaled(*reinterpret_cast<const uint4*>(p.src + u * 16), p.f32, f);
        } else if (any(p, u)) {
          const int step = p.f32 ? 4 : 2;
          for (int b = 0; b < 16; b += step) {
            const uint64_t at = u * 16 + b;
            if (at < p.lo || at >= p.hi) continue;
            if (p.f32)
              *reinterpret_cast<float*>(p.dst + at) = *reinterpret_cast<const float*>(p.src + at) * f;
            else
              *reinterpret_cast<uint16_t*>(p.dst + at) = (uint16_t)bf16_pack2(
                  bf16_to_f32(*reinterpret_cast<const uint16_t*>(p.src + at)) * f, 0.f);
          }
        }
      }
    }
  }
}

int parts_of(int64_t sets) {  // partial sums that one of `sets` launches may leave
  const int64_t v = kMaxParts / sets;
  return (int)(v < 64 ? 64 : v);
}

int64_t chunks_of(const void* p, int64_t numel, bool f32) {
  const uint64_t bytes = ((uintptr_t)p & 15) + ((uint64_t)numel << (f32 ? 2 : 1));
  return (int64_t)((bytes + kChunkUnits * 16 - 1) / (kChunkUnits * 16));
}

struct Range {
  uintptr_t lo, hi;
  int32_t tensor;
  bool out;
};

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_clip_grad_norm_workspace(int32_t n) {
  if (n < 0) return 0;
  const int64_t sets = n ? ((int64_t)n + kSet - 1) / kSet : 1;
  return ((size_t)sets * parts_of(sets) * sizeof(double) + 255) / 256 * 256;
}

extern "C" int moe_clip_grad_norm(int32_t n, const void* const* grads, const int64_t* numel,
                                  const int32_t* types, float max_norm, void* const* clipped,
                                  float* norm_scale, void* ws, size_t ws_bytes, moe_stream_t stream) {
  const char* who = "moe_clip_grad_norm";
  if (n < 0 || n > 1 << 16)
    return set_error(MOE_ERR_INVALID_ARG, "%s: need 0 <= n <= 65536 (n=%d)", who, n);
  if (!(max_norm >= 0.f)) return set_error(MOE_ERR_INVALID_ARG, "%s: max_norm must be >= 0", who);
  if (n > 0 && (!grads || !numel || !types))
    return set_error(MOE_ERR_INVALID_ARG, "%s: null array", who);
  if (!norm_scale || !aligned16(norm_scale) || !ws || !aligned16(ws))
    return set_error(MOE_ERR_INVALID_ARG, "%s: null or misaligned pointer", who);
  if (ws_bytes < moe_clip_grad_norm_workspace(n))
    return set_error(MOE_ERR_WORKSPACE, "%s: workspace %zu too small", who, ws_bytes);
  int64_t bytes = 0;
  for (int i = 0; i < n; ++i) {
    if (types[i] != MOE_T_BF16 && types[i] != MOE_T_F32)
      return set_error(MOE_ERR_UNSUPPORTED, "%s: tensor %d: type %d (bf16 or fp32)", who, i, types[i]);
    if (numel[i] < 0 || numel[i] > (int64_t)1 << 40)
      return set_error(MOE_ERR_INVALID_ARG, "%s: tensor %d: %lld elements", who, i,
                       (long long)numel[i]);
    const uintptr_t mask = types[i] == MOE_T_F32 ? 3 : 1;
    if (numel[i] && (!grads[i] || ((uintptr_t)grads[i] & mask)))
      return set_error(MOE_ERR_INVALID_ARG, "%s: tensor %d: null or misaligned pointer", who, i);
    if (numel[i] && clipped && (!clipped[i] || ((uintptr_t)clipped[i] & mask)))
      return set_error(MOE_ERR_INVALID_ARG, "%s: output %d: null or misaligned pointer", who, i);
    bytes += numel[i] << (types[i] == MOE_T_F32 ? 2 : 1);
  }
  if (clipped && n > 0) {
    // an output may be its own gradient; else no output may touch another or any gradient
    try {
      std::vector<Range> r;
      r.reserve((size_t)2 * n);
      for (int i = 0; i < n; ++i) {
        if (!numel[i]) continue;
        const uintptr_t bytes = (uintptr_t)numel[i] << (types[i] == MOE_T_F32 ? 2 : 1);
        const uintptr_t g = (uintptr_t)grads[i], c = (uintptr_t)clipped[i];
        r.push_back({c, c + bytes, i, true});
        if (g != c) r.push_back({g, g + bytes, i, false});
      }
      std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
      uintptr_t out_end = 0, any_end = 0;  // furthest ends so far, of outputs and of all
      for (const Range& q : r) {
        if (q.lo < out_end || (q.out && q.lo < any_end))
          return set_error(MOE_ERR_INVALID_ARG, "%s: tensor %d overlaps another one or an output", who,
                           q.tensor);
        if (q.out) out_end = std::max(out_end, q.hi);
        any_end = std::max(any_end, q.hi);
      }
    } catch (const std::bad_alloc&) {
      return set_error(MOE_ERR_CAPACITY, "%s: out of host memory", who);
    }
  }
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  double* parts = static_cast<double*>(ws);
  const int64_t sets = n ? ((int64_t)n + kSet - 1) / kSet : 1;
  const int most = parts_of(sets);
  int n_parts = 0;
  // a set of tensors as kernel arguments; its chunks
  auto fill = [&](int first, ClipSet& a) -> int64_t {
    int64_t chunks = 0;
    a.n = 0;
    for (int i = first; i < n && i < first + kSet; ++i) {
      if (!numel[i]) continue;
      const bool f32 = types[i] == MOE_T_F32;
      a.src[a.n] = static_cast<const uint8_t*>(grads[i]);
      a.dst[a.n] = static_cast<uint8_t*>(clipped ? clipped[i] : nullptr);
      a.numel[a.n] = (uint64_t)numel[i] | (f32 ? 1ull << 63 : 0);
      a.first_chunk[a.n] = (uint32_t)chunks;
      chunks += chunks_of(grads[i], numel[i], f32);
      ++a.n;
      if (chunks > ((int64_t)1 << 32) - 1 - kMaxParts) return -1;
    }
    a.first_chunk[a.n] = (uint32_t)chunks;
    return chunks;
  };
  ClipSet a;
  for (int first = 0; first < n; first += kSet)
    if (fill(first, a) < 0) return set_error(MOE_ERR_UNSUPPORTED, "%s: too many elements", who);
  const bool nt = bytes >= kMemorySideCache;
  for (int first = 0; first < n; first += kSet) {
    const int64_t chunks = sets == 1 ? a.first_chunk[a.n] : fill(first, a);
    if (chunks == 0) continue;
    const int grid = (int)(chunks < most ? chunks : most);
    if (nt) norm_kernel<true><<<grid, 256, 0, s>>>(a, (uint32_t)chunks, parts + n_parts);
    else norm_kernel<false><<<grid, 256, 0, s>>>(a, (uint32_t)chunks, parts + n_parts);
    if (int st = check_launch(who)) return st;
    n_parts += grid;
  }
  if (!clipped || sets > 1 || n_parts == 0) {
    finish_kernel<<<1, 256, 0, s>>>(parts, n_parts, max_norm, norm_scale);
    if (int st = check_launch(who)) return st;
    if (!clipped) return MOE_OK;
  }
  for (int first = 0; first < n; first += kSet) {
    const int64_t chunks = sets == 1 ? a.first_chunk[a.n] : fill(first, a);
    if (chunks == 0) continue;
    const int grid = (int)(chunks < kMaxParts ? chunks : kMaxParts);
    auto launch = [&](auto kernel) {
      kernel<<<grid, 256, 0, s>>>(a, (uint32_t)chunks, parts, n_parts, max_norm, norm_scale);
    };
    if (sets == 1) launch(nt ? clip_kernel<true, true> : clip_kernel<true, false>);
    else launch(nt ? clip_kernel<false, true> : clip_kernel<false, false>);
    if (int st = check_launch(who)) return st;
  }
  return MOE_OK;
}
