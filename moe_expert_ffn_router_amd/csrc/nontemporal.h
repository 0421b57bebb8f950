// 16-byte accesses that may bypass the caches: data of more than the memory-side cache holds, that
// is touched once, otherwise only turns out what other accesses (and the write-back of what they
// leave behind) could use.
#pragma once

#include "moe_internal.h"

namespace moe {

constexpr int64_t kMemorySideCache = (int64_t)256 << 20;  // bytes

typedef unsigned int nt_u32x4 __attribute__((ext_vector_type(4)));

template <bool NT>
__device__ __forceinline__ uint4 load16(const void* p) {
  const nt_u32x4* a = static_cast<const nt_u32x4*>(p);
  const nt_u32x4 v = NT ? __builtin_nontemporal_load(a) : *a;
  return uint4{v[0], v[1], v[2], v[3]};
}

template <bool NT>
__device__ __forceinline__ void store16(void* p, const uint4& v) {
  const nt_u32x4 w = {v.x, v.y, v.z, v.w};
  nt_u32x4* a = static_cast<nt_u32x4*>(p);
  if (NT) __builtin_nontemporal_store(w, a);
  else *a = w;
}

}  // namespace moe
