// 32 bytes a lane: one access where the address is 32-byte aligned, else two of 16.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace clsa {

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* x) {  // p 32-byte aligned
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
               "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}
__device__ __forceinline__ void st_32(void* p, const uint32_t* x, bool wide) {
  if (wide) {
    st_global_v8(p, x);
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    static_cast<uint4*>(p)[1] = make_uint4(x[4], x[5], x[6], x[7]);
  }
}
// read once: not kept in L1
__device__ __forceinline__ void ld_stream_32(const void* p, uint4& a, uint4& b, bool wide) {
  if (wide) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
  } else {
    a = ld_stream_v4(p);
    b = ld_stream_v4(static_cast<const char*>(p) + 16);
  }
}

}  // namespace clsa
