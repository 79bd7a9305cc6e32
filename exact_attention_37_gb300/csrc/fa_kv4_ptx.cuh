// PTX that only the kernel for trees with many rows uses.
#pragma once
#include "ptx.cuh"

namespace fa {

// warp_wait for a kernel of many warps that wait most of the time: the first look is the whole warp's,
// and a warp that has to wait sleeps in the barrier for up to kNapNs at a time instead of asking again
// and again, which would take issue slots from the warps that work.
constexpr uint32_t kNapNs = 100000;
__device__ __forceinline__ uint32_t mbar_nap(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kNapNs)
      : "memory");
  return ok;
}
__device__ __forceinline__ bool warp_nap(uint32_t bar, uint32_t parity, uint32_t* err, uint32_t code) {
  if (__all_sync(0xffffffffu, mbar_nap(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!__all_sync(0xffffffffu, mbar_nap(bar, parity))) {
    const bool late = globaltimer_ns() - t0 > kWaitLimitNs;
    if (__any_sync(0xffffffffu, late || (*reinterpret_cast<volatile uint32_t*>(err) & kErrAborted))) {
      if (late) record_timeout(err, code, bar);
      __syncwarp();
      return false;
    }
  }
  return true;
}

// A bulk copy's bytes brought into L2 only (a multiple of 16 bytes from an address that is one).
__device__ __forceinline__ void bulk_prefetch(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// One lane of a whole warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t mine;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(mine));
  return mine != 0;
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(tm(taddr, 16)));
}
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(tm(taddr, 8)), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// reg_fence32 for any count.
template <int N>
__device__ __forceinline__ void reg_fence(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i])::"memory");
}

}  // namespace fa
