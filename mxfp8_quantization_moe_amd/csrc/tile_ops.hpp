// Building blocks of the matrix products: loads straight into LDS, the waits
// that go with them, fragment reads, the order of workgroups over the XCDs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float float4v __attribute__((ext_vector_type(4)));

// 16 bytes per lane from global memory straight into LDS: lane l's bytes go to
// lds + 16 l (lds wave-uniform).  The waits are explicit (wait_tiles).
__device__ __forceinline__ void load_lds16(const void *src, uint32_t lds)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                     (__attribute__((address_space(3))) void *)(uintptr_t)lds, 16, 0, 0);
}

// At most PENDING of this wave's loads into LDS are still on their way and its
// LDS reads have returned; then the workgroup meets.
template <int PENDING>
__device__ __forceinline__ void wait_stage()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\t"
                 "s_barrier"
                 :
                 : "n"(PENDING)
                 : "memory");
}

// four rows (summed dim) by 16 columns of f16, one column per lane: lane i of
// 16 points at row i / 4, columns 4 (i % 4) and receives column i of all four
__device__ __forceinline__ half4 read_transposed(uint32_t a)
{
    typedef short short4v __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(half4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) short4v *)(uintptr_t)a));
}

__device__ __forceinline__ half8 read_lds(uint32_t a)
{
    return *(__attribute__((address_space(3))) const half8 *)(uintptr_t)a;
}

// Workgroups go to the 8 XCDs in turn; this numbering gives each XCD a
// contiguous run of 0..total-1.
__device__ __forceinline__ int xcd_run(int block, int total)
{
    const int xcd = block & 7;
    return xcd * (total >> 3) + min(xcd, total & 7) + (block >> 3);
}

// End of a phase: this wave's LDS reads have returned, at most PENDING of its
// loads are still on their way (-1: whatever), and the workgroup meets.
template <int PENDING>
__device__ __forceinline__ void phase_end()
{
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (PENDING >= 0)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(PENDING) : "memory");
    else
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

}  // namespace mxq
