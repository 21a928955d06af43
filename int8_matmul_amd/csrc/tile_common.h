// What the tiled products (gemm.hip, backward.hip) share: loads from global
// memory straight into LDS, the chunk permutations of their LDS rows, and the
// barrier that ends a stage.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

namespace li8 {

#define LI8_LDS __attribute__((address_space(3)))

// Buffer resource over `bytes` bytes at p (raw buffer, offsets in bytes).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *p, int bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, bytes, 0x00020000);
}

// 16 bytes per lane from rsrc at voffset + soffset into LDS at lds + 16*lane.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, void *lds, int voffset,
                                            int soffset)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LI8_LDS void *)lds, 16, voffset, soffset, 0, 0);
}

// B (4 or 16) bytes per lane from rsrc at voffset into LDS at lds + B*lane.
// (Called from a device function: the builtin written inside a kernel's
// lambda makes the host pass drop the kernel's launch stub.)
template <int B>
__device__ __forceinline__ void load_to_lds_n(__amdgpu_buffer_rsrc_t r, void *lds, int voffset)
{
    static_assert(B == 4 || B == 16, "bytes per lane");
    if constexpr (B == 4)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LI8_LDS void *)lds, 4, voffset, 0, 0, 0);
    else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LI8_LDS void *)lds, 16, voffset, 0, 0, 0);
}

template <int CPR>
__device__ __forceinline__ int swz(int row)
{
    static_assert(CPR == 4 || CPR == 8, "16-byte chunks per LDS row");
    if constexpr (CPR == 8)
        return (row ^ (row >> 3)) & 7;
    else
        return ((row >> 1) ^ (row >> 3)) & 3;
}

// Wait until at most N buffer loads of this wave are in flight and all its
// LDS reads are done, then barrier.  The compiler does not track the LDS
// writes of buffer_load ... lds, so this wait is what orders them.
template <int N>
__device__ __forceinline__ void wait_loads_barrier()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

constexpr int kOutOfRange = (int)0x80000000;   // buffer offset past any operand

// f(integral_constant<int, I>) for each I of the sequence, in order.
template <int... I, class F>
__device__ __forceinline__ void for_each_index(std::integer_sequence<int, I...>, F &&f)
{
    (f(std::integral_constant<int, I>{}), ...);
}

// 16 bytes per lane from each lane's own global address into LDS at lds + 16*lane.
__device__ __forceinline__ void load_to_lds_at(const void *src, void *lds)
{
    __builtin_amdgcn_global_load_lds(
        (__attribute__((address_space(1))) void *)const_cast<void *>(src), (LI8_LDS void *)lds, 16, 0, 0);
}

// 16-byte chunk c of row r of a staging tile of CPR chunks a row without
// padding, as an offset in bytes: chunks are permuted so that 32 rows' writes of
// one column spread over the banks.
template <int CPR>
__device__ __forceinline__ int stage_off(int r, int c)
{
    static_assert(CPR == 4 || CPR == 8 || CPR == 12, "16-byte chunks per staging row");
    if constexpr (CPR == 8)
        return (r * CPR + (c ^ ((r >> 1) & 7))) * 16;
    else
        return (r * CPR + (c ^ ((r >> 2) & 3))) * 16;
}

} // namespace li8
