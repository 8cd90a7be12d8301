// Device helpers shared by the gfx950 kernels of this library.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <tuple>
#include <type_traits>
#include <utility>

namespace q4k {

typedef _Float16 f16;
typedef f16 f16x2 __attribute__((ext_vector_type(2)));
typedef f16 f16x4 __attribute__((ext_vector_type(4)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Bytes of one Q4_0 / Q8_0 block of 32 elements.
constexpr int kQ4Bytes = 18;
constexpr int kQ8Bytes = 34;

// 32-bit load from an address that is only 2-byte aligned. The HSA ABI runs
// gfx9 wavefronts in unaligned-access mode, so this is one global_load_dword.
__device__ __forceinline__ uint32_t load_u32_unaligned(const uint8_t *p)
{
    uint32_t v;
    __builtin_memcpy(&v, p, 4);
    return v;
}

// 16-bit load from a 2-byte aligned address.
__device__ __forceinline__ uint32_t load_u16(const uint8_t *p)
{
    return *reinterpret_cast<const uint16_t *>(p);
}

// Widen a binary16 bit pattern to f32 (exact).
__device__ __forceinline__ float f16_bits_to_f32(uint32_t bits)
{
    return (float)__builtin_bit_cast(f16, (uint16_t)bits);
}

// f32 -> binary16 bit pattern, round to nearest even (v_cvt_f16_f32).
__device__ __forceinline__ uint32_t f32_to_f16_bits(float v)
{
    return (uint32_t)__builtin_bit_cast(uint16_t, (f16)v);
}

template <typename T, typename U>
__device__ __forceinline__ T bitcast(U u)
{
    static_assert(sizeof(T) == sizeof(U), "size mismatch");
    return __builtin_bit_cast(T, u);
}

// Largest of a non-negative 32-bit value over the wavefront, in every lane:
// DPP within quads, half-rows and rows, then one readlane per row.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v)
{
    int x = (int)v;
    x = (int)max((uint32_t)x, (uint32_t)__builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, false));    // quad_perm 1,0,3,2
    x = (int)max((uint32_t)x, (uint32_t)__builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, false));    // quad_perm 2,3,0,1
    x = (int)max((uint32_t)x, (uint32_t)__builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, false));   // row_half_mirror
    x = (int)max((uint32_t)x, (uint32_t)__builtin_amdgcn_mov_dpp(x, 0x140, 0xF, 0xF, false));   // row_mirror
    return max(max((uint32_t)__builtin_amdgcn_readlane(x, 0), (uint32_t)__builtin_amdgcn_readlane(x, 16)),
               max((uint32_t)__builtin_amdgcn_readlane(x, 32), (uint32_t)__builtin_amdgcn_readlane(x, 48)));
}

// f(integral_constant<int, 0>{}) .. f(integral_constant<int, N - 1>{}), in order:
// a loop whose index is a constant, however long its body.
template <class F, int... I>
__device__ __forceinline__ void unroll_impl(F &&f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void unroll(F &&f)
{
    unroll_impl(f, std::make_integer_sequence<int, N>{});
}

// Direct-to-LDS loads of 16 and of 4 bytes a lane: lane l's bytes go to dst +
// 16 l (4 l).
__device__ __forceinline__ void load16_to_lds(__amdgpu_buffer_rsrc_t r, void *dst, uint32_t off, int base)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)dst, 16, off, base, 0, 0);
}
__device__ __forceinline__ void load4_to_lds(__amdgpu_buffer_rsrc_t r, void *dst, uint32_t off, int base)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)dst, 4, off, base, 0, 0);
}

// Launch a kernel and return the runtime's verdict on this launch alone. Each
// argument is first converted to the kernel's own parameter type. A grid
// dimension holds fewer than 2^32 threads; past that the runtime can launch a
// part of the grid and report success, so it is refused here.
template <typename Kernel, typename Tuple, size_t... I>
inline hipError_t launch_tuple(Kernel kernel, dim3 grid, dim3 block, size_t lds_bytes,
                               hipStream_t stream, Tuple &vals, std::index_sequence<I...>)
{
    void *argv[] = {reinterpret_cast<void *>(&std::get<I>(vals))...};
    return hipLaunchKernel(reinterpret_cast<const void *>(kernel), grid, block, argv, lds_bytes,
                           stream);
}

template <typename... Params, typename... Args>
inline hipError_t launch_kernel(void (*kernel)(Params...), dim3 grid, dim3 block, size_t lds_bytes,
                                hipStream_t stream, Args &&...args)
{
    static_assert(sizeof...(Params) == sizeof...(Args), "argument count");
    if ((uint64_t)grid.x * block.x > UINT32_MAX || (uint64_t)grid.y * block.y > UINT32_MAX ||
        (uint64_t)grid.z * block.z > UINT32_MAX)
        return hipErrorInvalidConfiguration;
    std::tuple<std::decay_t<Params>...> vals(std::forward<Args>(args)...);
    return launch_tuple(kernel, grid, block, lds_bytes, stream, vals,
                        std::index_sequence_for<Params...>{});
}

// A grid of any number of workgroups in x, 2^31 threads a launch (a multiple of
// 64 workgroups): the kernel's last parameter is the index of its first one.
template <typename... Params, typename... Args>
inline hipError_t launch_parts(void (*kernel)(Params...), long long blocks, unsigned blocks_y,
                               unsigned threads, hipStream_t stream, Args &&...args)
{
    const long long part = (1LL << 31) / threads / 64 * 64;
    hipError_t e = hipSuccess;
    for (long long first = 0; first < blocks && e == hipSuccess; first += part)
        e = launch_kernel(kernel, dim3((unsigned)(blocks - first < part ? blocks - first : part), blocks_y),
                          dim3(threads), 0, stream, args..., (int)first);
    return e;
}

}  // namespace q4k
