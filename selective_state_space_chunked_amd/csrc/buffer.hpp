// Buffer accesses: the address is scalar, a lane adds its byte offset in 32 bits, and offsets from `bytes` on read
// as zero and are not written.
#pragma once
#include "common.hpp"

namespace ssm {

typedef __amdgpu_buffer_rsrc_t buffer_t;
__device__ __forceinline__ buffer_t buffer_of(const void* at, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(at), 0, bytes, 0x00027000);
}
template <typename T> __device__ __forceinline__ T buffer_load(buffer_t r, uint32_t off, uint32_t row = 0);
template <> __device__ __forceinline__ int8_t buffer_load<int8_t>(buffer_t r, uint32_t off, uint32_t row) {
    return (int8_t)__builtin_amdgcn_raw_buffer_load_b8(r, off, row, 0);
}
template <> __device__ __forceinline__ bf16_t buffer_load<bf16_t>(buffer_t r, uint32_t off, uint32_t row) {
    return __builtin_amdgcn_raw_buffer_load_b16(r, off, row, 0);
}
template <> __device__ __forceinline__ float buffer_load<float>(buffer_t r, uint32_t off, uint32_t row) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off, row, 0));
}
__device__ __forceinline__ void buffer_store(buffer_t r, uint32_t off, bf16_t v) {
    __builtin_amdgcn_raw_buffer_store_b16(v, r, off, 0, 0);
}
__device__ __forceinline__ void buffer_store(buffer_t r, uint32_t off, float v) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, off, 0, 0);
}

}  // namespace ssm
