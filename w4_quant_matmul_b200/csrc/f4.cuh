// f4.cuh -- the microscaled 4-bit floating-point format shared by the f4_*
// translation units: scale-plane geometry, scale bytes, host argument checks.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace f4 {

constexpr int64_t kMaxK = 131072;
constexpr int64_t kMaxRows = int64_t(1) << 24;

constexpr int kRowTile = 128;    // rows of a scale tile
constexpr int kTileBytes = 512;  // 128 rows x 4 blocks

// Elements of k that share a scale, by format.
__host__ __device__ constexpr int block_of(int fmt) { return fmt == W4_F4_MX ? 32 : 16; }

// Scale tiles along K (4 blocks each).
__host__ __device__ constexpr int64_t scale_tiles_k(int64_t K, int fmt) {
    return (K / block_of(fmt) + 3) / 4;
}

__host__ __device__ constexpr int64_t row_tiles(int64_t R) {
    return (R + kRowTile - 1) / kRowTile;
}

// Byte offset, in its scale plane, of the 4-byte word that holds blocks
// 4 * kt ... 4 * kt + 3 of row r.
__device__ __forceinline__ int64_t scale_word(int64_t r, int64_t kt, int64_t tiles_k) {
    return ((r >> 7) * tiles_k + kt) * kTileBytes + (r & 31) * 16 + ((r & 127) >> 5) * 4;
}

// fp32 value of a scale byte.
template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t byte) {
    if constexpr (FMT == W4_F4_MX) {
        // 2^(byte - 127): the byte is the fp32 exponent; 0 is the subnormal
        // 2^-127 and 255 NaN
        return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
    } else {
        // Bits 0-6 alone: the tensor cores read the byte as an unsigned number too.  The
        // sign is dropped from the result, where it costs nothing (bit 7 cleared ahead
        // of the conversion: 1237 x 9728 dequantised to fp32 in 9.8 us instead of 8.5).
        const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3);
        return fabsf(__half2float(__half(h)));
    }
}

// A sum's factor a * b, as two factors to apply one after the other: 1 and their
// product where that is a normal number.  Elsewhere the product itself would lose its
// bits or overflow although the sum brings the result back into range (a tensor
// scale of 2^-100 times one of 2^-55, with sums up to 2^23 K): then the larger one
// first.  What that leaves of the sum only leaves the range where the result does:
// below 2^-126 the smaller one is less than 2^-63, above 2^128 more than 1.
struct Factors {
    float first, second;
};
__device__ __forceinline__ Factors factors(float a, float b) {
    const float p = __fmul_rn(a, b);
    if (fabsf(p) >= 0x1p-126f && fabsf(p) <= 3.402823466e38f) return {1.0f, p};
    return fabsf(a) >= fabsf(b) ? Factors{a, b} : Factors{b, a};
}
__device__ __forceinline__ float times(float v, const Factors& f) {
    return v * f.first * f.second;
}

// Programmatic dependent launch.  Every f4 kernel waits for the kernel before it
// ahead of its first access to global memory -- f4_gemv's product: to anything but
// weights; the tensor scale: to anything but x, which the kernel before it never
// writes -- and lets the kernel after it start once it has waited (the digit
// kernel of f4_gemv at once).  The quantiser, which writes what f4_gemv reads
// early, does not let the next kernel start early at all.  What another kernel may
// write while this one is already there is not loaded through the read-only path
// (__ldca, not __ldg).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launch that may start while the kernel before it on the stream still runs.
template <typename... Params, typename... Args>
int launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t stream,
                     Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
    if (e != cudaSuccess) return w4::cuda_fail(e);
    return w4::launch_status();
}

// Host checks of a format and an out_dtype.
inline bool known_format(int fmt) { return fmt == W4_F4_MX || fmt == W4_F4_NV; }
inline bool known_out(int t) { return t == W4_OUT_BF16 || t == W4_OUT_F32; }
inline bool known_in(int t) { return t == W4_IN_BF16 || t == W4_IN_F32 || t == W4_IN_F16; }

}  // namespace f4
