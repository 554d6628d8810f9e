// f4_quant.cu -- microscaled 4-bit floating point: tensor scale, quantiser,
// dequantiser and embedding lookup (formats and rounding rules in w4.h).
//
// All four move bytes and nothing else: the quantiser reads 2 or 4 bytes and
// writes 0.53 (MX) or 0.56 (NV) per element, the other way round for the
// dequantiser.  A lane owns 8 consecutive elements, so that a warp's loads and
// code stores are contiguous (128 bytes of codes, 512 or 1024 of elements);
// the lanes of a block (4 for MX, 2 for NV) find its largest magnitude with
// shuffles, and the lanes of 4 blocks join their scale bytes into the one
// 4-byte word that the scale tile holds for them.
#include <cuda_bf16.h>

#include "f4.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLaneElems = 8;
constexpr int kWarpElems = 32 * kLaneElems;  // 256 consecutive k

// ---------------------------------------------------------------------------
// loads and stores of 8 elements
// ---------------------------------------------------------------------------

template <int IN>
struct Raw8 {  // 8 elements as loaded
    uint4 a;
};
template <>
struct Raw8<W4_IN_F32> {
    uint4 a, b;
};

template <int IN>
__device__ __forceinline__ Raw8<IN> load8(const void* x, int64_t elem) {
    Raw8<IN> r;
    if constexpr (IN == W4_IN_F32) {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(x) + elem);
        r.a = __ldg(s);
        r.b = __ldg(s + 1);
    } else {
        r.a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + elem));
    }
    return r;
}

template <int IN>
__device__ __forceinline__ void widen8(const Raw8<IN>& r, float (&v)[8]) {
    if constexpr (IN == W4_IN_F32) {
        const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
        const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (IN == W4_IN_BF16) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
}

// Bits of the largest magnitude of 8 values: for non-negative floats the
// integer order of the bits is the numeric order, with infinity and then NaN
// on top.
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
}

constexpr uint32_t kInfBits = 0x7F800000u;

// Eight fp32 values -> eight e2m1 codes (nearest even, saturating), element i
// in bits 4i..4i+3.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}\n"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight e2m1 codes -> fp32.
__device__ __forceinline__ void from_e2m1x8(uint32_t c, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

template <int OUT>
__device__ __forceinline__ void store8(void* y, int64_t elem, const float (&v)[8]) {
    if constexpr (OUT == W4_OUT_F32) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(y) + elem);
        d[0] = make_float4(v[0], v[1], v[2], v[3]);
        d[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + elem) =
            make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// ---------------------------------------------------------------------------
// tensor scale
// ---------------------------------------------------------------------------

__device__ __forceinline__ float tensor_scale_of(uint32_t amax) {
    return fmaxf(__fdiv_rn(__uint_as_float(amax), 2688.0f), 0x1p-100f);
}

// g = max over blocks of threads of tensor_scale_of(their amax): the quotient
// and the lower bound are monotone in amax, so the maximum of the scales is
// the scale of the maximum, and the integer order of the positive floats makes
// it one atomicMax, whose result does not depend on the order.  *g is 0 before.
template <int IN>
__global__ void __launch_bounds__(kThreads) tensor_scale_kernel(const void* __restrict__ x,
                                                                int64_t chunks,
                                                                float* __restrict__ g, int* err) {
    constexpr int kU = 4;
    uint32_t m = 0;
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < chunks; i += stride * kU) {
        Raw8<IN> r[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            // past the end: the first chunk again, which changes no maximum
            const int64_t c = i + u * stride < chunks ? i + u * stride : i;
            if (W4_CHECK(c >= 0 && c < chunks, err)) r[u] = load8<IN>(x, c * kLaneElems);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            float v[8];
            widen8<IN>(r[u], v);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t b = __float_as_uint(v[k]) & 0x7FFFFFFFu;
                m = max(m, b < kInfBits ? b : 0u);
            }
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    __shared__ uint32_t part[kWarps];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < kWarps; ++i) m = max(m, part[i]);
        atomicMax(reinterpret_cast<unsigned int*>(g), __float_as_uint(tensor_scale_of(m)));
    }
}

// ---------------------------------------------------------------------------
// quantiser
// ---------------------------------------------------------------------------

// Scale byte of a block and the factor that its elements are multiplied by.
template <int FMT>
__device__ __forceinline__ void block_scale(uint32_t amax, float g, uint32_t& byte, float& inv) {
    if (amax >= kInfBits) {  // a NaN or an infinity in the block: codes 0, scale NaN
        byte = FMT == W4_F4_MX ? 255u : 127u;
        inv = 0.0f;
    } else if constexpr (FMT == W4_F4_MX) {
        // floor(log2(amax)) - 2 from the exponent field; fields 0..2 take 2^-127
        const uint32_t e = amax >> 23;
        byte = e > 2u ? e - 2u : 0u;
        inv = __uint_as_float((254u - byte) << 23);
    } else {
        const float t = __fdiv_rn(__uint_as_float(amax), __fmul_rn(6.0f, g));
        byte = __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
        const float den = __fmul_rn(f4::scale_value<W4_F4_NV>(byte), g);
        inv = den == 0.0f ? 0.0f : __frcp_rn(den);
    }
}

// One warp takes 256 consecutive k of one row at a time.  blockIdx.y walks the
// row's segments, blockIdx.x and the warp the rows, those that only pad the
// last scale tile among them.
template <int FMT, int IN>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const void* __restrict__ x, int64_t R,
                                                            int64_t K,
                                                            const float* __restrict__ gp,
                                                            uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales,
                                                            int* err) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kBlkLanes = f4::block_of(FMT) / kLaneElems;  // lanes of a block
    constexpr int kWordLanes = 4 * kBlkLanes;                  // lanes of a scale word
    const int lane = threadIdx.x & 31;
    const float g = FMT == W4_F4_NV ? __ldg(gp) : 1.0f;
    const int64_t tiles_k = f4::scale_tiles_k(K, FMT);
    const int64_t rows = f4::row_tiles(R) * f4::kRowTile;
    const int64_t kpad = tiles_k * 4 * f4::block_of(FMT);
    for (int64_t r = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); r < rows;
         r += (int64_t)gridDim.x * kWarps) {
        for (int64_t k0 = (int64_t)blockIdx.y * kWarpElems; k0 < kpad;
             k0 += (int64_t)gridDim.y * kWarpElems) {
            const int64_t k = k0 + lane * kLaneElems;
            const bool live = r < R && k < K;  // the same for all lanes of a block
            float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (live && W4_CHECK(k + kLaneElems <= K, err)) widen8<IN>(load8<IN>(x, r * K + k), v);
            uint32_t amax = amax_bits(v);
#pragma unroll
            for (int off = 1; off < kBlkLanes; off <<= 1)
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            uint32_t byte;
            float inv;
            block_scale<FMT>(amax, g, byte, inv);
            const bool bad = amax >= kInfBits;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = bad ? 0.0f : __fmul_rn(v[i], inv);
            const uint32_t c = e2m1x8(v);
            // the scale bytes of 4 blocks, joined across their lanes
            uint32_t word = live ? byte << (8 * (lane / kBlkLanes % 4)) : 0u;
#pragma unroll
            for (int off = kBlkLanes; off < kWordLanes; off <<= 1)
                word |= __shfl_xor_sync(0xffffffffu, word, off);
            if (live) *reinterpret_cast<uint32_t*>(codes + (r * K + k) / 2) = c;
            if (lane % kWordLanes == 0 && k < kpad) {
                const int64_t at = f4::scale_word(r, k / (4 * f4::block_of(FMT)), tiles_k);
                if (W4_CHECK(at + 4 <= f4::row_tiles(R) * tiles_k * f4::kTileBytes, err))
                    *reinterpret_cast<uint32_t*>(scales + at) = word;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// dequantiser and embedding lookup
// ---------------------------------------------------------------------------

// Output row t is table row ids[t] (or t, without ids) times `alpha` and g.
// A task is 256 consecutive k of one output row, one per warp and step.
template <int FMT, int OUT, bool LOOKUP>
__global__ void __launch_bounds__(kThreads)
    rows_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                const float* __restrict__ gp, int64_t V, int64_t K,
                const int64_t* __restrict__ ids, int64_t T, float alpha, void* __restrict__ y,
                int* err) {
    const int lane = threadIdx.x & 31;
    const float c = FMT == W4_F4_NV ? __fmul_rn(__ldg(gp), alpha) : alpha;
    const int64_t tiles_k = f4::scale_tiles_k(K, FMT);
    for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < T;
         t += (int64_t)gridDim.x * kWarps) {
        const int64_t row = LOOKUP ? __ldg(ids + t) : t;
        const bool live = row >= 0 && row < V;
        for (int64_t k0 = (int64_t)blockIdx.y * kWarpElems; k0 < K;
             k0 += (int64_t)gridDim.y * kWarpElems) {
            const int64_t k = k0 + lane * kLaneElems;
            if (k >= K || !W4_CHECK(k + kLaneElems <= K && t < T, err)) continue;
            float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (live) {
                const int64_t b = k / f4::block_of(FMT);
                const uint32_t q = __ldg(reinterpret_cast<const uint32_t*>(codes + (row * K + k) / 2));
                const float s = f4::scale_value<FMT>(
                    __ldg(scales + f4::scale_word(row, b >> 2, tiles_k) + (b & 3)));
                from_e2m1x8(q, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], s), c);
            }
            store8<OUT>(y, t * K + k, v);
        }
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

bool shape_ok(int64_t R, int64_t K) {
    return R >= 0 && R <= f4::kMaxRows && K >= 0 && K <= f4::kMaxK && K % 32 == 0;
}

// Rows over blockIdx.x, a row's 256-element segments over blockIdx.y: about
// eight CTAs per SM in all, the rows first.
dim3 grid_for(int64_t rows, int64_t segments) {
    const int64_t cap = (int64_t)w4::sm_count() * 8;
    int64_t gx = (rows + kWarps - 1) / kWarps;
    if (gx > cap) gx = cap;
    int64_t gy = cap / gx;
    if (gy > segments) gy = segments;
    return dim3((unsigned)gx, (unsigned)gy);
}

template <int FMT>
int launch_quantize(const void* x, int in, int64_t R, int64_t K, const float* g, uint8_t* codes,
                    uint8_t* scales, cudaStream_t st) {
    const int64_t rows = f4::row_tiles(R) * f4::kRowTile;
    const int64_t kpad = f4::scale_tiles_k(K, FMT) * 4 * f4::block_of(FMT);
    const dim3 grid = grid_for(rows, (kpad + kWarpElems - 1) / kWarpElems);
    int* err = w4::device_error_word();
    if (in == W4_IN_BF16)
        quantize_kernel<FMT, W4_IN_BF16><<<grid, kThreads, 0, st>>>(x, R, K, g, codes, scales, err);
    else if (in == W4_IN_F32)
        quantize_kernel<FMT, W4_IN_F32><<<grid, kThreads, 0, st>>>(x, R, K, g, codes, scales, err);
    else
        quantize_kernel<FMT, W4_IN_F16><<<grid, kThreads, 0, st>>>(x, R, K, g, codes, scales, err);
    return w4::launch_status();
}

template <int FMT, bool LOOKUP>
int launch_rows(const uint8_t* codes, const uint8_t* scales, const float* g, int64_t V, int64_t K,
                const int64_t* ids, int64_t T, float alpha, void* y, int out, cudaStream_t st) {
    const dim3 grid = grid_for(T, (K + kWarpElems - 1) / kWarpElems);
    int* err = w4::device_error_word();
    if (out == W4_OUT_F32)
        rows_kernel<FMT, W4_OUT_F32, LOOKUP>
            <<<grid, kThreads, 0, st>>>(codes, scales, g, V, K, ids, T, alpha, y, err);
    else
        rows_kernel<FMT, W4_OUT_BF16, LOOKUP>
            <<<grid, kThreads, 0, st>>>(codes, scales, g, V, K, ids, T, alpha, y, err);
    return w4::launch_status();
}

}  // namespace

extern "C" {

size_t f4_scale_bytes(int64_t R, int64_t K, int format) {
    if (!shape_ok(R, K) || !f4::known_format(format)) return 0;
    return (size_t)(f4::row_tiles(R) * f4::scale_tiles_k(K, format) * f4::kTileBytes);
}

int f4_tensor_scale(const void* x, int in_dtype, int64_t R, int64_t K, float* g, void* stream) {
    if (!shape_ok(R, K) || !f4::known_in(in_dtype)) return W4_ERR_SHAPE;
    const int64_t chunks = R * K / kLaneElems;
    if (!g || (chunks > 0 && !x)) return W4_ERR_NULL;
    if ((chunks > 0 && !w4::aligned16(x)) || (reinterpret_cast<uintptr_t>(g) & 3u))
        return W4_ERR_ALIGN;
    const int rc = w4::check_device();
    if (rc != W4_OK) return rc;
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = cudaMemsetAsync(g, 0, sizeof(float), st);
    if (e != cudaSuccess) return w4::cuda_fail(e);
    int64_t ctas = (chunks + kThreads - 1) / kThreads;
    const int64_t cap = (int64_t)w4::sm_count() * 8;
    if (ctas > cap) ctas = cap;
    if (ctas < 1) ctas = 1;  // no elements: g = 2^-100
    int* err = w4::device_error_word();
    if (in_dtype == W4_IN_BF16)
        tensor_scale_kernel<W4_IN_BF16><<<(int)ctas, kThreads, 0, st>>>(x, chunks, g, err);
    else if (in_dtype == W4_IN_F32)
        tensor_scale_kernel<W4_IN_F32><<<(int)ctas, kThreads, 0, st>>>(x, chunks, g, err);
    else
        tensor_scale_kernel<W4_IN_F16><<<(int)ctas, kThreads, 0, st>>>(x, chunks, g, err);
    return w4::launch_status();
}

int f4_quantize(const void* x, int in_dtype, int64_t R, int64_t K, int format, const float* g,
                uint8_t* codes, uint8_t* scales, void* stream) {
    if (!shape_ok(R, K) || !f4::known_in(in_dtype) || !f4::known_format(format))
        return W4_ERR_SHAPE;
    if (R == 0 || K == 0) return W4_OK;
    if (!x || !codes || !scales || (format == W4_F4_NV && !g)) return W4_ERR_NULL;
    if (!w4::aligned16(x) || !w4::aligned16(codes) || !w4::aligned16(scales) ||
        (format == W4_F4_NV && (reinterpret_cast<uintptr_t>(g) & 3u)))
        return W4_ERR_ALIGN;
    const int rc = w4::check_device();
    if (rc != W4_OK) return rc;
    return format == W4_F4_MX
               ? launch_quantize<W4_F4_MX>(x, in_dtype, R, K, g, codes, scales, (cudaStream_t)stream)
               : launch_quantize<W4_F4_NV>(x, in_dtype, R, K, g, codes, scales, (cudaStream_t)stream);
}

int f4_dequantize(const uint8_t* codes, const uint8_t* scales, const float* g, int64_t R,
                  int64_t K, int format, void* y, int out_dtype, void* stream) {
    if (!shape_ok(R, K) || !f4::known_format(format) || !f4::known_out(out_dtype))
        return W4_ERR_SHAPE;
    if (R == 0 || K == 0) return W4_OK;
    if (!codes || !scales || !y || (format == W4_F4_NV && !g)) return W4_ERR_NULL;
    if (!w4::aligned16(codes) || !w4::aligned16(scales) || !w4::aligned16(y) ||
        (format == W4_F4_NV && (reinterpret_cast<uintptr_t>(g) & 3u)))
        return W4_ERR_ALIGN;
    const int rc = w4::check_device();
    if (rc != W4_OK) return rc;
    const cudaStream_t st = (cudaStream_t)stream;
    return format == W4_F4_MX
               ? launch_rows<W4_F4_MX, false>(codes, scales, g, R, K, nullptr, R, 1.0f, y, out_dtype, st)
               : launch_rows<W4_F4_NV, false>(codes, scales, g, R, K, nullptr, R, 1.0f, y, out_dtype, st);
}

int f4_embed(const uint8_t* codes, const uint8_t* scales, const float* g, int64_t V, int64_t K,
             int format, const int64_t* ids, int64_t T, float alpha, void* y, int out_dtype,
             void* stream) {
    if (V < 1 || !shape_ok(V, K) || T < 0 || T > f4::kMaxRows || !f4::known_format(format) ||
        !f4::known_out(out_dtype))
        return W4_ERR_SHAPE;
    if (T == 0 || K == 0) return W4_OK;
    if (!codes || !scales || !ids || !y || (format == W4_F4_NV && !g)) return W4_ERR_NULL;
    if (!w4::aligned16(codes) || !w4::aligned16(scales) || !w4::aligned16(y) ||
        (reinterpret_cast<uintptr_t>(ids) & 7u) ||
        (format == W4_F4_NV && (reinterpret_cast<uintptr_t>(g) & 3u)))
        return W4_ERR_ALIGN;
    const int rc = w4::check_device();
    if (rc != W4_OK) return rc;
    const cudaStream_t st = (cudaStream_t)stream;
    return format == W4_F4_MX
               ? launch_rows<W4_F4_MX, true>(codes, scales, g, V, K, ids, T, alpha, y, out_dtype, st)
               : launch_rows<W4_F4_NV, true>(codes, scales, g, V, K, ids, T, alpha, y, out_dtype, st);
}

}  // extern "C"
