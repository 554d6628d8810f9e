// f4_quant.cu -- microscaled 4-bit floating point: tensor scale, quantiser,
// dequantiser and embedding lookup (formats and rounding rules in w4.h).
//
// All four move bytes and nothing else: the quantiser reads 2 or 4 bytes and
// writes 0.53 (MX) or 0.56 (NV) per element, the other way round for the
// dequantiser.  A lane owns 8 (NV: 16) consecutive elements, so that a warp's
// loads and code stores are contiguous; the lanes of a block find its largest
// magnitude with shuffles (4 lanes for MX, one for NV), and the lanes of 4 blocks
// join their scale bytes into the one 4-byte word that the scale tile holds for
// them.  HBM bounds them: 8192 x 9728 bf16 quantised in 33.4 us (MX, 6020 GB/s) and
// 35.2 (NV, 5730), turned back into bf16 in 33.8 (5970) and into fp32 in 60.6
// (5950); their scale found in 26.2 (6070).
#include <cuda_bf16.h>

#include "f4.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLaneElems = 8;
constexpr int kRowElems = 1024;  // elements of a row that a warp has in flight

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
        r.a = __ldca(s);
        r.b = __ldca(s + 1);
    } else {
        r.a = __ldca(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + elem));
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

constexpr uint32_t kInfBits = 0x7F800000u;

// Largest magnitude of 8 elements in the order of their own bits: for
// non-negative floats the integer order of the bits is the numeric order, with
// infinity and then NaN on top.  The 16-bit types go two at a time.
template <int IN>
__device__ __forceinline__ uint32_t amax_raw(const Raw8<IN>& r) {
    if constexpr (IN == W4_IN_F32) {
        const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
        return m;
    } else {
        const uint32_t m = __vmaxu2(__vmaxu2(r.a.x & 0x7FFF7FFFu, r.a.y & 0x7FFF7FFFu),
                                    __vmaxu2(r.a.z & 0x7FFF7FFFu, r.a.w & 0x7FFF7FFFu));
        return max(m >> 16, m & 0xFFFFu);
    }
}

// That magnitude as fp32 bits.
template <int IN>
__device__ __forceinline__ uint32_t amax_f32(uint32_t m) {
    if constexpr (IN == W4_IN_F32) return m;
    if constexpr (IN == W4_IN_BF16) return m << 16;
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
}

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

// Four e2m1 codes (low 16 bits) -> fp32.  As fp16 their low bytes are zero; the
// high bytes come from two byte permutations that use the codes as selectors,
// one for the magnitudes and one for the signs.
__device__ __forceinline__ void from_e2m1x4(uint32_t c, float* v) {
    const uint32_t mag = __byte_perm(0x3E3C3800u, 0x46444240u, c & 0x7777u);
    const uint32_t top = mag | __byte_perm(0x00008000u, 0u, (c >> 3) & 0x1111u);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t h = __byte_perm(top, 0u, i ? 0x3424 : 0x1404);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// ---------------------------------------------------------------------------
// tensor scale
// ---------------------------------------------------------------------------

__device__ __forceinline__ float tensor_scale_of(uint32_t amax) {
    return fmaxf(__fdiv_rn(__uint_as_float(amax), 2688.0f), 0x1p-100f);
}

__global__ void clear_scale_kernel(float* g) {
    f4::pdl_wait();
    f4::pdl_trigger();
    *g = 0.0f;
}

// g = max over blocks of threads of tensor_scale_of(their amax): the quotient
// and the lower bound are monotone in amax, so the maximum of the scales is
// the scale of the maximum, and the integer order of the positive floats makes
// it one atomicMax, whose result does not depend on the order.  *g is cleared by
// the kernel before, which let this one start when all before it was complete:
// only g has to be waited for.
constexpr int kScaleLoads = 4;  // of a thread, in flight together

template <int IN>
__global__ void __launch_bounds__(kThreads) tensor_scale_kernel(const void* __restrict__ x,
                                                                int64_t chunks,
                                                                float* __restrict__ g, int* err) {
    uint32_t m = 0;
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < chunks;
         i += stride * kScaleLoads) {
        Raw8<IN> r[kScaleLoads];
#pragma unroll
        for (int u = 0; u < kScaleLoads; ++u) {
            // past the end: the first chunk again, which changes no maximum
            const int64_t c = i + u * stride < chunks ? i + u * stride : i;
            if (W4_CHECK(c >= 0 && c < chunks, err)) r[u] = load8<IN>(x, c * kLaneElems);
        }
#pragma unroll
        for (int u = 0; u < kScaleLoads; ++u) {
            const uint32_t a = amax_f32<IN>(amax_raw<IN>(r[u]));
            if (a < kInfBits) {
                m = max(m, a);
            } else {  // a NaN or an infinity among them: the finite ones one by one
                float v[8];
                widen8<IN>(r[u], v);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t b = __float_as_uint(v[k]) & 0x7FFFFFFFu;
                    m = max(m, b < kInfBits ? b : 0u);
                }
            }
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    __shared__ uint32_t part[kWarps];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    f4::pdl_wait();
    f4::pdl_trigger();
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
// NV (g6 = 6 g, rcp = 1 / g6): the byte is that of the IEEE quotient amax / g6.
// amax * rcp lies within 2^-22 of it; where e4m3 rounds that product less and
// plus 2^-21 to one number, the quotient rounds to it too, and only else is the
// division made (one conversion instruction does both roundings).
template <int FMT>
__device__ __forceinline__ void block_scale(uint32_t amax, float g, float g6, float rcp,
                                            uint32_t& byte, float& inv) {
    if constexpr (FMT == W4_F4_MX) {
        // floor(log2(amax)) - 2 from the exponent field; fields 0..2 take 2^-127
        const uint32_t e = amax >> 23;
        byte = e > 2u ? e - 2u : 0u;
        inv = __uint_as_float((254u - byte) << 23);
    } else {
        const float q = __uint_as_float(amax) * rcp;
        const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(q * (1.0f - 0x1p-21f),
                                                                  q * (1.0f + 0x1p-21f)),
                                                      __NV_SATFINITE, __NV_E4M3);
        byte = two & 0xFFu;
        if (byte != two >> 8)
            byte = __nv_cvt_float_to_fp8(__fdiv_rn(__uint_as_float(amax), g6), __NV_SATFINITE,
                                         __NV_E4M3);
        const float den = __fmul_rn(f4::scale_value<W4_F4_NV>(byte), g);
        inv = den == 0.0f ? 0.0f : __frcp_rn(den);
    }
    if (amax >= kInfBits) byte = FMT == W4_F4_MX ? 255u : 127u;  // a NaN or an infinity
}

// Elements of a lane: half an MX block or a whole NV block, whose scale takes
// more work (8 elements a lane for NV: 8192 x 9728 bf16 in 41.9 us, now 35.4).
constexpr int quant_elems(int fmt) { return fmt == W4_F4_MX ? 8 : 16; }

// A warp takes up to 1024 consecutive k of one row, all loads before the first
// use.  blockIdx.x and the warp select the row, those that only pad the last
// scale tile among them, blockIdx.y the part of it.
template <int FMT, int IN>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const void* __restrict__ x, int64_t R,
                                                            int K,
                                                            const float* __restrict__ gp,
                                                            uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales,
                                                            int* err) {
    f4::pdl_wait();
    // no early start for the kernel after this one: it may be f4_gemv, which reads
    // the planes written here before it waits
    constexpr int kElems = quant_elems(FMT), kOct = kElems / 8;
    constexpr int kSpan = 32 * kElems;
    constexpr int kU = kRowElems / kSpan;
    constexpr int kBlkLanes = f4::block_of(FMT) / kElems;  // lanes of a block
    constexpr int kWordLanes = 4 * kBlkLanes;              // lanes of a scale word
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int tiles_k = (int)f4::scale_tiles_k(K, FMT);
    const int kpad = tiles_k * 4 * f4::block_of(FMT);
    const int k0 = blockIdx.y * kRowElems + lane * kElems;
    const bool row = r < R;
    Raw8<IN> raw[kU][kOct];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int k = k0 + u * kSpan;
#pragma unroll
        for (int o = 0; o < kOct; ++o) {
            raw[u][o] = Raw8<IN>{};
            if (row && k < K && W4_CHECK(k + kElems <= K, err))
                raw[u][o] = load8<IN>(x, r * K + k + 8 * o);
        }
    }
    const float g = FMT == W4_F4_NV ? __ldca(gp) : 1.0f;
    const float g6 = __fmul_rn(6.0f, g), rcp = __frcp_rn(g6);
    uint8_t* code_row = codes + r * (K / 2);
    uint8_t* scale_row = scales + f4::scale_word(r, 0, tiles_k);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int k = k0 + u * kSpan;
        if (k - lane * kElems >= kpad) break;  // the same for the whole warp
        const bool live = row && k < K;  // the same for all lanes of a block
        uint32_t m = amax_raw<IN>(raw[u][0]);
#pragma unroll
        for (int o = 1; o < kOct; ++o) m = max(m, amax_raw<IN>(raw[u][o]));
#pragma unroll
        for (int off = 1; off < kBlkLanes; off <<= 1)
            m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
        const uint32_t amax = amax_f32<IN>(m);
        uint32_t byte;
        float inv;
        block_scale<FMT>(amax, g, g6, rcp, byte, inv);
        uint32_t c[kOct];
#pragma unroll
        for (int o = 0; o < kOct; ++o) {
            float v[8];
            widen8<IN>(raw[u][o], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], inv);
            c[o] = amax >= kInfBits ? 0u : e2m1x8(v);
        }
        // the scale bytes of 4 blocks, joined across their lanes
        uint32_t word = live ? byte << (8 * (lane / kBlkLanes % 4)) : 0u;
#pragma unroll
        for (int off = kBlkLanes; off < kWordLanes; off <<= 1)
            word |= __shfl_xor_sync(0xffffffffu, word, off);
        if (live && W4_CHECK(r >= 0 && r < R && k + kElems <= K, err)) {
            if constexpr (kOct == 2)
                *reinterpret_cast<uint2*>(code_row + k / 2) = make_uint2(c[0], c[1]);
            else
                *reinterpret_cast<uint32_t*>(code_row + k / 2) = c[0];
        }
        if (lane % kWordLanes == 0 && k < kpad &&
            W4_CHECK(r < f4::row_tiles(R) * f4::kRowTile, err))
            *reinterpret_cast<uint32_t*>(scale_row + k / (4 * f4::block_of(FMT)) * f4::kTileBytes) =
                word;
    }
}

// ---------------------------------------------------------------------------
// dequantiser and embedding lookup
// ---------------------------------------------------------------------------

// Output row t is table row ids[t] (or t, without ids) times `alpha` and g.  A
// lane owns 16 bytes of output, so that a warp's stores are contiguous; a warp
// takes up to 1024 elements of one row, all loads before the first use (fp32 in
// halves of that: 39.4 us for 19456 x 2560 instead of 37.8).
template <int FMT, int OUT, bool LOOKUP>
__global__ void __launch_bounds__(kThreads)
    rows_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                const float* __restrict__ gp, int64_t V, int K,
                const int64_t* __restrict__ ids, int64_t T, float alpha, void* __restrict__ y,
                int* err) {
    f4::pdl_wait();
    f4::pdl_trigger();
    constexpr int kElems = OUT == W4_OUT_F32 ? 4 : 8;  // of a lane
    constexpr int kSpan = 32 * kElems;                 // of a warp
    constexpr int kU = kRowElems / kSpan;
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= T) return;
    const int64_t row = LOOKUP ? __ldca(ids + t) : t;
    const bool live = row >= 0 && row < V;
    const uint8_t* code_row = codes + row * (K / 2);
    const uint8_t* scale_row = scales + f4::scale_word(row, 0, f4::scale_tiles_k(K, FMT));
    const int k0 = blockIdx.y * kRowElems + lane * kElems;
    uint32_t q[kU], sb[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int k = k0 + u * kSpan;
        q[u] = sb[u] = 0u;
        if (live && k < K && W4_CHECK(k + kElems <= K, err)) {
            const uint8_t* c = code_row + k / 2;
            if constexpr (kElems == 8)
                q[u] = __ldca(reinterpret_cast<const uint32_t*>(c));
            else
                q[u] = __ldca(reinterpret_cast<const uint16_t*>(c));
            const int b = k / f4::block_of(FMT);
            sb[u] = __ldca(scale_row + (b >> 2) * f4::kTileBytes + (b & 3));
        }
    }
    const float c = FMT == W4_F4_NV ? __fmul_rn(__ldca(gp), alpha) : alpha;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int k = k0 + u * kSpan;
        if (k >= K) break;
        if (!W4_CHECK(t >= 0 && t < T && k + kElems <= K, err)) break;
        float v[kElems];
#pragma unroll
        for (int i = 0; i < kElems; i += 4) from_e2m1x4(q[u] >> (4 * i), v + i);
        const float s = f4::scale_value<FMT>(sb[u]);
#pragma unroll
        for (int i = 0; i < kElems; ++i) {
            v[i] = __fmul_rn(v[i], s);  // exact
            if constexpr (LOOKUP || FMT == W4_F4_NV) v[i] = __fmul_rn(v[i], c);
            if constexpr (LOOKUP) v[i] = live ? v[i] : 0.0f;
        }
        if constexpr (OUT == W4_OUT_F32) {
            *reinterpret_cast<float4*>(static_cast<float*>(y) + t * K + k) =
                make_float4(v[0], v[1], v[2], v[3]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + t * K + k) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

bool shape_ok(int64_t R, int64_t K) {
    return R >= 0 && R <= f4::kMaxRows && K >= 0 && K <= f4::kMaxK && K % 32 == 0;
}

// A warp for each row and kRowElems of its elements.
dim3 grid_for(int64_t rows, int64_t K) {
    return dim3((unsigned)((rows + kWarps - 1) / kWarps), (unsigned)((K + kRowElems - 1) / kRowElems));
}

template <int FMT>
int launch_quantize(const void* x, int in, int64_t R, int64_t K, const float* g, uint8_t* codes,
                    uint8_t* scales, cudaStream_t st) {
    const int64_t rows = f4::row_tiles(R) * f4::kRowTile;
    const int64_t kpad = f4::scale_tiles_k(K, FMT) * 4 * f4::block_of(FMT);
    const dim3 grid = grid_for(rows, kpad);
    int* err = w4::device_error_word();
    auto kernel = in == W4_IN_BF16  ? quantize_kernel<FMT, W4_IN_BF16>
                  : in == W4_IN_F32 ? quantize_kernel<FMT, W4_IN_F32>
                                    : quantize_kernel<FMT, W4_IN_F16>;
    return f4::launch_dependent(kernel, grid, kThreads, st, x, R, (int)K, g, codes, scales, err);
}

template <int FMT, bool LOOKUP>
int launch_rows(const uint8_t* codes, const uint8_t* scales, const float* g, int64_t V, int64_t K,
                const int64_t* ids, int64_t T, float alpha, void* y, int out, cudaStream_t st) {
    int* err = w4::device_error_word();
    const bool f32 = out == W4_OUT_F32;
    auto kernel = f32 ? rows_kernel<FMT, W4_OUT_F32, LOOKUP> : rows_kernel<FMT, W4_OUT_BF16, LOOKUP>;
    return f4::launch_dependent(kernel, grid_for(T, K), kThreads, st, codes, scales,
                                g, V, (int)K, ids, T, alpha, y, err);
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
    int rc = w4::check_device();
    if (rc != W4_OK) return rc;
    const cudaStream_t st = (cudaStream_t)stream;
    rc = f4::launch_dependent(clear_scale_kernel, dim3(1), 1, st, g);
    if (rc != W4_OK) return rc;
    constexpr int kMost = 8192;  // blocks of threads: one round of loads up to 67 M elements
    int64_t ctas = (chunks + kThreads * kScaleLoads - 1) / (kThreads * kScaleLoads);
    if (ctas > kMost) ctas = kMost;
    if (ctas < 1) ctas = 1;  // no elements: g = 2^-100
    int* err = w4::device_error_word();
    auto kernel = in_dtype == W4_IN_BF16  ? tensor_scale_kernel<W4_IN_BF16>
                  : in_dtype == W4_IN_F32 ? tensor_scale_kernel<W4_IN_F32>
                                          : tensor_scale_kernel<W4_IN_F16>;
    return f4::launch_dependent(kernel, dim3((unsigned)ctas), kThreads, st, x, chunks, g, err);
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
