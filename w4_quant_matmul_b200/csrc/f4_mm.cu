// f4_mm.cu -- products with matrices in microscaled 4-bit floating point on the
// block-scaled tensor cores (tcgen05.mma kind::mxf4 / kind::mxf4nvf4).
//
//   f4_mm    y[t][n] = gw ga sum_k (q s)_w[n][k] (q s)_a[t][k]
//   f4_gemv  y[t][n] = g sum_k (q s)[n][k] x[t][k],  x bf16, at most 8 tokens
//
// Both run one kernel (f4_mm of many tokens has its own: f4_pair.cu).  A tile is
// 128 weight rows (the MMA's M, TMEM lanes) by BN tokens (its N, TMEM columns);
// K advances in stages of 256 elements (128 bytes of codes a row, one
// 128B-swizzle atom), four MMAs of K = 64 each.
//   warp 0     TMA producer: the code tiles of weights and tokens and their
//              scale tiles into a ring of shared-memory stages.
//   warp 1     allocates TMEM; one lane copies each stage's scale tiles to TMEM
//              (tcgen05.cp: the scale planes are stored as the copy wants them)
//              and issues the MMAs.  tcgen05.cp and tcgen05.mma of one thread
//              run in issue order.
//   warps 2-5  epilogue: TMEM -> registers -> y; a thread owns one weight row,
//              so a warp's stores of one token are contiguous.
//   warps 6-   f4_gemv in one kernel: activation digits (below).
// When the tiles do not fill the GPU, a cluster of up to 6 CTAs splits a tile's
// K; each CTA leaves its fp32 partial tile in shared memory and the CTAs sum
// them through distributed shared memory in CTA order (deterministic, and no
// workspace).  Otherwise CTAs are persistent and their accumulators double
// buffered; f4_gemv, where they would take one or two tiles each, takes one and
// splits the others' K so.  What bounds it: bytes from HBM for large streams, and
// latency for small ones: one HBM access, the MMAs' completion, the sum over the
// cluster.  Above the time of its bytes a GEMV of one token takes 3 to 3.5 us (2560 x
// 4096 3.8, NV 4.25), a product of up to 64 tokens 3.5 to 6 (2560 x 4096 at 16 tokens
// 4.8, 6151 x 2592 at 33 7.2: more columns pass through the cluster's sum), one of 256
// tokens 8 (2560 x 9728 10.7: every weight tile is read from L2 once for each 64
// tokens, 79 MB), NV GEMVs with the digit kernel in front 6.5 (2560 x 9728 at eight
// tokens 8.6).  Tiles of 64 tokens at most: of 128 they were slower wherever the CTA
// pairs are not faster still (2560 x 9728 at 256 tokens 13.5 us against 12.6, both
// with an earlier split of K).
//
// f4_gemv keeps x exact to 22 bits of each block's largest magnitude without
// leaving the 4-bit tensor cores: x is written as fixed point in eight base-8
// digits -4..3, every one of them an e2m1 number, and digit j of token t becomes
// row 8 t + j of the token operand, with the block's power of two as its scale.
// The epilogue sums a token's 8 columns with weights 8^-j.  The weights are read
// once, whatever the number of tokens, and no CUDA core touches them: at 54
// weights a cycle and SM, unpacking them there would take most of the issue slots
// at one token and several times too many at eight.  lm_head 151936 x 2560 (MX):
// 31.0 us at one token, 34.4 at eight (6670 and 6010 GB/s of weights).  That every
// tile loads the digits of many tokens from L2 again costs nothing (34.8 without).
#include <cuda_bf16.h>

#include "f4_pair.cuh"
#include "f4_tc.cuh"

namespace {

using namespace f4;

constexpr int BM = 128;   // weight rows of a tile
constexpr int kEpiWarp0 = 2;
constexpr int kEpiWarps = 4;
constexpr int kDigitWarp0 = kEpiWarp0 + kEpiWarps;  // fused f4_gemv: more warps
constexpr int kDigits = 8;      // base-8 digits of an activation
constexpr int kMaxTokens = 8;   // f4_gemv

// Tokens up to which f4_gemv is one kernel whatever the sizes, and up to which it
// may be where K is split as far as it goes (see one_kernel).
constexpr int fused_tokens(int fmt) { return fmt == W4_F4_MX ? 5 : 4; }
constexpr int most_fused_tokens(int fmt) { return fmt == W4_F4_MX ? 8 : 6; }
constexpr int kMaxSplit = 6;    // CTAs of a cluster that share a tile's K
constexpr size_t kSmemTwo = 113 * 1024;  // of each of two CTAs on an SM (228 KB, 1 KB reserved a CTA)

// What a kernel computes.
enum Mode {
    kMm,          // f4_mm: the token operand is a 4-bit matrix
    kGemvPlanes,  // f4_gemv: it is digit rows that the preceding kernel wrote
    kGemvFused    // f4_gemv: the kernel makes the digits itself
};

template <int FMT, int BN>
struct Cfg {
    static constexpr int chunks = BK / (4 * f4::block_of(FMT));  // scale tiles of a stage
    static constexpr int mma_per_chunk = 4 / chunks;             // 2 (MX) or 1 (NV)
    static constexpr int a_bytes = BM * kRowBytes;
    static constexpr int b_bytes = BN * kRowBytes;
    static constexpr int sa_bytes = chunks * f4::kTileBytes;
    static constexpr int sb_bytes = chunks * f4::kTileBytes;
    static constexpr int stage_bytes = a_bytes + b_bytes + sa_bytes + sb_bytes;
    // two CTAs run on an SM, so that one streams while the other starts or
    // ends; each takes as many stages as its half holds
    static constexpr int stages = (int)((kSmemTwo - 512) / stage_bytes);
    static constexpr int acc_stages = 2;
    static constexpr int sf_cols = chunks * 4 * 2;  // TMEM columns per slot
    static constexpr int sf_slots = 2;
    static constexpr int used_cols = acc_stages * (BN < 32 ? 32 : BN) + sf_slots * sf_cols;
    static constexpr int tmem_cols = used_cols <= 128 ? 128 : 256;
    static constexpr int acc_cols = BN < 32 ? 32 : BN;
    static constexpr int nbars = 2 * stages + 2 * acc_stages + 1;
    static constexpr int bars = stages * stage_bytes;
    static constexpr int misc = bars + nbars * 8;      // TMEM base, abort flag
    static constexpr int amax = misc + 16;             // fused f4_gemv: largest magnitude of each token
    static constexpr size_t total = (size_t)amax + kMaxTokens * 4;
    static_assert(used_cols <= 256, "TMEM has 512 columns, for two CTAs");
    static_assert(stage_bytes % 1024 == 0, "operand tiles start on swizzle atoms");
    static_assert(total <= kSmemTwo, "shared memory of an SM, for two CTAs");
    static_assert((size_t)BN * BM * 4 <= (size_t)stages * stage_bytes, "a partial tile fits the ring");
};

struct Params {
    const uint8_t* sa;  // weight scales
    const uint8_t* sb;  // token scales
    const float* gw;    // NV: tensor scales (token: f4_mm only)
    const float* ga;
    const float* row_factor;  // f4_gemv with digit planes: factor of each token
    const uint16_t* x;        // fused f4_gemv: activations
    void* y;
    int M, N;          // tokens, weight rows
    int b_rows;        // rows of the token operand (f4_gemv: 8 M)
    int K;
    int stages_k;      // ceil(K / BK)
    int tiles_k;       // scale tiles along K
    int tiles_n, tiles_m;
    int whole;         // tiles that each CTA takes in whole, before
    int splits;        // the CTAs of a cluster share one along K
    int out_f32;
    int* err;
};

__device__ __forceinline__ void store_y(const Params& p, int64_t t, int n, float v) {
    const int64_t at = t * p.N + n;
    if (!W4_CHECK(t >= 0 && t < p.M && n >= 0 && n < p.N, p.err)) return;
    if (p.out_f32)
        static_cast<float*>(p.y)[at] = v;
    else
        static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
}

// Four consecutive weight rows of token t.
__device__ __forceinline__ void store_y4(const Params& p, int64_t t, int n, const float4& v,
                                         const f4::Factors& scale) {
    const float f[4] = {f4::times(v.x, scale), f4::times(v.y, scale), f4::times(v.z, scale),
                        f4::times(v.w, scale)};
    if (p.N % 4 == 0 && n < p.N) {  // y's rows start on 4 elements: one vector
        if (!W4_CHECK(t >= 0 && t < p.M && n >= 0 && n + 4 <= p.N, p.err)) return;
        const int64_t at = t * p.N + n;
        if (p.out_f32) {
            *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) =
                make_float4(f[0], f[1], f[2], f[3]);
        } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0], f[1]);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(f[2], f[3]);
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.y) + at) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                           *reinterpret_cast<const uint32_t*>(&hi));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < p.N) store_y(p, t, n + i, f[i]);
    }
}

// ---------------------------------------------------------------------------
// activation digits of f4_gemv
// ---------------------------------------------------------------------------
//
// With E = floor(log2 amax) of a block, v = x * 2^(21 - E) rounded to an integer
// has |v| < 2^22, and
//   v = sum_j d_j 8^(7-j),  d_j in -4..3,  from the base-8 digits of
//   v + 4 (8^8 - 1) / 7 (each digit shifted by 4),
// so x = 2^E sum_j d_j 8^-j: digit rows 8 t + j of token t with block scale 2^E.
// NV: e4m3 scales span 2^-9..2^8, so E is taken relative to the largest exponent
// Emax among the k that one accumulation sees, and the rest, 2^(Emax - 8), is a
// factor in the epilogue.

// bf16 magnitude: exponent field, at least 1 (subnormals share the exponent of
// the smallest normal number).
__device__ __forceinline__ int exp_field(uint32_t h) {
    const int e = (int)((h >> 7) & 0xFFu);
    return e > 0 ? e : 1;
}

// Largest magnitude (15 bits) of 8 bf16 numbers.
__device__ __forceinline__ uint32_t amax8(const uint4& v) {
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    return max(m >> 16, m & 0xFFFFu);
}

// The factor 2^(emax - 127 - 8) of an exponent field, as a product where the
// power itself is subnormal.
__device__ __forceinline__ float nv_factor(int emax) {
    return __uint_as_float((uint32_t)emax << 23) * 0x1p-8f;
}

// The 8 digits of each of a lane's 8 elements: out[j] holds digit j's e2m1
// codes, element i in bits 4i..4i+3; `word` the scale bytes of the 4 blocks that
// this lane's block shares a scale word with.  All 32 lanes take part; `live` is
// false past the end of K (zero digits, zero scale).  emax: NV only.
template <int FMT>
__device__ __forceinline__ void digits8(const uint4& raw, bool live, int emax, int lane,
                                        uint32_t (&out)[kDigits], uint32_t& word) {
    constexpr int kBlkLanes = block_of(FMT) / 8;
    constexpr int kWordLanes = 4 * kBlkLanes;
    uint32_t amax = amax8(raw);
#pragma unroll
    for (int off = 1; off < kBlkLanes; off <<= 1)
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    const bool bad = amax >= 0x7F80u;  // a NaN or an infinity: the scale becomes NaN
    int eb = exp_field(amax);
    uint32_t byte;
    if constexpr (FMT == W4_F4_MX) {
        byte = bad ? 255u : (uint32_t)eb;
    } else {
        if (eb < emax - 17) eb = emax - 17;  // the smallest scale, 2^-9
        const int s = eb - emax + 8;         // -9..8
        byte = bad ? 127u : (uint32_t)(s >= -6 ? (s + 7) << 3 : 1 << (s + 9));
    }
    word = live ? byte << (8 * (lane / kBlkLanes % 4)) : 0u;
#pragma unroll
    for (int off = kBlkLanes; off < kWordLanes; off <<= 1)
        word |= __shfl_xor_sync(0xffffffffu, word, off);

    // v = x * 2^(21 - E) rounded to an integer (ties to even): added to 3 * 2^22 it
    // is the low bits of the sum.  In two factors, as the power itself leaves the
    // range of fp32 for the smallest E; the first is exact.  (A bad block's digits
    // may be any: its scale is NaN.)
    const float up = eb < 64 ? 0x1p64f : 1.0f;
    const float to_int = __uint_as_float((uint32_t)(eb < 64 ? 275 - 64 - eb : 275 - eb) << 23);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t lo[4], hi[4];  // codes of digits 7..4 and 3..0, a byte each, by pair of elements
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        uint32_t u = __float_as_uint(fmaf(x * up, to_int, 12582912.0f));
        u += 9586980u - 0x4B400000u;  // v + 4 (8^8 - 1) / 7
        // octal digits to nibbles (a field moves up n bits by 2^n - 1 times itself),
        // then each to its e2m1 code by table
        u += (u & 0x00FFF000u) * 15u;
        u += (u & 0x0FC00FC0u) * 3u;
        u += u & 0x38383838u;
        // -4 -3 -2 -1 | 0 1 2 3
        const uint32_t a = __byte_perm(0x0A0C0D0Eu, 0x05040200u, u);
        const uint32_t b = __byte_perm(0x0A0C0D0Eu, 0x05040200u, u >> 16);
        lo[i / 2] = i & 1 ? lo[i / 2] + (a << 4) : a;
        hi[i / 2] = i & 1 ? hi[i / 2] + (b << 4) : b;
    }
    // byte i of the four pairs -> one word
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint32_t(&p)[4] = q ? hi : lo;
        const uint32_t t0 = __byte_perm(p[0], p[1], 0x5140), t1 = __byte_perm(p[2], p[3], 0x5140);
        const uint32_t t2 = __byte_perm(p[0], p[1], 0x7362), t3 = __byte_perm(p[2], p[3], 0x7362);
        out[7 - 4 * q] = __byte_perm(t0, t1, 0x5410);
        out[6 - 4 * q] = __byte_perm(t0, t1, 0x7632);
        out[5 - 4 * q] = __byte_perm(t2, t3, 0x5410);
        out[4 - 4 * q] = __byte_perm(t2, t3, 0x7632);
    }
}

// ---------------------------------------------------------------------------
// kernel
// ---------------------------------------------------------------------------

// Digit warps of the fused f4_gemv: two a token, as far as the registers of two
// CTAs on an SM allow.
constexpr int digit_warps(int bn) { return bn <= 48 ? bn / kDigits * 2 : 12; }

// Whether CTAs of a grid without K slices work on several tiles each.
__host__ __device__ constexpr bool many_tiles(int64_t tiles, int64_t ctas) { return tiles > ctas; }

constexpr int threads_of(int bn, Mode mode) {
    return 32 * (kDigitWarp0 + (mode == kGemvFused ? digit_warps(bn) : 0));
}

// Digit and epilogue warps meet: the maxima of the tokens are in shared memory.
template <int BN>
__device__ __forceinline__ void digit_barrier() {
    asm volatile("bar.sync 1, %0;" ::"n"(32 * (kEpiWarps + digit_warps(BN))) : "memory");
}

// Two CTAs run on an SM in any case; asking for them lets the compiler take more
// registers, and the loads of the sum over a cluster overlap (2560 x 4096 at 4
// tokens, MX and NV: 5.87 -> 5.63, 6.85 -> 6.53 us).
template <int FMT, int BN, Mode MODE>
__global__ void __launch_bounds__(threads_of(BN, MODE), 2)
    f4_mm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                 const Params p) {
    using C = Cfg<FMT, BN>;
    constexpr bool GEMV = MODE != kMm;
    constexpr bool FUSED = MODE == kGemvFused;
    // Operand tiles start on 1024 bytes.  Dynamic shared memory does too (there
    // is no static one here); slack to round its start up would cost the widest
    // NV tile its fourth stage, so a start elsewhere is refused instead.
    extern __shared__ __align__(1024) uint8_t smem[];
    if (w4::smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0) atomicCAS(p.err, 0, (int)W4_ERR_ALIGN);
        return;
    }
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::bars);  // stage loaded     [stages]
    uint64_t* empty = full + C::stages;                            // stage consumed   [stages]
    uint64_t* afull = empty + C::stages;                           // tile accumulated [acc_stages]
    uint64_t* aempty = afull + C::acc_stages;                      // tile read out    [acc_stages]
    uint64_t* drain = aempty + C::acc_stages;                      // last MMA complete
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::misc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::misc + 4);
    [[maybe_unused]] uint32_t* amax = reinterpret_cast<uint32_t*>(smem + C::amax);  // [tokens]

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int tiles = p.tiles_n * p.tiles_m;
    const int split = p.splits > 1 ? (int)cluster_rank() : 0;
    // unit u of this CTA: a whole tile, at the end its K slice of the cluster's
    const int shared = p.whole * gridDim.x + blockIdx.x / p.splits;
    const int units = p.whole + (shared < tiles ? 1 : 0);
    const int kb = (int)((int64_t)p.stages_k * split / p.splits);
    const int ke = (int)((int64_t)p.stages_k * (split + 1) / p.splits);
    auto tile_of = [&](int u) {
        return u < p.whole ? u * (int)gridDim.x + (int)blockIdx.x : shared;
    };
    auto k_from = [&](int u) { return u < p.whole ? 0 : kb; };
    auto k_to = [&](int u) { return u < p.whole ? p.stages_k : ke; };

    const int chunks_last = p.tiles_k - (p.stages_k - 1) * C::chunks;
    auto chunks_of = [&](int ks) { return ks + 1 < p.stages_k ? C::chunks : chunks_last; };
    auto load_a = [&](int s, int ks, int tn) {
        const int ch = chunks_of(ks);
        w4::mbar_arrive_expect_tx(&full[s], C::a_bytes + ch * f4::kTileBytes +
                                                (FUSED ? 0 : C::b_bytes + ch * f4::kTileBytes));
        uint8_t* st = smem + s * C::stage_bytes;
        w4::tma_load_2d(st, &tm_a, &full[s], ks * kRowBytes, tn * BM);
        w4::bulk_load_1d(st + C::a_bytes + C::b_bytes,
                         p.sa + ((int64_t)tn * p.tiles_k + (int64_t)ks * C::chunks) *
                                    f4::kTileBytes,
                         (uint32_t)(ch * f4::kTileBytes), &full[s]);
    };
    auto load_b = [&](int s, int ks, int tm) {
        const int ch = chunks_of(ks);
        uint8_t* st = smem + s * C::stage_bytes;
        w4::tma_load_2d(st + C::a_bytes, &tm_b, &full[s], ks * kRowBytes, tm * BN);
        w4::bulk_load_1d(st + C::a_bytes + C::b_bytes + C::sa_bytes,
                         p.sb + ((int64_t)(tm * BN / f4::kRowTile) * p.tiles_k +
                                 (int64_t)ks * C::chunks) *
                                    f4::kTileBytes,
                         (uint32_t)(ch * f4::kTileBytes), &full[s]);
    };

    // f4_gemv: the first tile's first weights are requested ahead of the set-up
    // that all warps share and of the wait for the kernel before (w4.h says which
    // kernels may not be it).  With the digits made here only where a CTA has
    // several tiles to stream: lm_head 33.0 -> 31.5 us in a row of them, but
    // 19456 x 2560 6.6 -> 7.8, where the requests delay what the kernel before
    // still has to load.
    int pre = 0;
    if constexpr (GEMV)
        if (units > 0 && (!FUSED || many_tiles(tiles, gridDim.x))) {
            pre = k_to(0) - k_from(0);
            if (pre > C::stages) pre = C::stages;
        }

    if (threadIdx.x == 0) {
        w4::prefetch_tmap(&tm_a);
        if constexpr (!FUSED) w4::prefetch_tmap(&tm_b);
        for (int i = 0; i < C::stages; ++i) {
            // the producer, and a warp's arrival for each token
            w4::mbar_init(&full[i], FUSED ? 1 + p.M : 1);
            w4::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::acc_stages; ++i) {
            w4::mbar_init(&afull[i], 1);
            w4::mbar_init(&aempty[i], kEpiWarps);
        }
        w4::mbar_init(drain, 1);
        *abort_flag = 0;
        if constexpr (FUSED && FMT == W4_F4_NV)
            for (int t = 0; t < p.M; ++t) amax[t] = 0u;
        w4::fence_mbar_init();
        for (int i = 0; i < pre; ++i) load_a(i, k_from(0) + i, tile_of(0));
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         w4::smem_u32((const void*)tmem_slot)),
                     "r"(C::tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // The producer warp, which set the barriers up and needs nothing else, does
    // not wait for the TMEM allocation (2560 x 4096 at one token, cold: 0.5 us).
    uint32_t tmem = 0;
    if (warp == 0) {
        __syncwarp();
        asm volatile("bar.arrive 2, %0;" ::"n"(threads_of(BN, MODE)) : "memory");
    } else {
        tc_fence_before();
        asm volatile("bar.sync 2, %0;" ::"n"(threads_of(BN, MODE)) : "memory");
        tc_fence_after();
        tmem = *tmem_slot;
    }

    Factors scale{1.0f, 1.0f};  // f4_mm, epilogue: both tensor scales (f4_gemv's are in the tiles)
    if (warp == 0) {
        // ---------------- TMA producer ----------------
        if (w4::elect_one()) {
            int it = 0;  // stages issued
            bool ok = true;
            pdl_wait();
            pdl_trigger();
            for (int u = 0; u < units && ok; ++u) {
                const int tile = tile_of(u), k0 = k_from(u), k1 = k_to(u);
                const int tn = GEMV ? tile : tile / p.tiles_m;
                const int tm = GEMV ? 0 : tile % p.tiles_m;
                (void)W4_CHECK(tn < p.tiles_n && tm < p.tiles_m && k0 < k1, p.err);
                for (int ks = k0; ks < k1; ++ks, ++it) {
                    const int s = it % C::stages;
                    if (it >= pre) {
                        if (!w4::mbar_wait(&empty[s], ((uint32_t)(it / C::stages) & 1u) ^ 1u,
                                           abort_flag, p.err)) {
                            ok = false;
                            break;
                        }
                        load_a(s, ks, tn);
                    }
                    if constexpr (!FUSED) load_b(s, ks, tm);
                }
            }
            // drain: every issued load must land before the CTA exits
            for (int k = it - C::stages < 0 ? 0 : it - C::stages; k < it; ++k)
                w4::mbar_wait(&full[k % C::stages], (uint32_t)(k / C::stages) & 1u, nullptr, p.err);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        if (w4::elect_one()) {
            const uint32_t sf0 = tmem + C::acc_stages * C::acc_cols;
            int it = 0;
            bool ok = true;
            for (int ti = 0; ti < units && ok; ++ti) {
                const int k0 = k_from(ti), k1 = k_to(ti);
                // an odd 64-token tile starts in the middle of its 128-row scale
                // tile, at TMEM column 2 (32 rows a column; scale addresses must
                // be even, so narrower tiles come one to a product)
                const uint32_t sb_col = !GEMV && BN == 64 ? (uint32_t)(tile_of(ti) % p.tiles_m & 1) * 2 : 0u;
                const int as = ti % C::acc_stages;
                const uint32_t d = tmem + as * C::acc_cols;
                if (!w4::mbar_wait(&aempty[as], ((uint32_t)(ti / C::acc_stages) & 1u) ^ 1u,
                                   abort_flag, p.err))
                    break;
                tc_fence_after();
                for (int ks = k0; ks < k1; ++ks, ++it) {
                    const int s = it % C::stages;
                    if (!w4::mbar_wait(&full[s], (uint32_t)(it / C::stages) & 1u, abort_flag,
                                       p.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = w4::smem_u32(smem + s * C::stage_bytes);
                    const uint32_t b = a + C::a_bytes;
                    const uint32_t sa = b + C::b_bytes;
                    const uint32_t sb = sa + C::sa_bytes;
                    const uint32_t sf = sf0 + (it % C::sf_slots) * C::sf_cols;
                    const uint32_t sfb = sf + C::chunks * 4;
                    // K = 64 steps of this stage that hold elements
                    int steps = (p.K - ks * BK + kMmaK - 1) / kMmaK;
                    if (steps > BK / kMmaK) steps = BK / kMmaK;
                    // (a chunk's scales directly before its MMAs: see f4_pair.cu)
#pragma unroll
                    for (int j = 0; j < BK / kMmaK; ++j) {
                        if (j >= steps) break;
                        const int c = j / C::mma_per_chunk;
                        const int id = j % C::mma_per_chunk * 2;
                        if (id == 0) {
                            copy_scales(sf + c * 4, scale_desc(sa + c * f4::kTileBytes));
                            copy_scales(sfb + c * 4, scale_desc(sb + c * f4::kTileBytes));
                        }
                        mma_f4<FMT>(d, operand_desc(a + j * (kMmaK / 2)),
                                    operand_desc(b + j * (kMmaK / 2)), instr_desc<FMT, BM, BN>(id),
                                    sf + c * 4, sfb + c * 4 + sb_col,
                                    ks > k0 || j > 0);
                    }
                    mma_commit(&empty[s]);
                }
                if (ok) mma_commit(&afull[as]);
            }
            // drain: nothing may still write TMEM or read shared memory
            mma_commit(drain);
            w4::mbar_wait(drain, 0u, nullptr, p.err);
        }
    } else if (FUSED && warp >= kDigitWarp0) {
        // ---------------- activation digits ----------------
        // The warps take the tokens of the stages in turn: 8 rows of 128 bytes of
        // a stage's token operand (one swizzle atom) and their scale words.
        constexpr int kDigitWarps = digit_warps(BN);
        constexpr int kWordLanes = block_of(FMT) / 2;
        const int w = warp - kDigitWarp0;
        pdl_wait();
        if constexpr (FMT == W4_F4_NV) {
            // the largest magnitude of each token over this CTA's k (its first
            // tile's hold the others')
            constexpr int kTokens = BN / kDigits;
            const int k_end = k_to(0) * BK < p.K ? k_to(0) * BK : p.K;
            uint32_t m[kTokens] = {};
#pragma unroll 2
            for (int k = k_from(0) * BK + (w * 32 + lane) * 8; k < k_end; k += kDigitWarps * 32 * 8)
#pragma unroll
                for (int t = 0; t < kTokens; ++t)
                    if (t < p.M)
                        m[t] = max(m[t], amax8(__ldca(reinterpret_cast<const uint4*>(
                                             p.x + (int64_t)t * p.K + k))));
#pragma unroll
            for (int t = 0; t < kTokens; ++t) {
                m[t] = __reduce_max_sync(0xffffffffu, m[t]);
                if (t < p.M && lane == 0) atomicMax(&amax[t], m[t]);
            }
            digit_barrier<BN>();
        }
        // a warp's next activations are loaded before it works on the present
        // ones; the stages of one tile follow those of the tile before
        const int total = p.whole * p.stages_k + (shared < tiles ? ke - kb : 0);
        // a tile's last stage is followed by the next one's first: kb, which is
        // 0 unless a shared tile follows the only whole one
        auto wrap = [&](int ks) {
            while (ks >= p.stages_k) ks += kb - p.stages_k;
            return ks;
        };
        auto load_x = [&](int i, int ks, int t) {
            const int k = ks * BK + lane * 8;
            if (i < total && k < p.K && W4_CHECK(k + 8 <= p.K && t < p.M, p.err))
                return __ldca(reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.K + k));
            return make_uint4(0u, 0u, 0u, 0u);
        };
        const int stages_on = kDigitWarps / p.M, tokens_on = kDigitWarps % p.M;
        int it_next = w / p.M, t_next = w % p.M;
        int ks_next = wrap(k_from(0) + it_next);
        uint4 next = load_x(it_next, ks_next, t_next);
        while (it_next < total) {
            const uint4 raw = next;
            const int it = it_next, t = t_next;
            const bool live = ks_next * BK + lane * 8 < p.K;
            const int on = stages_on + (t + tokens_on >= p.M ? 1 : 0);
            t_next += tokens_on - (t + tokens_on >= p.M ? p.M : 0);
            it_next += on;
            ks_next = wrap(ks_next + on);
            next = load_x(it_next, ks_next, t_next);
            uint32_t out[kDigits], word;
            const int emax = FMT == W4_F4_NV ? exp_field(*(volatile uint32_t*)&amax[t]) : 0;
            digits8<FMT>(raw, live, emax, lane, out, word);
            const int s = it % C::stages;
            if (!w4::mbar_wait(&empty[s], ((uint32_t)(it / C::stages) & 1u) ^ 1u, abort_flag, p.err))
                break;
            uint8_t* rows = smem + s * C::stage_bytes + C::a_bytes + t * kDigits * kRowBytes;
#pragma unroll
            for (int j = 0; j < kDigits; ++j)
                *reinterpret_cast<uint32_t*>(rows + j * kRowBytes + (((lane >> 2) ^ j) << 4) +
                                             (lane & 3) * 4) = out[j];
            // scale rows 8 t .. 8 t + 7 of the word's tile: rows r and r + 32
            // share a 16-byte line
            uint8_t* sc = smem + s * C::stage_bytes + C::a_bytes + C::b_bytes + C::sa_bytes +
                          lane / kWordLanes * kTileBytes + t % 4 * kDigits * 16 + t / 4 * 4;
            if (lane % kWordLanes < kDigits)
                *reinterpret_cast<uint32_t*>(sc + lane % kWordLanes * 16) = word;
            w4::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) w4::mbar_arrive(&full[s]);
        }
    } else {
        // ---------------- epilogue ----------------
        const int quarter = warp & 3;  // the TMEM lanes this warp may read
        const int row = quarter * 32 + lane;
        float alpha = 1.0f;  // the weights' tensor scale
        float* part = reinterpret_cast<float*>(smem);  // split K: [column][128] in the ring
        pdl_wait();
        if constexpr (FMT == W4_F4_NV) {
            alpha = __ldca(p.gw);
            if constexpr (!GEMV) scale = factors(alpha, __ldca(p.ga));
        }
        if constexpr (FUSED && FMT == W4_F4_NV) digit_barrier<BN>();
        // f4_gemv, NV: what the digits of token `lane` leave out of its sums
        Factors own{1.0f, 1.0f};
        if constexpr (GEMV && FMT == W4_F4_NV) {
            if (lane < p.M)
                own = factors(FUSED ? nv_factor(exp_field(*(volatile uint32_t*)&amax[lane]))
                                    : __ldca(p.row_factor + lane),
                              alpha);
        }
        for (int ti = 0; ti < units; ++ti) {
            const int tile = tile_of(ti);
            const bool partial = p.splits > 1 && (!GEMV || ti == p.whole);
            const int tn = GEMV ? tile : tile / p.tiles_m;
            const int tm = GEMV ? 0 : tile % p.tiles_m;
            const int as = ti % C::acc_stages;
            const int n = tn * BM + row;
            if (!w4::mbar_wait(&afull[as], (uint32_t)(ti / C::acc_stages) & 1u, abort_flag, p.err))
                break;
            tc_fence_after();
            const uint32_t acc = tmem + as * C::acc_cols + ((uint32_t)(quarter * 32) << 16);
            if constexpr (GEMV) {
                // two tokens per 16 columns: y = sum_j 8^-j D[8 t + j]
#pragma unroll 1
                for (int c = 0; c < BN; c += 16) {
                    uint32_t r[16];
                    tmem_ld16(acc + c, r);
                    tmem_wait16(r);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int t = c / 8 + h;
                        float v = __uint_as_float(r[8 * h + 7]);
#pragma unroll
                        for (int j = 6; j >= 0; --j)
                            v = fmaf(v, 0.125f, __uint_as_float(r[8 * h + j]));
                        if (t < p.M) {
                            if constexpr (FMT == W4_F4_NV)
                                v = times(v, Factors{__shfl_sync(0xffffffffu, own.first, t),
                                                     __shfl_sync(0xffffffffu, own.second, t)});
                            if (partial)
                                part[t * BM + row] = v;
                            else if (n < p.N)
                                store_y(p, t, n, v);
                        }
                    }
                }
            } else {
#pragma unroll 2
                for (int c = 0; c < BN; c += 16) {
                    const int t0 = tm * BN + c;
                    if (t0 >= p.M) break;
                    uint32_t r[16];
                    tmem_ld16(acc + c, r);
                    tmem_wait16(r);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float v = __uint_as_float(r[i]);
                        if (partial)
                            part[(c + i) * BM + row] = v;
                        else if (t0 + i < p.M && n < p.N)
                            store_y(p, t0 + i, n, times(v, scale));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) w4::mbar_arrive(&aempty[as]);
        }
    }

    if (p.splits > 1) {
        // the cluster's tile: the partial tiles, summed in CTA order; the
        // columns are dealt out to the CTAs
        cluster_sync();
        if (warp >= kEpiWarp0 && warp < kDigitWarp0 && shared < tiles && !*abort_flag) {
            const int tn = GEMV ? shared : shared / p.tiles_m;
            const int t0 = GEMV ? 0 : shared % p.tiles_m * BN;
            const int row = lane * 4, n = tn * BM + row;  // four weight rows a thread
            const int cols = p.M - t0 < BN ? p.M - t0 : BN;
            const uint32_t base = w4::smem_u32(smem) + row * 4;
            // columns split, split + splits, ...: one a warp and step; f4_mm has two
            // steps' loads in flight (four were no faster)
            constexpr int kSteps = GEMV ? 1 : 2;
            const int cstep = p.splits * kEpiWarps;
#pragma unroll 1
            for (int c = split + p.splits * (warp - kEpiWarp0); c < cols; c += kSteps * cstep) {
                float4 v[kSteps][kMaxSplit];
#pragma unroll
                for (int u = 0; u < kSteps; ++u) {
                    const int cu = c + u * cstep;
#pragma unroll
                    for (int q = 0; q < kMaxSplit; ++q)
                        v[u][q] = q < p.splits && cu < cols ? ld_cluster(base + cu * BM * 4, q)
                                                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
#pragma unroll
                for (int u = 0; u < kSteps; ++u) {
                    const int cu = c + u * cstep;
                    if (cu >= cols) break;
                    float4 sum = v[u][0];
#pragma unroll
                    for (int q = 1; q < kMaxSplit; ++q) {
                        sum.x += v[u][q].x;
                        sum.y += v[u][q].y;
                        sum.z += v[u][q].z;
                        sum.w += v[u][q].w;
                    }
                    store_y4(p, t0 + cu, n, sum, scale);
                }
            }
        }
        cluster_sync();  // no CTA leaves while another reads its shared memory
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(C::tmem_cols)
                     : "memory");
    }
}

// ---------------------------------------------------------------------------
// f4_gemv in two kernels (see one_kernel): the digits in global memory
// ---------------------------------------------------------------------------

constexpr int kDigitThreads = 256;
constexpr int kDigitElems = kDigitThreads * 8;  // k of one block of threads

// Token t = blockIdx.y, 8 consecutive k a thread.
template <int FMT>
__global__ void __launch_bounds__(kDigitThreads)
    digits_kernel(const uint16_t* __restrict__ x, int K, uint8_t* __restrict__ codes,
                  uint8_t* __restrict__ scales, float* __restrict__ row_factor, bool early,
                  int* err) {
    // the product may start and read its weights; it waits for this kernel, and
    // so for all before it, ahead of anything else.  Where it streams several
    // tiles a CTA it starts before this kernel's own wait.
    if (early) pdl_trigger();
    pdl_wait();
    if (!early) pdl_trigger();
    constexpr int kWordLanes = block_of(FMT) / 2;
    const int t = blockIdx.y;
    const int lane = threadIdx.x & 31;
    const uint16_t* xt = x + (int64_t)t * K;

    const int64_t tiles_k = scale_tiles_k(K, FMT);
    const int kpad = (int)tiles_k * 4 * block_of(FMT);
    const int k = blockIdx.x * kDigitElems + threadIdx.x * 8;
    const bool live = k < K;
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (live && W4_CHECK(k + 8 <= K, err)) raw = __ldca(reinterpret_cast<const uint4*>(xt + k));

    int emax = 0;  // NV: largest exponent field of the token
    if constexpr (FMT == W4_F4_NV) {
        __shared__ uint32_t part[kDigitThreads / 32];
        uint32_t m = 0;
#pragma unroll 4
        for (int i = 1; i < (int)gridDim.x; ++i) {  // the other blocks' elements
            const int other = blockIdx.x + i < gridDim.x ? blockIdx.x + i : blockIdx.x + i - gridDim.x;
            const int ko = other * kDigitElems + threadIdx.x * 8;
            if (ko < K) m = max(m, amax8(__ldca(reinterpret_cast<const uint4*>(xt + ko))));
        }
        m = __reduce_max_sync(0xffffffffu, max(m, amax8(raw)));
        if (lane == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kDigitThreads / 32; ++i) m = max(m, part[i]);
        emax = exp_field(m);
        if (blockIdx.x == 0 && threadIdx.x == 0) row_factor[t] = nv_factor(emax);
    }

    // whole warps run or skip; in a warp that runs, the lanes past kpad only
    // take part in the shuffles
    if (k - lane * 8 >= kpad) return;
    uint32_t out[kDigits], word;
    digits8<FMT>(raw, live, emax, lane, out, word);
    if (live && W4_CHECK(t < kMaxTokens && k + 8 <= K, err)) {
#pragma unroll
        for (int j = 0; j < kDigits; ++j)
            *reinterpret_cast<uint32_t*>(codes + ((int64_t)(t * kDigits + j) * K + k) / 2) = out[j];
    }
    if (lane % kWordLanes == 0 && k < kpad &&
        W4_CHECK(t * kDigits + kDigits <= kRowTile && k / (4 * block_of(FMT)) < tiles_k, err)) {
#pragma unroll
        for (int j = 0; j < kDigits; ++j)
            *reinterpret_cast<uint32_t*>(
                scales + scale_word(t * kDigits + j, k / (4 * block_of(FMT)), tiles_k)) = word;
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

template <int FMT, int BN, Mode MODE>
int launch_tiles(const uint8_t* codes, const uint8_t* bcodes, Params p, cudaStream_t stream) {
    using C = Cfg<FMT, BN>;
    p.tiles_n = (p.N + BM - 1) / BM;
    p.tiles_m = (p.b_rows + BN - 1) / BN;
    const int64_t tiles = (int64_t)p.tiles_n * p.tiles_m;
    CUtensorMap ma, mb;
    if (!make_map(&ma, codes, p.K, p.N, BM)) return W4_ERR_CUDA;
    if (MODE == kGemvFused)
        mb = ma;  // not read
    else if (!make_map(&mb, bcodes, p.K, p.b_rows, BN))
        return W4_ERR_CUDA;
    auto kernel = f4_mm_kernel<FMT, BN, MODE>;
    // of the device: whether the shared-memory limit is raised, and how many
    // clusters of each size run at once (0: not asked yet)
    static thread_local int dev_of = -1;
    static thread_local int clusters[kMaxSplit + 1];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return w4::cuda_fail(e);
    if (dev_of != dev) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::total);
        // all of the SM's memory as shared memory: two CTAs
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return w4::cuda_fail(e);
        for (int& c : clusters) c = 0;
        dev_of = dev;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(threads_of(BN, MODE));
    cfg.dynamicSmemBytes = C::total;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    // CTAs of clusters of s that run at once
    auto cluster_slots = [&](int s, int64_t* ctas) {
        if (clusters[s] == 0) {
            attr[0].val.clusterDim.x = (unsigned)s;
            cfg.gridDim = dim3((unsigned)s);
            cfg.numAttrs = 1;
            const cudaError_t err = cudaOccupancyMaxActiveClusters(&clusters[s], kernel, &cfg);
            if (err != cudaSuccess) return err;
            if (clusters[s] == 0) clusters[s] = -1;  // asked, none
        }
        // the query counts one CTA an SM where two run: 48 tiles still start at
        // once in clusters of 5 (26 by the query) and no longer in 6 (22), 80 in
        // 3 (45) and not in 4 (33), each step too far costing half as much again
        *ctas = clusters[s] > 0 ? (int64_t)clusters[s] * 2 * s : 0;
        return cudaSuccess;
    };
    const int64_t slots = (int64_t)w4::sm_count() * 2;
    int64_t grid = tiles < slots ? tiles : slots;
    p.splits = 1;
    p.whole = (int)(tiles / grid);
    if (!many_tiles(tiles, slots)) {
        // CTAs along K of each tile: as many as still run all at once, with at
        // least two stages each
        for (int s = kMaxSplit; s > 1; --s) {
            int64_t ctas;
            if (p.stages_k / s < 2 || tiles * s > slots) continue;
            if ((e = cluster_slots(s, &ctas)) != cudaSuccess) return w4::cuda_fail(e);
            if (tiles * s <= ctas) {
                p.splits = s;
                p.whole = 0;
                grid = tiles * s;
                break;
            }
        }
    } else if (MODE != kMm && tiles < 2 * slots) {
        // f4_gemv: one whole tile each, and clusters for what is left over, of
        // the size that ends soonest (us at one and eight tokens: 40000 x 8192
        // MX 33.8 -> 29.0 and 37.4 -> 32.1, NV 38.2 -> 31.3 and 44.6 -> 35.4;
        // 50304 x 4096 MX 20.9 -> 19.7).  In longer streams the CTAs drift apart
        // and fill the end by themselves, and clusters leave slots empty: 128256
        // x 2560 was 26.7 -> 28.4.  f4_mm gained nothing (50304 x 4096 at 16
        // tokens 21.2, 21.1), and its narrow streams lost by the longer code.
        int64_t best = 2 * 60;  // two tiles' time, in 60ths of a tile's
        for (int s = 2; s <= kMaxSplit; ++s) {
            int64_t ctas;
            if (p.stages_k / s < 2) break;
            if ((e = cluster_slots(s, &ctas)) != cudaSuccess) return w4::cuda_fail(e);
            if (ctas == 0) continue;
            const int64_t rest = tiles % ctas, t = 60 * (tiles / ctas) + (rest > 0 ? 60 / s : 0);
            if (rest * s <= ctas && t < best) {
                best = t;
                p.splits = s;
                p.whole = (int)(tiles / ctas);
                grid = ctas;
            }
        }
    }
    attr[0].val.clusterDim.x = (unsigned)p.splits;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kernel, ma, mb, p);
    if (e != cudaSuccess) return w4::cuda_fail(e);
    return w4::launch_status();
}

template <int FMT>
int launch_mm(const uint8_t* codes, const uint8_t* qa, const Params& p, cudaStream_t st) {
    // tiles narrower than a 128-row scale tile hold all tokens, so that every
    // tile starts on one
    if (p.M <= 16) return launch_tiles<FMT, 16, kMm>(codes, qa, p, st);
    if (p.M <= 32) return launch_tiles<FMT, 32, kMm>(codes, qa, p, st);
    if (p.M <= 48) return launch_tiles<FMT, 48, kMm>(codes, qa, p, st);
    return launch_tiles<FMT, 64, kMm>(codes, qa, p, st);
}

// Whether the product makes its digits itself, every CTA those of its own k and so
// all of them once for each 128 weight rows, instead of reading what a kernel of
// their own made once.  us, in one and in two kernels:
//   tokens               MX 4       MX 5       MX 6       NV 3       NV 4       NV 5
//   2560 x 9728       6.1  7.3   6.4  7.4   6.5  7.4   6.5  8.0   6.8  8.0   7.4  8.15
//   19456 x 2560      7.9  8.6   8.9  8.8   9.7  8.8   8.4  9.1   9.25 9.2  10.6  9.4
//   128256 x 4096    45.8 45.8  47.6 47.1  49.7 47.1  48.6 49.0  49.2 48.8  52.1 49.0
//   151936 x 2560    32.5 32.8  33.4 34.8  35.0 34.8  35.9 35.3  35.9 35.6  36.0 36.0
// Up to fused_tokens it is one.  From there on the digits take the longer time, but
// for the tiles that clusters of kMaxSplit share: few stages a CTA, and two launches
// that count (MX at 8 tokens 1024 x 2560 4.3, 4.95; 2560 x 4096 5.15, 5.9; NV at 6
// 2560 x 9728 7.6, 8.3).  At about 50 token stages a CTA both are equal (MX at 8
// tokens 2560 x 9728, 56 of them, 7.65, 7.6); NV, which looks for the largest
// magnitudes first, loses there (4096 x 14336 at 5 tokens, 50: 11.6, 10.9).
bool one_kernel(int64_t M, int64_t N, int64_t K, int fmt) {
    if (M <= fused_tokens(fmt)) return true;
    (void)w4::check_device();  // sm_count knows the device from here on
    const int64_t stages = ((K + BK - 1) / BK + kMaxSplit - 1) / kMaxSplit;
    const int64_t most = fmt == W4_F4_MX ? 50 : 45;  // token stages a CTA
    return M <= most_fused_tokens(fmt) && stages * M <= most &&
           row_tiles(N) * kMaxSplit <= (int64_t)w4::sm_count() * 2;
}

template <int FMT>
int launch_fused(const uint8_t* codes, const Params& p, cudaStream_t st) {
    if (p.M <= 2) return launch_tiles<FMT, 16, kGemvFused>(codes, nullptr, p, st);
    if (p.M <= 4) return launch_tiles<FMT, 32, kGemvFused>(codes, nullptr, p, st);
    if constexpr (most_fused_tokens(FMT) > 6)
        if (p.M > 6) return launch_tiles<FMT, 64, kGemvFused>(codes, nullptr, p, st);
    return launch_tiles<FMT, 48, kGemvFused>(codes, nullptr, p, st);
}

template <int FMT>
int launch_planes(const uint8_t* codes, const uint8_t* digits, const Params& p, cudaStream_t st) {
    if (p.M <= 6) return launch_tiles<FMT, 48, kGemvPlanes>(codes, digits, p, st);
    return launch_tiles<FMT, 64, kGemvPlanes>(codes, digits, p, st);
}

// Whether f4_mm runs the CTA pairs (f4_pair.cu): wide tiles for many tokens, unless
// one round of 128 x 64 tiles covers y.  us of the 128 x 64 tiles and of the pairs, NV;
// the rule takes the pairs from | on:
//   tokens               65           128           256           448           512          1024
//   2560 x 4096      7.1  8.4      7.6  8.8      8.6  8.9      9.9  9.2  |  11.3  9.2     16.0   9.9
//   2560 x 9728      9.1 15.4      9.7 15.9     11.5 15.9     14.1 16.0  |  19.4 16.0     30.2  16.8
//   6144 x 2560      8.3  7.2      8.3  7.5  |   9.2  7.6     12.4  8.2     12.4  8.2     17.1  11.8
//   19456 x 2560  | 16.5 16.1     14.4 12.6     17.3 12.2     21.5 15.5     24.8 15.7     45.5  29.0
//   50257 x 2560  | 27.8 37.4     20.6 30.3     33.0 30.3     55.9 59.0     62.1 60.6    119.7 117.0
// (MX alike.)  It is off where it turns a few tokens too late (6144 x 2560 at 65 to 192
// tokens up to a fifth, 2560 x 4096 at 384 and 448 a tenth) and where absent tokens
// fill the pairs' 256-token tiles and their rows of y start off 16 bytes (50257 rows
// at 65 to 192 and at 384 tokens: a fifth to a half more).
bool pairs(int64_t M, int64_t N) {
    return M > 64 && row_tiles(N) * ((M + 63) / 64) > w4::sm_count();
}

bool bad_scalar(const float* g) { return (reinterpret_cast<uintptr_t>(g) & 3u) != 0; }

int fill(Params& p, const uint8_t* scales, const float* g, int64_t N, int64_t K, int format,
         int64_t M, void* y, int out_dtype) {
    p = Params{};
    p.err = w4::device_error_word();
    if (!p.err) return W4_ERR_CUDA;
    p.sa = scales;
    p.gw = g;
    p.y = y;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.stages_k = (int)((K + BK - 1) / BK);
    p.tiles_k = (int)f4::scale_tiles_k(K, format);
    p.out_f32 = out_dtype == W4_OUT_F32;
    return W4_OK;
}

// f4_gemv's workspace: digit codes, their scale tiles, a factor for each token.
struct GemvWs {
    size_t scales, factors, total;
};
GemvWs gemv_ws(int64_t M, int64_t K, int format) {
    GemvWs w;
    w.scales = (size_t)(M * kDigits * K / 2 + 511) / 512 * 512;
    w.factors = w.scales + (size_t)f4::scale_tiles_k(K, format) * f4::kTileBytes;
    w.total = w.factors + kMaxTokens * sizeof(float);
    return w;
}

constexpr int64_t kMaxGemvK = 65536;

bool gemv_range(int64_t M, int64_t N, int64_t K) {
    return M >= 1 && M <= kMaxTokens && N >= 1 && N <= f4::kMaxRows && K >= 32 && K % 32 == 0 &&
           K <= kMaxGemvK;
}

}  // namespace

extern "C" {

int f4_mm(const uint8_t* codes, const uint8_t* scales, const float* g, int64_t N, int64_t K,
          int format, const uint8_t* qa, const uint8_t* sa, const float* ga, int64_t M, void* y,
          int out_dtype, void* stream) {
    if (M < 1 || N < 1 || K < 32 || K % 32 != 0 || K > f4::kMaxK || M > f4::kMaxRows ||
        N > f4::kMaxRows || !f4::known_format(format) || !f4::known_out(out_dtype))
        return W4_ERR_SHAPE;
    const bool nv = format == W4_F4_NV;
    if (!codes || !scales || !qa || !sa || !y || (nv && (!g || !ga))) return W4_ERR_NULL;
    if (!w4::aligned16(codes) || !w4::aligned16(scales) || !w4::aligned16(qa) ||
        !w4::aligned16(sa) || !w4::aligned16(y) || (nv && (bad_scalar(g) || bad_scalar(ga))))
        return W4_ERR_ALIGN;
    int rc = w4::check_device();
    if (rc != W4_OK) return rc;
    if (pairs(M, N)) {
        const PairArgs a{codes, scales, g, N, K, qa, sa, ga, M, y, w4::device_error_word()};
        return launch_pair(a, format, out_dtype, (cudaStream_t)stream);
    }
    Params p;
    rc = fill(p, scales, g, N, K, format, M, y, out_dtype);
    if (rc != W4_OK) return rc;
    p.sb = sa;
    p.ga = ga;
    p.b_rows = (int)M;
    return nv ? launch_mm<W4_F4_NV>(codes, qa, p, (cudaStream_t)stream)
              : launch_mm<W4_F4_MX>(codes, qa, p, (cudaStream_t)stream);
}

int w4_test_f4_mm_pairs(int64_t M, int64_t N) {
    if (M < 1 || N < 1 || M > f4::kMaxRows || N > f4::kMaxRows) return -1;
    (void)w4::check_device();  // sm_count knows the device from here on
    return pairs(M, N) ? 1 : 0;
}

size_t f4_gemv_workspace_size(int64_t M, int64_t N, int64_t K, int format) {
    if (!gemv_range(M, N, K) || !f4::known_format(format) || one_kernel(M, N, K, format)) return 0;
    return gemv_ws(M, K, format).total;
}

int f4_gemv(const uint8_t* codes, const uint8_t* scales, const float* g, int64_t N, int64_t K,
            int format, const uint16_t* x_bf16, int M, void* y, int out_dtype, void* workspace,
            size_t ws_bytes, void* stream) {
    if (!gemv_range(M, N, K) || !f4::known_format(format) || !f4::known_out(out_dtype))
        return W4_ERR_SHAPE;
    const bool nv = format == W4_F4_NV;
    if (!codes || !scales || !x_bf16 || !y || (nv && !g)) return W4_ERR_NULL;
    if (!w4::aligned16(codes) || !w4::aligned16(scales) || !w4::aligned16(x_bf16) ||
        !w4::aligned16(y) || (nv && bad_scalar(g)))
        return W4_ERR_ALIGN;
    const bool fused = one_kernel(M, N, K, format);
    const GemvWs ws = gemv_ws(M, K, format);
    if (!fused) {
        if (!workspace || ws_bytes < ws.total) return W4_ERR_WORKSPACE;
        if (!w4::aligned16(workspace)) return W4_ERR_ALIGN;
    }
    int rc = w4::check_device();
    if (rc != W4_OK) return rc;
    Params p;
    rc = fill(p, scales, g, N, K, format, M, y, out_dtype);
    if (rc != W4_OK) return rc;
    p.b_rows = M * kDigits;
    const cudaStream_t st = (cudaStream_t)stream;
    if (fused) {
        p.x = x_bf16;
        return nv ? launch_fused<W4_F4_NV>(codes, p, st) : launch_fused<W4_F4_MX>(codes, p, st);
    }
    uint8_t* base = static_cast<uint8_t*>(workspace);
    float* factors = reinterpret_cast<float*>(base + ws.factors);
    p.sb = base + ws.scales;
    p.row_factor = factors;
    const int kpad = p.tiles_k * 4 * f4::block_of(format);
    const dim3 grid((unsigned)((kpad + kDigitElems - 1) / kDigitElems), (unsigned)M);
    rc = launch_dependent(nv ? digits_kernel<W4_F4_NV> : digits_kernel<W4_F4_MX>, grid, kDigitThreads,
                          st, x_bf16, (int)K, base, base + ws.scales, factors,
                          many_tiles(row_tiles(N), (int64_t)w4::sm_count() * 2), p.err);
    if (rc != W4_OK) return rc;
    return nv ? launch_planes<W4_F4_NV>(codes, base, p, st)
              : launch_planes<W4_F4_MX>(codes, base, p, st);
}

}  // extern "C"
