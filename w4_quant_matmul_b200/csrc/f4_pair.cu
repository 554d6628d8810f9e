// f4_pair.cu -- the f4_mm kernel for many tokens: CTA pairs on 256 x 192 tiles.
//
//   y[t][n] = gw ga sum_k (q s)_w[n][k] (q s)_a[t][k]
//
// Two CTAs of a cluster work one tile with tcgen05.mma.cta_group::2 (M = 256
// tokens, 128 in each CTA's TMEM lanes; N = 192 weight rows, 96 of them staged
// by each CTA), so that an SM's shared memory delivers 7 KB of operands for
// every 96 tensor cycles.  K advances in stages of 256.
//   warp 0     of each CTA: TMA loads of its token rows, its half of the weight
//              rows and their scale tiles (the weights' scales for all 192 rows:
//              each CTA's TMEM needs them), all counted by the leader's barrier.
//   warp 1     TMEM allocation; in the leader, scale copies and MMAs.
//   warps 2-9  epilogue.  Tokens are TMEM lanes, so a thread holds consecutive
//              columns of one row of y; a warp turns 32 rows x 32 columns through
//              shared memory and stores them 16 bytes a lane, along the rows.
// 192 columns is the widest tile whose accumulators fit TMEM twice beside the
// scales (2 * 192 + 2 * 48 of 512 columns), so the epilogue of a tile runs under
// the MMAs of the next.  192 rows of weights are one and a half scale tiles:
// two are staged, and odd tiles start at the TMEM column of row 64.
#include <cuda_bf16.h>

#include "f4_pair.cuh"
#include "f4_tc.cuh"

namespace {

using namespace f4;

constexpr int PM = 128;          // tokens of a CTA
constexpr int PN = 192;          // weight rows of the pair
constexpr int PH = PN / 2;       // staged by a CTA
constexpr int kEpiWarps = 8;     // two to a TMEM lane quarter
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kChunk = 32;       // columns that an epilogue warp stages at a time
constexpr int kAccStages = 2;
constexpr int kSfSlots = 2;

template <int FMT>
struct Cfg {
    static constexpr int chunks = BK / (4 * block_of(FMT));
    static constexpr int mma_per_chunk = 4 / chunks;
    static constexpr int a_bytes = PM * kRowBytes;
    static constexpr int b_bytes = PH * kRowBytes;
    static constexpr int sa_bytes = chunks * kTileBytes;
    static constexpr int sb_bytes = 2 * chunks * kTileBytes;
    static constexpr int stage_bytes = a_bytes + b_bytes + sa_bytes + sb_bytes;
    static constexpr int stages = FMT == W4_F4_MX ? 6 : 5;
    static constexpr int sf_cols = 3 * chunks * 4;  // 4 a chunk for tokens, 8 for weights
    static constexpr int out = stages * stage_bytes;  // 32 rows x kChunk columns a warp
    static constexpr int bars = out + kEpiWarps * 32 * kChunk * 4;
    static constexpr int nbars = 2 * stages + 2 * kAccStages + 1;
    static constexpr int misc = bars + nbars * 8;
    static constexpr size_t total = (size_t)misc + 16 + 1024;
    static_assert(kAccStages * PN + kSfSlots * sf_cols <= 512, "TMEM has 512 columns");
    static_assert(stage_bytes % 1024 == 0 && b_bytes % 1024 == 0, "tiles start on swizzle atoms");
    static_assert(total <= kSmemMax, "shared memory of one CTA");
};
constexpr int kTmemCols = 512;

struct Params {
    const float* gw;
    const float* ga;
    void* y;
    int M, N, K;
    int stages_k;
    int tiles_k;
    int tiles_n, tiles_m;
    int* err;
};

// Address of the same shared-memory object in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(w4::smem_u32(p)), "r"(rank));
    return a;
}
// Relaxed: what it reports are TMEM reads, ordered by tcgen05.fence on both sides;
// a release at cluster scope would also wait for the warp's stores to y (2560 x
// 9728 at 2048 tokens and 1965 MHz: NV 28.6 -> 27.9 us, MX 25.3 -> 24.6).
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}
// 2-D tiled load into this CTA's shared memory, counted by a barrier of the pair.
__device__ __forceinline__ void load_pair(void* dst, const void* tmap, uint32_t bar, int32_t c0,
                                          int32_t c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(w4::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void copy_scales_pair(uint32_t tmem, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                 : "memory");
}
template <int FMT>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if constexpr (FMT == W4_F4_MX)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X"
            " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X"
            " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}
// Arrives at the barrier in both CTAs once all earlier MMAs are complete.
__device__ __forceinline__ void commit_both(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(w4::smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
        "[%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
          "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
          "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
          "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
          "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
          "+r"(r[31])
        :
        : "memory");
}

// 16-byte piece j of row r of a warp's staging tile with `pieces` (4 or 8) to a
// row, permuted so that a column of pieces and a row of them both spread over
// all banks.
template <int PIECES>
__device__ __forceinline__ uint32_t stage_at(int r, int j) {
    return r * (PIECES * 16) + ((j ^ ((PIECES == 8 ? r : r >> 1) & (PIECES - 1))) << 4);
}

template <int FMT, int OUT>
__global__ void __launch_bounds__(kThreads)
    f4_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                   const __grid_constant__ CUtensorMap tm_sa,
                   const __grid_constant__ CUtensorMap tm_sb, const Params p) {
    using C = Cfg<FMT>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // both CTAs start at the same offset, so an object has the same address in each
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::bars);  // leader: both CTAs' loads [stages]
    uint64_t* empty = full + C::stages;                            // stage consumed          [stages]
    uint64_t* afull = empty + C::stages;                           // tile accumulated        [2]
    uint64_t* aempty = afull + kAccStages;                         // leader: read out by both [2]
    uint64_t* drain = aempty + kAccStages;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::misc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::misc + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int tiles = p.tiles_n * p.tiles_m;
    const int first = blockIdx.x / 2, step = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::stages; ++i) {
            w4::mbar_init(&full[i], 1);
            w4::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kAccStages; ++i) {
            w4::mbar_init(&afull[i], 1);
            w4::mbar_init(&aempty[i], 2 * kEpiWarps);
        }
        w4::mbar_init(drain, 1);
        *abort_flag = 0;
        w4::fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         w4::smem_u32((const void*)tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer's barriers and TMEM are ready
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        if (w4::elect_one()) {
            w4::prefetch_tmap(&tm_a);
            w4::prefetch_tmap(&tm_b);
            w4::prefetch_tmap(&tm_sa);
            w4::prefetch_tmap(&tm_sb);
            pdl_wait();
            pdl_trigger();
            int it = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                const int tn = tile / p.tiles_m, tm = tile % p.tiles_m;
                (void)W4_CHECK(tn < p.tiles_n && tm < p.tiles_m, p.err);
                const int sa_row = (tm * 2 + (int)rank) * p.tiles_k;
                const int sb_row = tn * PN / kRowTile * p.tiles_k;
                for (int ks = 0; ks < p.stages_k; ++ks, ++it) {
                    const int s = it % C::stages;
                    if (!w4::mbar_wait(&empty[s], ((uint32_t)(it / C::stages) & 1u) ^ 1u, abort_flag,
                                       p.err)) {
                        ok = false;
                        break;
                    }
                    // the leader announces both CTAs' bytes
                    if (rank == 0) w4::mbar_arrive_expect_tx(&full[s], 2 * C::stage_bytes);
                    const uint32_t bar = in_cta(&full[s], 0);
                    uint8_t* st = smem + s * C::stage_bytes;
                    load_pair(st, &tm_a, bar, ks * kRowBytes, (tm * 2 + (int)rank) * PM);
                    load_pair(st + C::a_bytes, &tm_b, bar, ks * kRowBytes, tn * PN + (int)rank * PH);
                    uint8_t* sc = st + C::a_bytes + C::b_bytes;
                    load_pair(sc, &tm_sa, bar, 0, sa_row + ks * C::chunks);
                    load_pair(sc + C::sa_bytes, &tm_sb, bar, 0, sb_row + ks * C::chunks);
                    load_pair(sc + 2 * C::sa_bytes, &tm_sb, bar, 0,
                              sb_row + p.tiles_k + ks * C::chunks);
                }
            }
            // drain: the pair's loads must land before either CTA exits (both
            // CTAs meet once more after this)
            if (rank == 0)
                for (int k = it - C::stages < 0 ? 0 : it - C::stages; k < it; ++k)
                    w4::mbar_wait(&full[k % C::stages], (uint32_t)(k / C::stages) & 1u, nullptr,
                                  p.err);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer (leader) ----------------
        if (rank == 0 && w4::elect_one()) {
            const uint32_t sf0 = tmem + kAccStages * PN;
            int it = 0, ti = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step, ++ti) {
                const int tn = tile / p.tiles_m;
                const uint32_t sb_col = (uint32_t)(tn * PN % kRowTile / 32);
                const int as = ti % kAccStages;
                const uint32_t d = tmem + as * PN;
                if (!w4::mbar_wait(&aempty[as], ((uint32_t)(ti / kAccStages) & 1u) ^ 1u, abort_flag,
                                   p.err))
                    break;
                tc_fence_after();
                for (int ks = 0; ks < p.stages_k; ++ks, ++it) {
                    const int s = it % C::stages;
                    if (!w4::mbar_wait(&full[s], (uint32_t)(it / C::stages) & 1u, abort_flag, p.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = w4::smem_u32(smem + s * C::stage_bytes);
                    const uint32_t b = a + C::a_bytes;
                    const uint32_t sa = b + C::b_bytes;
                    const uint32_t sb = sa + C::sa_bytes;
                    const uint32_t sf = sf0 + (it % kSfSlots) * C::sf_cols;
                    const uint32_t sfb = sf + C::chunks * 4;
                    int steps = (p.K - ks * BK + kMmaK - 1) / kMmaK;
                    if (steps > BK / kMmaK) steps = BK / kMmaK;
                    // a chunk's scales directly before its MMAs, where their copies
                    // run beside the MMAs before (2048 x 19456 x 2560 of NV at
                    // 1965 MHz: 46.5 us; all of a stage's copies first 49.8, each
                    // chunk's one MMA earlier 50.8)
#pragma unroll
                    for (int j = 0; j < BK / kMmaK; ++j) {
                        if (j >= steps) break;
                        const int c = j / C::mma_per_chunk;
                        const int id = j % C::mma_per_chunk * 2;
                        if (id == 0) {
                            copy_scales_pair(sf + c * 4, scale_desc(sa + c * kTileBytes));
                            copy_scales_pair(sfb + c * 8, scale_desc(sb + c * kTileBytes));
                            copy_scales_pair(sfb + c * 8 + 4,
                                             scale_desc(sb + C::sa_bytes + c * kTileBytes));
                        }
                        mma_pair<FMT>(d, operand_desc(a + j * (kMmaK / 2)),
                                      operand_desc(b + j * (kMmaK / 2)),
                                      instr_desc<FMT, 2 * PM, PN>(id), sf + c * 4,
                                      sfb + c * 8 + sb_col, ks > 0 || j > 0);
                    }
                    commit_both(&empty[s]);
                }
                if (ok) commit_both(&afull[as]);
            }
            asm volatile(
                "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                    w4::smem_u32(drain))
                : "memory");
            w4::mbar_wait(drain, 0u, nullptr, p.err);
        }
    } else {
        // ---------------- epilogue ----------------
        constexpr bool f32 = OUT == W4_OUT_F32;
        constexpr int esize = f32 ? 4 : 2;
        constexpr int vec = 16 / esize;             // columns of a 16-byte piece
        constexpr int pieces = kChunk / vec;        // 16-byte pieces of a staged row
        constexpr int rows_step = 32 / pieces;      // rows that a warp stores at once
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        uint8_t* st = smem + C::out + (warp - 2) * 32 * kChunk * 4;
        pdl_wait();
        Factors scale{1.0f, 1.0f};
        if constexpr (FMT == W4_F4_NV) scale = factors(__ldca(p.gw), __ldca(p.ga));
        const bool aligned = p.N % vec == 0;  // rows of y start on 16 bytes
        int ti = 0;
        for (int tile = first; tile < tiles; tile += step, ++ti) {
            const int tn = tile / p.tiles_m, tm = tile % p.tiles_m;
            const int as = ti % kAccStages;
            const int t0 = (tm * 2 + (int)rank) * PM + quarter * 32;
            if (!w4::mbar_wait(&afull[as], (uint32_t)(ti / kAccStages) & 1u, abort_flag, p.err)) break;
            tc_fence_after();
            const uint32_t acc = tmem + as * PN + ((uint32_t)(quarter * 32) << 16);
            // chunks half, half + 2, half + 4; each is on its way from TMEM while
            // the one before it is stored
            uint32_t r[32];
            tmem_ld32(acc + half * kChunk, r);
#pragma unroll
            for (int i3 = 0; i3 < PN / kChunk / 2; ++i3) {
                const int c0 = (2 * i3 + half) * kChunk;
                const int n0 = tn * PN + c0;
                tmem_wait32(r);
                if (scale.first != 1.0f) {  // hardly ever: a multiply each else (51.2 -> 51.7 us)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        r[i] = __float_as_uint(__uint_as_float(r[i]) * scale.first);
                }
                __syncwarp();  // the previous chunk has been read
#pragma unroll
                for (int j = 0; j < pieces; ++j) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (f32) {
                            w[i] = __float_as_uint(__uint_as_float(r[4 * j + i]) * scale.second);
                        } else {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(
                                __uint_as_float(r[8 * j + 2 * i]) * scale.second,
                                __uint_as_float(r[8 * j + 2 * i + 1]) * scale.second);
                            w[i] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                    }
                    *reinterpret_cast<uint4*>(st + stage_at<pieces>(lane, j)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
                __syncwarp();
                if (i3 + 1 < PN / kChunk / 2) {
                    tmem_ld32(acc + c0 + 2 * kChunk, r);
                } else {  // the accumulators have been read
                    tc_fence_before();
                    if (lane == 0) arrive_at(in_cta(&aempty[as], 0));
                }
                if (t0 >= p.M || n0 >= p.N) continue;
                if (aligned) {
                    const int j = lane % pieces;
                    const bool in = n0 + (j + 1) * vec <= p.N;
                    const int64_t at =
                        ((int64_t)(t0 + lane / pieces) * p.N + n0 + j * vec) * esize;
                    uint8_t* y = static_cast<uint8_t*>(p.y) + at;
#pragma unroll
                    for (int i = 0; i < pieces; ++i) {
                        const int row = i * rows_step + lane / pieces;
                        const uint4 v = *reinterpret_cast<const uint4*>(st + stage_at<pieces>(row, j));
                        if (in && t0 + row < p.M &&
                            W4_CHECK(at >= 0 && at + (int64_t)i * rows_step * p.N * esize + 16 <=
                                                    (int64_t)p.M * p.N * esize, p.err))
                            *reinterpret_cast<uint4*>(y + (int64_t)i * rows_step * p.N * esize) = v;
                    }
                } else if (n0 + lane < p.N) {  // one column a lane
                    const uint32_t in_piece = lane % vec * esize;
                    for (int row = 0; row < 32 && t0 + row < p.M; ++row) {
                        const uint8_t* v = st + stage_at<pieces>(row, lane / vec) + in_piece;
                        const int64_t o = (int64_t)(t0 + row) * p.N + n0 + lane;
                        if (!W4_CHECK(o >= 0 && o < (int64_t)p.M * p.N, p.err)) continue;
                        if constexpr (f32)
                            static_cast<uint32_t*>(p.y)[o] = *reinterpret_cast<const uint32_t*>(v);
                        else
                            static_cast<uint16_t*>(p.y)[o] = *reinterpret_cast<const uint16_t*>(v);
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the pair still works on its memory
    tc_fence_after();
    if (warp == 1) {
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols)
                     : "memory");
    }
}

// Scale plane as rows of one tile each (128 words); a box is one stage's tiles.
bool make_scale_map(CUtensorMap* map, const void* scales, int64_t rows, int chunks) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {kTileBytes / 4, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {kTileBytes};
    const cuuint32_t box[2] = {kTileBytes / 4, (cuuint32_t)chunks};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(scales), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <int FMT, int OUT>
int launch(const PairArgs& g, cudaStream_t stream) {
    using C = Cfg<FMT>;
    Params p{};
    p.gw = g.gw;
    p.ga = g.ga;
    p.y = g.y;
    p.M = (int)g.M;
    p.N = (int)g.N;
    p.K = (int)g.K;
    p.stages_k = (int)((g.K + BK - 1) / BK);
    p.tiles_k = (int)scale_tiles_k(g.K, FMT);
    p.tiles_n = (p.N + PN - 1) / PN;
    p.tiles_m = (p.M + 2 * PM - 1) / (2 * PM);
    p.err = g.err;
    const int64_t tiles = (int64_t)p.tiles_n * p.tiles_m;
    if (tiles > INT32_MAX / 2) return W4_ERR_SHAPE;
    CUtensorMap ma, mb, msa, msb;
    if (!make_map(&ma, g.qa, g.K, g.M, PM) || !make_map(&mb, g.codes, g.K, g.N, PH) ||
        !make_scale_map(&msa, g.sa, row_tiles(g.M) * p.tiles_k, C::chunks) ||
        !make_scale_map(&msb, g.scales, row_tiles(g.N) * p.tiles_k, C::chunks))
        return W4_ERR_CUDA;
    auto kernel = f4_pair_kernel<FMT, OUT>;
    static thread_local int attr_dev = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return w4::cuda_fail(e);
    if (attr_dev != dev) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::total);
        if (e != cudaSuccess) return w4::cuda_fail(e);
        attr_dev = dev;
    }
    const int64_t pairs = w4::sm_count() / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::total;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kernel, ma, mb, msa, msb, p);
    if (e != cudaSuccess) return w4::cuda_fail(e);
    return w4::launch_status();
}

}  // namespace

namespace f4 {

int launch_pair(const PairArgs& g, int format, int out_dtype, cudaStream_t stream) {
    if (format == W4_F4_MX)
        return out_dtype == W4_OUT_F32 ? launch<W4_F4_MX, W4_OUT_F32>(g, stream)
                                       : launch<W4_F4_MX, W4_OUT_BF16>(g, stream);
    return out_dtype == W4_OUT_F32 ? launch<W4_F4_NV, W4_OUT_F32>(g, stream)
                                   : launch<W4_F4_NV, W4_OUT_BF16>(g, stream);
}

}  // namespace f4
