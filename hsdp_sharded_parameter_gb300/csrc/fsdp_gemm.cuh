// Products of 16-bit matrices on the tensor cores, D = sum of A B^T in
// binary32, with what becomes of D's elements left to the caller (an epilogue:
// `once`, what a thread works out before its first tile; `bring`, what it loads
// while a granule's sums are under way; and the call on the sums). Included by
// the operators that need one.
//
// A pair of SMs (a cluster of two blocks) computes tiles of 256 x kN, one
// after the other: each block brings its 128 rows of A and its half of B's kN
// rows into shared memory (TMA, a ring of stages of 64 along k), one thread
// of the first block issues the tensor cores' instructions for both, which
// read both blocks' shared memory and leave 128 x kN sums in each block's
// tensor memory, and four warps of each block take them from there while the
// next tile is computed into the tensor memory's other half.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "fsdp_ops.cuh"

namespace fsdp {
namespace {

// ------------------------------------------------------------------ on the host

// Element (i, k) of a factor: data[i * stride + k], or, where its rows are the
// neighbours in memory (mn), data[k * stride + i].
struct Product {
    int64_t m, n;
    int terms;     // products summed: 1 or 2
    int64_t k[2];  // their lengths
    Mat a[2], b[2];
    int a_mn, b_mn;
    int half;       // binary16 values instead of bfloat16
    int paired;     // two products with the same A and k, by b[0] and b[1], side by side
    int symmetric;  // D is: what lies above the diagonal's tiles is mirrored
};

constexpr int kTileM = 256, kStep = 64;
constexpr int kMaxGroup = 3;
constexpr int kPairs = 76;  // of SMs, for what depends on the sizes alone

// What a launch computes: one product, or up to three with the same k.
struct Tiles {
    CUtensorMap a[kMaxGroup], b[kMaxGroup];  // one a term, or one a product of the group
    int m[kMaxGroup], n[kMaxGroup];
    int tiles_m[kMaxGroup], tiles_n[kMaxGroup], first[kMaxGroup + 1];
    int group, paired, symmetric;
    int steps[2];  // along k, of each term
    int splits, each;  // parts of all steps, and steps a part
    int a_mn, b_mn;
    uint32_t kind;
};

// ------------------------------------------------------------------ barriers

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t* b, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ bool bar_test(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(smem_addr(b)), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint64_t clock_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Set by a product whose wait ran out.
__device__ int gave_up;
constexpr uint64_t kWaitNs = 2000000000ull;
// Waits for the phase of a parity: false, and said so, once two seconds have
// passed. (The clock is read seldom: a read takes longer than a step of the
// products, and the wait does not see its phase end meanwhile.)
__device__ __noinline__ bool bar_wait_long(uint64_t* b, uint32_t parity) {
    const uint64_t from = clock_ns();
    for (uint32_t i = 0; i < (1u << 20); ++i) {
        for (int k = 0; k < 256; ++k)
            if (bar_test(b, parity)) return true;
        if (clock_ns() - from > kWaitNs) break;
    }
    atomicOr(&gave_up, 1);
    return false;
}
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity) {
#pragma unroll 1
    for (int i = 0; i < 1024; ++i)
        if (bar_test(b, parity)) return true;
    return bar_wait_long(b, parity);
}
__device__ __forceinline__ uint32_t in_first_block(const void* p) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_addr(p)));
    return r;
}
__device__ __forceinline__ void bar_arrive_remote(uint32_t at) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(at) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// One lane of a warp, which the compiler knows to be one: the operands of the
// copies and of the tensor cores' instructions are a warp's, and behind a
// comparison of lanes each is brought there by a loop over the lanes.
__device__ __forceinline__ bool one_lane() {
    uint32_t one;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(one));
    return one != 0;
}

// --------------------------------------------------- tensor core instructions

__device__ __forceinline__ void tmem_alloc(uint32_t* where, int columns) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t at, int columns) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}
// D (+)= A B^T of one step of 16 along k, of both blocks, by one thread.
__device__ __forceinline__ void mma_step(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, uint32_t add) {
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a), "l"(b),
                 "r"(kind), "r"(add)
                 : "memory");
}
// Arrives on a barrier of both blocks once the thread's products so far are done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t at, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// A box of a matrix into this block's shared memory; its bytes count on a
// barrier of the first block.
__device__ __forceinline__ void tma_load(uint32_t to, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(to),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// What a step's instruction does: binary32 sums of M x N, both factors of one
// 16-bit type, each either with its k or with its rows as neighbours.
inline uint32_t mma_kind(bool half, bool a_mn, bool b_mn, int m, int n) {
    const uint32_t type = half ? 0u : 1u;
    return 1u << 4 | type << 7 | type << 10 | (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16 | (uint32_t)(n >> 3) << 17 |
           (uint32_t)(m >> 4) << 24;
}
// A factor's tile in shared memory: rows of 128 bytes, their 16-byte pieces
// swapped by the row's last three bits (the 128-byte swizzle). With k as
// neighbours a row holds 64 of k; with rows as neighbours it holds 64 rows of
// one k, and the next 64 rows lie a box of 64 of those further.
constexpr uint32_t kBoxBytes = 64 * 128;
__device__ __forceinline__ uint64_t tile_descriptor(uint32_t at, bool mn) {
    const uint64_t lead = mn ? kBoxBytes >> 4 : 1, step = 1024 >> 4;
    return (uint64_t)(at >> 4 & 0x3fff) | lead << 16 | step << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// --------------------------------------------------------------- the product

constexpr int kEpiWarps = 4, kThreads = 128 + 32 * kEpiWarps;
constexpr int kPitch = 36;  // floats: a row of 32 and a shift that keeps rows on different banks
constexpr int kStageRoom = 32 * kPitch * 4;
template <int kN>
constexpr int kStageBytes = (128 + kN / 2) * 128;
template <int kN>
constexpr int kStages = kN == 256 ? 6 : 8;
template <int kN>
constexpr int kProductSmem = kStages<kN> * kStageBytes<kN> + kEpiWarps * kStageRoom + 1024;

// A tile's place in its product.
struct Place {
    int product, tm, tn;
};
// Tiles in bands of 8 rows of tiles, whose rows of A and columns of B the L2
// cache holds while the band's tiles are computed.
__device__ __forceinline__ Place place_of(const Tiles& t, int tile) {
    Place p = {0, 0, 0};
    if (t.symmetric) {
        // row i of tiles holds the first (i + 1) * wide of its columns
        const int wide = t.symmetric;
        int i = (int)((sqrtf(1.0f + 8.0f * (float)tile / (float)wide) - 1.0f) * 0.5f);
        while (i > 0 && (int64_t)i * (i + 1) / 2 * wide > tile) --i;
        while ((int64_t)(i + 1) * (i + 2) / 2 * wide <= tile) ++i;
        p.tm = i;
        p.tn = (int)(tile - (int64_t)i * (i + 1) / 2 * wide);
        return p;
    }
    while (p.product + 1 < t.group && tile >= t.first[p.product + 1]) ++p.product;
    tile -= t.first[p.product];
    const int tiles_m = t.tiles_m[p.product], tiles_n = t.tiles_n[p.product];
    constexpr int kBand = 8;
    const int band = tile / (kBand * tiles_n), in = tile - band * kBand * tiles_n;
    const int rows = min(kBand, tiles_m - band * kBand);
    p.tm = band * kBand + in % rows;
    p.tn = in / rows;
    return p;
}

// The 32 x 32 sums of a warp's rows, from a row a lane to 8 columns of the rows
// lane / 4, + 8, + 16, + 24.
__device__ __forceinline__ void across(float* stage, const float (&v)[32], Cols (&out)[4], int lane) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *reinterpret_cast<float4*>(stage + lane * kPitch + 4 * j) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4* q = reinterpret_cast<const float4*>(stage + (8 * i + lane / 4) * kPitch + lane % 4 * 8);
        const float4 a = q[0], b = q[1];
        out[i] = {{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
    }
}

template <int kN, typename Epi>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ Tiles t, const Epi epi) {
    constexpr int kStg = kStages<kN>, kBytes = kStageBytes<kN>;
    extern __shared__ char raw[];
    __shared__ uint64_t full[kStg], empty[kStg], done[2], taken[2], drained;
    __shared__ uint32_t tmem_at;
    char* base = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
    float* stages = reinterpret_cast<float*>(base + kStg * kBytes);
    const int warp = __shfl_sync(kFull, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStg; ++i) {
            bar_init(&full[i], 1);
            bar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&done[i], 1);
            bar_init(&taken[i], 2 * kEpiWarps);
        }
        bar_init(&drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    if (warp == 2) tmem_alloc(&tmem_at, 2 * kN);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_meet();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_at;
    allow_next();
    wait_for_previous();

    const int tiles = t.first[t.group], items = tiles * t.splits, steps = t.steps[0] + t.steps[1];
    const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    if (warp == 0) {
        if (one_lane()) {
            // brings the tiles' rows
            int stage = 0, brought = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int item = pair; item < items && ok; item += pairs) {
                const int split = item % t.splits;
                const Place p = place_of(t, item / t.splits);
                const int row = p.tm * kTileM + (int)rank * 128;
                const int col = t.paired ? p.tn * (kN / 2) : p.tn * kN + (int)rank * (kN / 2);
                const int from = split * t.each, to = min(steps, from + t.each);
                for (int s = from; s < to; ++s) {
                    ok = bar_wait(&empty[stage], phase ^ 1);
                    if (!ok) break;
                    const int term = s >= t.steps[0];
                    const CUtensorMap* ma = &t.a[t.group > 1 ? p.product : term];
                    const CUtensorMap* mb = &t.b[t.group > 1 ? p.product : (t.paired ? (int)rank : term)];
                    const int k = (s - (term ? t.steps[0] : 0)) * kStep;
                    const uint32_t at = smem_addr(base + stage * kBytes), bar = in_first_block(&full[stage]);
                    if (rank == 0) bar_expect(&full[stage], 2 * kBytes);
                    if (t.a_mn) {
                        tma_load(at, ma, row, k, bar);
                        tma_load(at + kBoxBytes, ma, row + 64, k, bar);
                    } else {
                        tma_load(at, ma, k, row, bar);
                    }
                    if (t.b_mn) {
#pragma unroll
                        for (int j = 0; j < kN / 128; ++j) tma_load(at + 128 * 128 + j * kBoxBytes, mb, col + 64 * j, k, bar);
                    } else {
                        tma_load(at + 128 * 128, mb, k, col, bar);
                    }
                    ++brought;
                    if (++stage == kStg) stage = 0, phase ^= 1;
                }
            }
            // What is on its way here has to arrive before the block ends. The
            // first block sees it on its barriers. The second's copies count
            // there too: it waits until its last stages have been read, and
            // where that does not come, for a time in which copies do.
            const int last = min(brought, kStg);
            if (rank == 0) {
                for (int j = brought - 1; j >= brought - last; --j)
                    if (!bar_wait(&full[j % kStg], (uint32_t)(j / kStg & 1))) break;
            } else {
                for (int j = brought - 1; j >= brought - last && ok; --j) ok = bar_wait(&empty[j % kStg], (uint32_t)(j / kStg & 1));
                if (!ok) {
                    const uint64_t from = clock_ns();
                    for (int i = 0; i < 100000 && clock_ns() - from < 100000000ull; ++i) __nanosleep(1000);
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && one_lane()) {
            // issues the products
            int stage = 0, n_done = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int item = pair; item < items && ok; item += pairs, ++n_done) {
                const int split = item % t.splits, from = split * t.each, to = min(steps, from + t.each);
                const int half = n_done & 1;
                ok = bar_wait(&taken[half], (uint32_t)(n_done >> 1 & 1) ^ 1);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                for (int s = from; s < to; ++s) {
                    ok = bar_wait(&full[stage], phase);
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t at = smem_addr(base + stage * kBytes);
                    const uint64_t a = tile_descriptor(at, t.a_mn), b = tile_descriptor(at + 128 * 128, t.b_mn);
                    const uint64_t da = (t.a_mn ? 2048 : 32) >> 4, db = (t.b_mn ? 2048 : 32) >> 4;
#pragma unroll
                    for (int i = 0; i < kStep / 16; ++i) mma_step(tmem + half * kN, a + i * da, b + i * db, t.kind, s > from || i > 0);
                    mma_commit(&empty[stage]);
                    if (++stage == kStg) stage = 0, phase ^= 1;
                }
                if (ok) mma_commit(&done[half]);
            }
            // None of the tensor cores' work is under way when the blocks end: the
            // takers of the last sums would see it end, but may have given up.
            mma_commit(&drained);
            bar_wait(&drained, 0);
        }
    } else if (warp >= 4) {
        // takes the sums
        const int quarter = warp % 4;
        const typename Epi::Once once = epi.once();
        float* stage = stages + (warp - 4) * (kStageRoom / 4);
        int n_done = 0;
        for (int item = pair; item < items; item += pairs, ++n_done) {
            const int split = item % t.splits;
            const Place p = place_of(t, item / t.splits);
            const int half = n_done & 1;
            const int64_t row0 = (int64_t)p.tm * kTileM + rank * 128 + quarter * 32, m = t.m[p.product], n = t.n[p.product];
            const int64_t col0 = (int64_t)p.tn * (t.paired ? kN / 2 : kN);
            const bool mirror = Epi::kMirror && t.symmetric && p.tn < p.tm * t.symmetric;
            if (!__all_sync(kFull, bar_wait(&done[half], (uint32_t)(n_done >> 1 & 1)))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t at = tmem + half * kN + ((uint32_t)(quarter * 32) << 16);
            const int width = t.paired ? kN / 2 : kN;
            for (int c = 0; c < width; c += 32) {
                typename Epi::Before before[4];
                const int64_t col = col0 + c + lane % 4 * 8;
                const int cols = (int)(n - col < 8 ? (n > col ? n - col : 0) : 8);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t row = row0 + 8 * i + lane / 4;
                    if (row < m && cols > 0) epi.bring(p.product, row, col, cols, before[i]);
                }
                __syncwarp();
                Cols x[4], y[4];
                {
                    float v[32];
                    tmem_load32(at + c, v);
                    across(stage, v, x, lane);
                }
                if (t.paired) {
                    float v[32];
                    tmem_load32(at + kN / 2 + c, v);
                    across(stage, v, y, lane);
                }
                if (c + 32 >= width) {
                    // the last sums are out: the next tile but one may follow
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) bar_arrive_remote(in_first_block(&taken[half]));
                }
                Raw<uint16_t> r[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t row = row0 + 8 * i + lane / 4;
                    if (row < m && cols > 0) epi(p.product, split, row, col, cols, x[i], y[i], before[i], once, r[i]);
                }
                if constexpr (Epi::kMirror) {
                    if (mirror) {
                        // the same 32 x 32 values with rows and columns exchanged (a tile below
                        // the diagonal has all its columns)
                        constexpr int kPitch16 = 40;
                        uint16_t* box = reinterpret_cast<uint16_t*>(stage);
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<uint4*>(box + (8 * i + lane / 4) * kPitch16 + lane % 4 * 8) = make_uint4(r[i].w[0], r[i].w[1], r[i].w[2], r[i].w[3]);
                        __syncwarp();
                        const int64_t to = row0 + lane % 4 * 8;
                        const int left = (int)(m - to < 8 ? (m > to ? m - to : 0) : 8);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int j = 8 * i + lane / 4;
                            Raw<uint16_t> q;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                q.w[e] = (uint32_t)box[(lane % 4 * 8 + 2 * e) * kPitch16 + j] | (uint32_t)box[(lane % 4 * 8 + 2 * e + 1) * kPitch16 + j] << 16;
                            if (left > 0) epi.put(col0 + c + j, to, left, q);
                        }
                        __syncwarp();
                    }
                }
            }
        }
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_meet();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    __syncwarp();
    if (warp == 2) tmem_free(tmem, 2 * kN);
}

// --------------------------------------------------------- parts along k

// A part's sums as they are, [split][plane][m][ld].
struct Parts {
    static constexpr bool kMirror = false;
    struct Before {};
    struct Once {};
    float* sums;
    int64_t m, ld;
    int planes;
    __device__ __forceinline__ Once once() const { return {}; }
    __device__ __forceinline__ void bring(int, int64_t, int64_t, int, Before&) const {}
    __device__ __forceinline__ void operator()(int, int split, int64_t row, int64_t col, int, const Cols& x, const Cols& y, const Before&,
                                               Once, Raw<uint16_t>&) const {
        // ld is whole granules: the columns past n are sums of zeros
        float4* p = reinterpret_cast<float4*>(sums + ((int64_t)split * planes * m + row) * ld + col);
        p[0] = make_float4(x.p[0].x, x.p[0].y, x.p[1].x, x.p[1].y);
        p[1] = make_float4(x.p[2].x, x.p[2].y, x.p[3].x, x.p[3].y);
        if (planes == 2) {
            p = reinterpret_cast<float4*>(sums + (((int64_t)split * 2 + 1) * m + row) * ld + col);
            p[0] = make_float4(y.p[0].x, y.p[0].y, y.p[1].x, y.p[1].y);
            p[1] = make_float4(y.p[2].x, y.p[2].y, y.p[3].x, y.p[3].y);
        }
    }
};

// The parts' sums, in order (no parts: zeros), to the product's epilogue.
template <typename Epi>
__global__ void __launch_bounds__(256) join_kernel(const float* sums, int splits, int planes, int64_t m, int64_t n, int64_t ld, const Epi epi) {
    allow_next();
    wait_for_previous();
    const int64_t per = (n + kGran - 1) / kGran, granules = m * per;
    const typename Epi::Once once = epi.once();
    for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < granules; g += (int64_t)gridDim.x * 256) {
        const int64_t row = g / per, col = (g - row * per) * kGran;
        const int cols = n - col < kGran ? (int)(n - col) : kGran;
        typename Epi::Before before;
        epi.bring(0, row, col, cols, before);
        Cols x = all(0.0f), y = all(0.0f);
        for (int s = 0; s < splits; ++s) {
            for (int plane = 0; plane < planes; ++plane) {
                const float4* p = reinterpret_cast<const float4*>(sums + (((int64_t)s * planes + plane) * m + row) * ld + col);
                const float4 a = p[0], b = p[1];
                Cols& to = plane ? y : x;
                to = to + Cols{{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
            }
        }
        Raw<uint16_t> r;
        epi(0, 0, row, col, cols, x, y, before, once, r);
    }
}

// ------------------------------------------------------------------ launches

// The driver's call that describes a matrix to the copies (this library links
// no driver; nullptr where there is none).
inline decltype(&cuTensorMapEncodeTiled) map_encoder() {
    static const auto f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(p);
    }();
    return f;
}

// Whether the copies can read a matrix as it lies: rows on the 16-byte grid,
// none inside another.
inline bool copies_read(const Mat& f, int64_t rows, int64_t cols) {
    return on_grid(f, 2) && (rows <= 1 || f.stride >= cols) && f.stride < (int64_t)1 << 38;
}

// A rows x cols matrix in boxes of 64 columns and `box` rows.
inline cudaError_t make_map(CUtensorMap* map, const Mat& f, int64_t rows, int64_t cols, int box) {
    const auto encode = map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(rows > 1 ? f.stride : (cols + 7) / 8 * 8) * 2};
    const cuuint32_t boxes[2] = {64, (cuuint32_t)box}, ones[2] = {1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, f.data, dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
// A factor's map, whose rows and k are what the product says.
inline cudaError_t factor_map(CUtensorMap* map, const Mat& f, int64_t rows, int64_t k, int mn, int tile_rows) {
    return mn ? make_map(map, f, k, rows, kStep) : make_map(map, f, rows, k, tile_rows);
}

inline int64_t tiles_over(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }

// How a product is cut: the tile's width, and parts along k where whole tiles
// would leave most of the GPU idle.
struct Cut {
    int width, splits, each;
};
constexpr int kMostSplits = 64, kFewestSteps = 8;
inline int64_t tiles_of(const Product& p, int width) {
    const int64_t tm = tiles_over(p.m, kTileM), tn = tiles_over(p.n, p.paired ? width / 2 : width);
    if (!p.symmetric) return tm * tn;
    const int64_t wide = kTileM / width, whole = (tm - 1) * tm / 2 * wide;
    return whole + tn;  // the last row of tiles holds all columns
}
inline Cut cut_of(const Product& p, bool may_split) {
    // A tile half as wide is taken for 0.55 of a wide one. Measured, a wave of
    // them takes 0.5 to 0.7 of the time where the epilogue or a tile's start is
    // most of it (GatedGrad of 517 x 2048 33 us and 54, Gram of 1111 x 2049 17
    // and 24), and 0.7 to 0.8 where the products are, so near the border this is
    // too kind to slim tiles (4096 x 4096 x 4096 in 7 waves 113 us, 82 in 4 wide
    // ones) and right on either side of it (4096 x 11008, 10 wide waves 213 us
    // and 19 slim ones 305; 48 x 8192, one wave each, 129 and 108).
    const int64_t wide = tiles_of(p, 256), slim = tiles_of(p, 128);
    const double w = (double)tiles_over(wide, kPairs), s = 0.55 * (double)tiles_over(slim, kPairs);
    Cut c = {w <= s ? 256 : 128, 1, 0};
    const int64_t steps = tiles_over(p.k[0], kStep) + (p.terms > 1 ? tiles_over(p.k[1], kStep) : 0);
    // Parts of at least 8 steps, where they bring twice as many pairs to work: the
    // last product of one token, 32 tiles of 172 steps, takes 57 us whole, 41 in
    // parts and 3 to join them. Shorter ones lose (128 x 384, three products of 27
    // us whole, 21 in parts and 8 to join); those of 39 to 76 tiles are left whole,
    // though long ones would gain. In parts a symmetric product computes all tiles.
    Product full = p;
    full.symmetric = 0;
    const int64_t tiles = tiles_of(full, c.width);
    int64_t splits = 1;
    if (may_split && 2 * tiles <= kPairs) {
        splits = std::min<int64_t>({kPairs / std::max<int64_t>(tiles, 1), steps / kFewestSteps, kMostSplits});
        splits = std::max<int64_t>(splits, 1);
    }
    c.each = (int)std::max<int64_t>(tiles_over(steps, splits), 1);
    c.splits = (int)std::max<int64_t>(tiles_over(steps, c.each), 1);
    return c;
}
inline int64_t whole_granules(int64_t n) { return (n + kGran - 1) / kGran * kGran; }
// Bytes of the parts' sums of a product, and the most of any with as many rows or fewer.
inline size_t parts_bytes(const Product& p) {
    const Cut c = cut_of(p, true);
    return c.splits > 1 ? (size_t)(c.splits * (p.paired ? 2 : 1) * p.m * whole_granules(p.n)) * 4 : 0;
}
inline size_t parts_most_bytes(int64_t m, int64_t n, int planes) {
    const size_t each = (size_t)(m * whole_granules(n)) * 4 * planes, most = (size_t)kPairs * kTileM * 256 * 4;
    return each >= most / kMostSplits ? most : each * kMostSplits;
}

template <int kN, typename Epi>
cudaError_t launch_tiles(const Tiles& t, const Epi& epi, cudaStream_t s, bool first) {
    auto kernel = product_kernel<kN, Epi>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), kProductSmem<kN>, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {2, 1, 1};
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kProductSmem<kN>;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    // how many pairs fit the GPU at once, by device
    static std::atomic<int> fit[64];
    int dev = 0, pairs = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64) pairs = fit[dev].load(std::memory_order_relaxed);
    if (pairs == 0) {
        cfg.gridDim = dim3((unsigned)(sm_count() / 2 * 2));
        e = cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg);
        if (e != cudaSuccess) return e;
        if (pairs < 1) return cudaErrorInvalidConfiguration;
        if (dev < 64) fit[dev].store(pairs, std::memory_order_relaxed);
    }
    const int64_t items = (int64_t)t.first[t.group] * t.splits;
    cfg.gridDim = dim3(2 * (unsigned)std::min<int64_t>(pairs, items));
    cfg.numAttrs = first ? 1 : 2;
    count_launch();
    return cudaLaunchKernelEx(&cfg, kernel, t, epi);
}

// Up to three products with the same k, each with its own factors, in one
// launch. The first one's types and layouts are all of theirs.
template <typename Epi>
cudaError_t launch_group(const Product* p, int count, const Epi& epi, const Cut& c, cudaStream_t s, bool first) {
    Tiles t = {};
    t.group = count;
    t.paired = p[0].paired;
    t.symmetric = p[0].symmetric && c.splits == 1 ? kTileM / c.width : 0;
    t.splits = c.splits;
    t.each = c.each;
    t.a_mn = p[0].a_mn;
    t.b_mn = p[0].b_mn;
    t.kind = mma_kind(p[0].half, p[0].a_mn, p[0].b_mn, kTileM, c.width);
    for (int i = 0; i < p[0].terms; ++i) t.steps[i] = (int)tiles_over(p[0].k[i], kStep);
    int64_t tiles = 0;
    for (int g = 0; g < count; ++g) {
        Product q = p[g];
        q.symmetric = t.symmetric;
        t.m[g] = (int)q.m;
        t.n[g] = (int)q.n;
        t.tiles_m[g] = (int)tiles_over(q.m, kTileM);
        t.tiles_n[g] = (int)tiles_over(q.n, q.paired ? c.width / 2 : c.width);
        t.first[g] = (int)tiles;
        tiles += tiles_of(q, c.width);
        const int terms = count > 1 ? 1 : q.terms;
        cudaError_t e = cudaSuccess;
        for (int i = 0; i < terms && e == cudaSuccess; ++i) e = factor_map(&t.a[g + i], q.a[i], q.m, q.k[i], q.a_mn, 128);
        for (int i = 0; i < (q.paired ? 2 : terms) && e == cudaSuccess; ++i)
            e = factor_map(&t.b[g + i], q.b[i], q.n, q.k[q.paired ? 0 : i], q.b_mn, c.width / 2);
        if (e != cudaSuccess) return e;
    }
    if (tiles * t.splits > INT32_MAX - 1024) return cudaErrorInvalidValue;
    t.first[count] = (int)tiles;
    return c.width == 256 ? launch_tiles<256>(t, epi, s, first) : launch_tiles<128>(t, epi, s, first);
}

template <typename Epi>
cudaError_t launch_join(const float* sums, int splits, const Product& p, const Epi& epi, cudaStream_t s) {
    const int64_t granules = p.m * tiles_over(p.n, kGran);
    const int grid = (int)std::min<int64_t>(tiles_over(granules, 256), 8 * sm_count());
    count_launch();
    return launch_next(join_kernel<Epi>, dim3(grid), 256, 0, s, sums, splits, p.paired ? 2 : 1, p.m, p.n, whole_granules(p.n), epi);
}

// A product; `sums` has room for its parts, or is nullptr for none. `first`: of
// its call's kernels.
template <typename Epi>
cudaError_t launch_product(const Product& p, const Epi& epi, float* sums, cudaStream_t s, bool first) {
    if (p.m == 0 || p.n == 0) return cudaSuccess;
    if (p.k[0] == 0) return launch_join(nullptr, 0, p, epi, s);
    const Cut c = cut_of(p, sums != nullptr);
    if (c.splits == 1) return launch_group(&p, 1, epi, c, s, first);
    const cudaError_t e = launch_group(&p, 1, Parts{sums, p.m, whole_granules(p.n), p.paired ? 2 : 1}, c, s, first);
    return e == cudaSuccess ? launch_join(sums, c.splits, p, epi, s) : e;
}

// ------------------------------------------------- matrices off the grid

struct Copies {
    Mat from[5], to[5];
    int64_t rows[5], cols[5];
    int n;
};

// 16-bit matrices of any alignment and stride into rows on the 16-byte grid.
__global__ void __launch_bounds__(256) align_kernel(const Copies c) {
    allow_next();
    wait_for_previous();
    for (int i = 0; i < c.n; ++i) {
        const int64_t per = (c.cols[i] + kGran - 1) / kGran, granules = c.rows[i] * per;
        for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < granules; g += (int64_t)gridDim.x * 256) {
            const int64_t row = g / per, k = g - row * per;
            Raw<uint16_t> r;
            load_granule(r, static_cast<const uint16_t*>(c.from[i].data) + row * c.from[i].stride, k * kGran, granule_cols(k, c.cols[i]));
            store_raw(static_cast<uint16_t*>(c.to[i].data) + row * c.to[i].stride + k * kGran, r);
        }
    }
}
inline size_t aligned_room(int64_t rows, int64_t cols) { return (size_t)((rows * whole_granules(cols) * 2 + 255) / 256 * 256); }
// The matrix where the copies can read it: where it is, or, noted in `c`, at
// *room, which moves on.
inline Mat readable(const Mat& f, int64_t rows, int64_t cols, Copies* c, char** room) {
    if (copies_read(f, rows, cols)) return f;
    const Mat to = {*room, whole_granules(cols)};
    c->from[c->n] = f;
    c->to[c->n] = to;
    c->rows[c->n] = rows;
    c->cols[c->n] = cols;
    ++c->n;
    *room += aligned_room(rows, cols);
    return to;
}
inline cudaError_t launch_copies(const Copies& c, cudaStream_t s) {
    int64_t granules = 0;
    for (int i = 0; i < c.n; ++i) granules = std::max(granules, c.rows[i] * tiles_over(c.cols[i], kGran));
    if (granules == 0) return cudaSuccess;
    const int grid = (int)std::min<int64_t>(tiles_over(granules, 256), 8 * sm_count());
    count_launch();
    align_kernel<<<grid, 256, 0, s>>>(c);
    return cudaGetLastError();
}

// gave_up after what `s` holds, cleared.
inline cudaError_t take_gave_up(int* value, cudaStream_t s) {
    const int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(value, gave_up, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && *value) e = cudaMemcpyToSymbolAsync(gave_up, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace
}  // namespace fsdp
