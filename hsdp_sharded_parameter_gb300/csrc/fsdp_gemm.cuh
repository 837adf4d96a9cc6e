// Products of 16-bit matrices on the tensor cores, D = sum of A B^T in
// binary32, with what becomes of D's elements left to the caller (an
// epilogue). Included by the operators that need one.
#pragma once

#include <cuda_fp16.h>

#include "fsdp_ops.cuh"

namespace fsdp {
namespace {

// Element (i, k) of a factor: data[i * stride + k], or, where its rows are
// the neighbours in memory (mn), data[k * stride + i].
struct Product {
    int64_t m, n;
    int terms;     // products summed: 1 or 2
    int64_t k[2];  // their lengths
    Mat a[2], b[2];
    int a_mn, b_mn;
    int half;    // binary16 values instead of bfloat16
    int paired;  // two products with the same A and k, by b[0] and b[1], side by side
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// --------------------------------------------------- tensor core instructions

__device__ __forceinline__ void tmem_alloc(uint32_t* where, int columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t at, int columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}
// D (+)= A B^T of one step of 16 along k, by one thread.
__device__ __forceinline__ void mma_step(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, bool add) {
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a), "l"(b),
        "r"(kind), "r"((uint32_t)add)
        : "memory");
}
// Arrives on a barrier once the thread's products so far are done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t at, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
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
// one k, `block` bytes further the next 64 rows.
__device__ __forceinline__ uint64_t tile_descriptor(uint32_t at, bool mn, uint32_t block) {
    const uint64_t lead = mn ? block >> 4 : 1, step = 1024 >> 4;
    return (uint64_t)(at >> 4 & 0x3fff) | lead << 16 | step << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// ------------------------------------------------------------------ barriers

__device__ __forceinline__ void bar_init(uint64_t* b, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ bool bar_test(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
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
// Waits for the phase of a parity: false once two seconds have passed.
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity) {
    if (bar_test(b, parity)) return true;
    const uint64_t from = clock_ns();
    for (uint32_t i = 0; i < (1u << 30); ++i) {
        if (bar_test(b, parity)) return true;
        if (clock_ns() - from > kWaitNs) return false;
    }
    return false;
}

// --------------------------------------------------------------- the product

// The first form: a block of 128 threads and a tile of 128 x 128, 64 of k at a
// time, brought into shared memory by plain loads at any alignment.
constexpr int kTile = 128, kStep = 64, kTileBytes = kTile * kStep * 2;

__device__ __forceinline__ void bring(char* to, const Mat& f, int mn, int64_t r0, int64_t rows, int64_t k0, int64_t ks, int nrows,
                                      int first) {
    const uint16_t* data = static_cast<const uint16_t*>(f.data);
    for (int c = threadIdx.x; c < nrows * 8; c += blockDim.x) {
        Raw<uint16_t> v;
        zero_raw(v);
        uint32_t at;
        if (!mn) {
            const int r = c >> 3, j = c & 7;
            const int64_t left = ks - (k0 + 8 * j);
            if (r0 + r < rows && left > 0) load_granule(v, data + (r0 + r) * f.stride, k0 + 8 * j, left < 8 ? (int)left : 8);
            at = (uint32_t)(first + r) * 128 + (uint32_t)((j ^ ((first + r) & 7)) << 4);
        } else {
            const int per = nrows >> 3, kk = c / per, g = c % per, r = first + 8 * g;
            const int64_t left = rows - (r0 + 8 * g);
            if (k0 + kk < ks && left > 0) load_granule(v, data + (k0 + kk) * f.stride, r0 + 8 * g, left < 8 ? (int)left : 8);
            at = (uint32_t)(r >> 6) * (kStep * 128) + (uint32_t)kk * 128 + (uint32_t)((((r & 63) >> 3) ^ (kk & 7)) << 4);
        }
        *reinterpret_cast<uint4*>(to + at) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    }
}

template <typename Epi>
__global__ void __launch_bounds__(128) product_kernel(Product p, Epi epi, uint32_t kind) {
    extern __shared__ char raw[];
    char* base = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
    __shared__ uint64_t done;
    __shared__ uint32_t tmem;
    wait_for_previous();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (warp == 0) tmem_alloc(&tmem, kTile);
    if (threadIdx.x == 0) {
        bar_init(&done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const int width = p.paired ? kTile / 2 : kTile;
    const int64_t r0 = (int64_t)blockIdx.y * kTile, c0 = (int64_t)blockIdx.x * width;
    uint32_t phase = 0;
    bool any = false, ok = true;
    for (int t = 0; t < p.terms && ok; ++t) {
        for (int64_t k0 = 0; k0 < p.k[t] && ok; k0 += kStep) {
            bring(base, p.a[t], p.a_mn, r0, p.m, k0, p.k[t], kTile, 0);
            if (p.paired) {
                bring(base + kTileBytes, p.b[0], p.b_mn, c0, p.n, k0, p.k[t], width, 0);
                bring(base + kTileBytes, p.b[1], p.b_mn, c0, p.n, k0, p.k[t], width, width);
            } else {
                bring(base + kTileBytes, p.b[t], p.b_mn, c0, p.n, k0, p.k[t], kTile, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncthreads();
            if (threadIdx.x == 0) {
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint64_t a = tile_descriptor(smem_addr(base), p.a_mn, kStep * 128);
                const uint64_t b = tile_descriptor(smem_addr(base + kTileBytes), p.b_mn, kStep * 128);
#pragma unroll
                for (int i = 0; i < kStep / 16; ++i)
                    mma_step(tmem, a + i * (p.a_mn ? 2048 : 32) / 16, b + i * (p.b_mn ? 2048 : 32) / 16, kind, any || i > 0);
                mma_commit(&done);
            }
            any = true;
            ok = __syncthreads_and(bar_wait(&done, phase));
            phase ^= 1;
        }
    }
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (!ok) {
        if (threadIdx.x == 0) atomicOr(&gave_up, 1);
    } else {
        const int64_t row = r0 + warp * 32 + lane;
        for (int c = 0; c < width; c += 32) {
            float v[32], u[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = u[i] = 0.0f;
            if (any) {
                tmem_load32(tmem + ((uint32_t)(warp * 32) << 16) + c, v);
                if (p.paired) tmem_load32(tmem + ((uint32_t)(warp * 32) << 16) + width + c, u);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int64_t col = c0 + c + 8 * g, left = p.n - col;
                Cols x, y;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x.set(e, v[8 * g + e]);
                    y.set(e, u[8 * g + e]);
                }
                if (row < p.m && left > 0) epi(row, col, left < 8 ? (int)left : 8, x, y);
            }
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 0) tmem_free(tmem, kTile);
}

template <typename Epi>
cudaError_t launch_product(const Product& p, const Epi& epi, cudaStream_t s, bool first) {
    if (p.m == 0 || p.n == 0) return cudaSuccess;
    static std::atomic<uint64_t> done{0};
    const int smem = 2 * kTileBytes + 1024;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(product_kernel<Epi>), smem, done);
    if (e != cudaSuccess) return e;
    const int width = p.paired ? kTile / 2 : kTile;
    const dim3 grid((unsigned)((p.n + width - 1) / width), (unsigned)((p.m + kTile - 1) / kTile));
    const uint32_t kind = mma_kind(p.half, p.a_mn, p.b_mn, kTile, kTile);
    count_launch();
    if (!first) return launch_next(product_kernel<Epi>, grid, 128, smem, s, p, epi, kind);
    product_kernel<Epi><<<grid, 128, smem, s>>>(p, epi, kind);
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
