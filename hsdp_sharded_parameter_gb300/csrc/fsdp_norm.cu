// Layer norm with the residual addition and dropout ahead of it, and its
// gradient.
//
// Forward: h = residual + drop(x), out = (h - mean) * rstd * weight + bias.
// A group of warps holds a row of h in registers, so mean and variance are
// two sums over registers and the variance is that of h - mean (a large mean
// costs no digits).
//
// Gradient: with g = grad_out * weight and u = (h - mean) * rstd,
//   t = rstd * (g - mean(g) - u * mean(g * u)) + grad_hidden,
// and each thread keeps its columns' sums of grad_out * u and grad_out over
// the rows its group takes; a second kernel adds the blocks' sums.
//
// Rows in registers: V granules of 8 columns a thread, gw warps a row, blocks
// that take rows in turn. Each warp copies its spans of the next rows' inputs
// into shared memory, `depth` rows ahead, so that the loads in flight do not
// depend on how many warps fit beside the row's registers.
#include "fsdp_ops.cuh"

namespace fsdp {
namespace {

constexpr int kWarps = 16;  // largest block
constexpr int kWideThreads = 512;
constexpr int kNormCols = kWarps * 4 * kSpan;  // widest row kept in registers

// Sums N values over a row's group of gw warps; warp is the one inside the
// group. Every thread of the block takes part (groups of one warp need no
// barrier). slot alternates between calls, so one barrier a call is enough.
template <int N>
__device__ __forceinline__ void group_sum(float (&x)[N], int gw, int group, int warp, int lane, int slot) {
    __shared__ float part[2][N][kWarps];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = warp_sum(x[i]);
    if (gw == 1) return;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) part[slot][i][group * gw + warp] = x[i];
    __syncthreads();
    // every warp adds the group's parts, at most 16, in the same order
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = (lane & 15) < gw ? part[slot][i][group * gw + (lane & 15)] : 0.0f;
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
        x[i] = s;
    }
}

// A parameter's granule, every row's again: it stays in the L1 cache, and held
// in registers it would cost half the warps.
template <bool kAligned, typename P>
__device__ __forceinline__ Cols load_param_as(const void* p, int64_t c, int n) {
    Raw<P> r;
    if constexpr (kAligned) {
        if (n) {
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const P*>(p) + c);
#pragma unroll
            for (int v = 0; v < Raw<P>::kVec; ++v) put(r.w + 4 * v, ld_reuse(q + v));
        }
    } else {
        load_granule(r, static_cast<const P*>(p), c, n);
    }
    return widened(r);
}
template <bool kAligned>
__device__ __forceinline__ Cols load_param(const void* p, int dt, int64_t c, int n, float none) {
    if (!p) return all(none);
    return dt == FSDP_F32 ? load_param_as<kAligned, float>(p, c, n) : load_param_as<kAligned, uint16_t>(p, c, n);
}

// Granule g of a parameter on the 16-byte grid in two steps: its first block,
// all of it in bf16, and what makes it whole.
__device__ __forceinline__ const uint4* param_block(const void* p, int dt, int g) {
    return reinterpret_cast<const uint4*>(p) + (dt == FSDP_F32 ? 2 * g : g);
}
__device__ __forceinline__ Cols param_after(uint4 first, const void* p, int dt, int g, int n) {
    if (dt != FSDP_F32) {
        Raw<uint16_t> r;
        put(r.w, first);
        return widened(r);
    }
    Raw<float> r;
    put(r.w, first);
    if (n) put(r.w + 4, ld_reuse(param_block(p, dt, g) + 1));
    return widened(r);
}

// What h is made of, and what its gradient takes: a kernel's kMode holds
// kResidual (a residual; a gradient past the norm) and kDrops as bits, or
// leaves both to the call (kEither).
constexpr int kResidual = 1, kDrops = 2, kEither = -1;
template <int kMode>
__device__ __forceinline__ bool has(int bit, bool given) {
    return kMode == kEither ? given : (kMode & bit) != 0;
}

// Waits until all but the newest `left` groups of this thread's copies are in.
__device__ __forceinline__ void async_wait_but(int left) {
    if (left == 3)
        async_wait<3>();
    else if (left == 2)
        async_wait<2>();
    else if (left == 1)
        async_wait<1>();
    else
        async_wait<0>();
}

// ------------------------------------------------------------------ forward

template <int kMode, typename T>
__device__ __forceinline__ Cols make_hidden(const Raw<T>& x, const Raw<T>& res, const NormArgs& a, int64_t row,
                                            int64_t g) {
    Cols h = has<kMode>(kResidual, a.res.data) ? widened(res) : all(0.0f);
    if (has<kMode>(kDrops, a.mask.drops))
        add_dropped(h, widened(x), a.mask, row, (uint32_t)g);
    else
        h = has<kMode>(kResidual, a.res.data) ? h + widened(x) : widened(x);
    return h;
}

template <typename T, int V, bool kAligned, int kMode>
__global__ void __launch_bounds__(V == 2 ? 256 : (V == 1 ? 128 : 512), V == 2 ? 4 : (V == 1 ? 8 : 1))
    norm_kernel(NormArgs a, int gw, int depth) {
    extern __shared__ uint4 ring[];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, group = w / gw, warp = w - group * gw;
    const int groups = (blockDim.x >> 5) / gw, streams = has<kMode>(kResidual, a.res.data) ? 2 : 1;
    const uint32_t rows = (uint32_t)a.rows, step = gridDim.x * groups;
    const uint32_t xs = (uint32_t)a.x.stride * sizeof(T), rs = (uint32_t)a.res.stride * sizeof(T);
    const uint32_t hs = (uint32_t)a.hidden.stride * sizeof(T), os = (uint32_t)a.out.stride * sizeof(T);
    uint4* const mine = ring + (size_t)w * depth * streams * V * kSlot<kAligned, T>;
    const int cols = (int)a.cols;
    const float inv = 1.0f / (float)cols;

    auto fetch = [&](uint32_t row, int slot) {
        if (row < rows) {
            uint4* s = mine + slot * streams * V * kSlot<kAligned, T>;
            const T* x = row_at<const T>(a.x.data, row, xs);
            const T* res = row_at<const T>(a.res.data, row, rs);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c0 = (v * gw + warp) * kSpan;
                span_fetch<kAligned>(s + v * kSlot<kAligned, T>, x, c0, cols, lane);
                if (has<kMode>(kResidual, a.res.data)) span_fetch<kAligned>(s + (V + v) * kSlot<kAligned, T>, res, c0, cols, lane);
            }
        }
        async_commit();
    };

    uint32_t row = blockIdx.x * groups + group;
    for (int d = 0; d + 1 < depth; ++d) fetch(row + d * step, d);
    int slot = 0;
    // every group of a block goes round as often, for the barriers
    for (uint32_t r0 = blockIdx.x * groups; r0 < rows; r0 += step, row += step) {
        __syncwarp();  // the slot's last reads
        fetch(row + (depth - 1) * step, slot == 0 ? depth - 1 : slot - 1);
        async_wait_but(depth - 1);
        __syncwarp();
        const bool on = row < rows;
        const T* x = row_at<const T>(a.x.data, row, xs);
        const T* res = row_at<const T>(a.res.data, row, rs);
        Cols h[V];
        float2 s = both(0.0f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int g = (v * gw + warp) * 32 + lane, c0 = (v * gw + warp) * kSpan;
            const int n = on ? granule_cols(g, cols) : 0;
            const uint4* from = mine + (slot * streams * V + v) * kSlot<kAligned, T>;
            Raw<T> r, q;
            span_read<kAligned>(r, from, x, c0, lane);
            if (has<kMode>(kResidual, a.res.data)) span_read<kAligned>(q, from + V * kSlot<kAligned, T>, res, c0, lane);
            h[v] = make_hidden<kMode>(r, q, a, row, g);
            if (a.hidden.data) {
                round_to(h[v], r);
                store_cols<kAligned>(row_at<T>(a.hidden.data, row, hs) + g * kGran, r, n, lane);
            }
            if (!kAligned) cut(h[v], n);
            if (!kAligned || n) sum_into(s, h[v]);
        }
        float sum[1] = {s.x + s.y};
        group_sum(sum, gw, group, warp, lane, 0);
        // one rounding: where the sum of equal values is exact (few bits, or few
        // columns) they give their own, which a product with 1 / cols may not;
        // else their mean is off by the sum's roundings
        const float mean = sum[0] / (float)cols;
        s = both(0.0f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int n = on ? granule_cols((v * gw + warp) * 32 + lane, cols) : 0;
            h[v] = h[v] + all(-mean);
            if (!kAligned) cut(h[v], n);
            if (!kAligned || n) dot_into(s, h[v], h[v]);
        }
        sum[0] = s.x + s.y;
        // the weight's loads run while the group meets (without: 179 us for
        // 16384 rows of 8192, with: 171)
        uint4 ahead[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int g = (v * gw + warp) * 32 + lane;
            if (kAligned && a.weight && g * kGran < cols) ahead[v] = ld_reuse(param_block(a.weight, a.param_dt, g));
        }
        group_sum(sum, gw, group, warp, lane, 1);
        slot = slot + 1 == depth ? 0 : slot + 1;
        if (!on) continue;
        const float rstd = rsqrtf(__fmaf_rn(sum[0], inv, a.eps));
        if (warp == 0 && lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int g = (v * gw + warp) * 32 + lane;
            const int n = granule_cols(g, cols);
            Raw<T> r;
            const Cols wt = kAligned && a.weight ? param_after(ahead[v], a.weight, a.param_dt, g, n)
                                                 : load_param<kAligned>(a.weight, a.param_dt, g * kGran, n, 1.0f);
            round_to(fma(h[v] * all(rstd), wt, load_param<kAligned>(a.bias, a.param_dt, g * kGran, n, 0.0f)), r);
            store_cols<kAligned>(row_at<T>(a.out.data, row, os) + g * kGran, r, n, lane);
        }
    }
}

// The columns of granule g of h, straight from memory.
template <typename T>
__device__ __forceinline__ Cols load_hidden(const NormArgs& a, int64_t row, int64_t g, int n) {
    Raw<T> r, q;
    load_granule(r, static_cast<const T*>(a.x.data) + row * a.x.stride, g * kGran, n);
    if (a.res.data) load_granule(q, static_cast<const T*>(a.res.data) + row * a.res.stride, g * kGran, n);
    Cols h = make_hidden<kEither>(r, q, a, row, g);
    cut(h, n);
    return h;
}

// Rows too wide for registers, or too far apart for 32-bit strides: a block
// reads the row's inputs once for each of the mean, the variance and the
// output.
template <typename T>
__global__ void __launch_bounds__(kWideThreads) norm_wide_kernel(NormArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gw = kWideThreads / 32;
    const int64_t row = blockIdx.x, end = (a.cols + kSpan - 1) / kSpan * 32;
    float sum[1] = {0.0f};
    for (int64_t g = threadIdx.x; g < end; g += kWideThreads) {
        float2 s = both(0.0f);
        sum_into(s, load_hidden<T>(a, row, g, granule_cols(g, a.cols)));
        sum[0] += s.x + s.y;
    }
    group_sum(sum, gw, 0, warp, lane, 0);
    const float mean = sum[0] / (float)a.cols;
    sum[0] = 0.0f;
    for (int64_t g = threadIdx.x; g < end; g += kWideThreads) {
        const int n = granule_cols(g, a.cols);
        Cols d = load_hidden<T>(a, row, g, n) + all(-mean);
        cut(d, n);
        float2 s = both(0.0f);
        dot_into(s, d, d);
        sum[0] += s.x + s.y;
    }
    group_sum(sum, gw, 0, warp, lane, 1);
    const float rstd = rsqrtf(sum[0] / (float)a.cols + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    for (int64_t g = threadIdx.x; g < end; g += kWideThreads) {
        const int n = granule_cols(g, a.cols);
        const Cols h = load_hidden<T>(a, row, g, n);
        Raw<T> r;
        if (a.hidden.data) {
            round_to(h, r);
            store_span(static_cast<T*>(a.hidden.data) + row * a.hidden.stride + g * kGran, r, n, lane);
        }
        round_to(fma((h + all(-mean)) * all(rstd), load_param<false>(a.weight, a.param_dt, g * kGran, n, 1.0f),
                     load_param<false>(a.bias, a.param_dt, g * kGran, n, 0.0f)),
                 r);
        store_span(static_cast<T*>(a.out.data) + row * a.out.stride + g * kGran, r, n, lane);
    }
}

// ----------------------------------------------------------------- gradient

// grad_hidden's share and the dropout behind it, rounded and stored. (What t
// holds past the row's end is not stored.)
template <bool kAligned, int kMode, typename T>
__device__ __forceinline__ void store_grad(const NormGradArgs& a, const Cols& t, int64_t row, int64_t g, int n, int lane,
                                           T* grad_res, T* grad_x) {
    Raw<T> r;
    round_to(t, r);
    if (a.grad_res.data) store_cols<kAligned>(grad_res + g * kGran, r, n, lane);
    if (has<kMode>(kDrops, a.mask.drops)) {
        Cols y = all(0.0f);
        add_dropped(y, t, a.mask, row, (uint32_t)g);
        round_to(y, r);
    }
    store_cols<kAligned>(grad_x + g * kGran, r, n, lane);
}

// Two sums of a row over its group's warps, in two steps with one barrier of
// the block between them. Lanes 0 to 15 work on the first value, the others on
// the second.
__device__ __forceinline__ float pair_begin(float a, float b, int lane, float* part) {
    float v = lane < 16 ? a : b;
    v += __shfl_xor_sync(kFull, lane < 16 ? b : a, 16);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    if ((lane & 15) == 0) part[lane] = v;  // lane 0: the first sum, lane 16: the second
    return v;
}
__device__ __forceinline__ float2 pair_end(float v, int gw, int lane, const float* part) {
    if (gw > 1) {
        v = (lane & 15) < gw ? part[(lane & 15) * 32 + (lane & 16)] : 0.0f;
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    }
    return make_float2(__shfl_sync(kFull, v, 0), __shfl_sync(kFull, v, 16));
}

// parts[block][0 weight, 1 bias][stride]: the sums of a block's rows. A row is
// read twice from shared memory: for its two sums, and, an iteration later,
// for its gradient. One barrier an iteration, and between two of them the one
// row's gradient and the next one's sums, which do not depend on each other:
// with the gradient right behind its sums, the 16 warps that the columns'
// sums leave room for waited for each other (16384 rows of 8192: 327 us, now 232).
template <typename T, int V, bool kAligned, int kMode>
__global__ void __launch_bounds__(32 * kWarps, V == 1 ? 2 : 1)
    norm_grad_kernel(NormGradArgs a, int gw, int depth, int64_t stride) {
    extern __shared__ uint4 ring[];
    __shared__ float part[2][kWarps * 32];
    allow_next();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, group = w / gw, warp = w - group * gw;
    const int groups = (blockDim.x >> 5) / gw, streams = has<kMode>(kResidual, a.grad_hidden.data) ? 3 : 2;
    const uint32_t rows = (uint32_t)a.rows, step = gridDim.x * groups;
    const uint32_t gs = (uint32_t)a.grad.stride * sizeof(T), hs = (uint32_t)a.hidden.stride * sizeof(T);
    const uint32_t as = (uint32_t)a.grad_hidden.stride * sizeof(T);
    const uint32_t rs = (uint32_t)a.grad_res.stride * sizeof(T), xs = (uint32_t)a.grad_x.stride * sizeof(T);
    constexpr int kOne = kSlot<kAligned, T>;
    constexpr bool kHold = V <= 2;  // the weight in registers
    uint4* const mine = ring + (size_t)w * depth * streams * V * kOne;
    const int cols = (int)a.cols;
    const float inv = 1.0f / (float)cols;

    auto fetch = [&](uint32_t row, int slot) {
        if (row < rows) {
            uint4* s = mine + slot * streams * V * kOne;
            const T* dy = row_at<const T>(a.grad.data, row, gs);
            const T* h = row_at<const T>(a.hidden.data, row, hs);
            const T* past = row_at<const T>(a.grad_hidden.data, row, as);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c0 = (v * gw + warp) * kSpan;
                span_fetch<kAligned>(s + v * kOne, dy, c0, cols, lane);
                span_fetch<kAligned>(s + (V + v) * kOne, h, c0, cols, lane);
                if (has<kMode>(kResidual, a.grad_hidden.data)) span_fetch<kAligned>(s + (2 * V + v) * kOne, past, c0, cols, lane);
            }
        }
        async_commit();
    };

    Cols dw[V], db[V], held[kHold ? V : 1];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int g = (v * gw + warp) * 32 + lane;
        dw[v] = db[v] = all(0.0f);
        if (kHold) held[kHold ? v : 0] = load_param<kAligned>(a.weight, a.param_dt, g * kGran, granule_cols(g, cols), 1.0f);
    }
    auto weight = [&](int v, int g, int n) {
        return kHold ? held[kHold ? v : 0] : load_param<kAligned>(a.weight, a.param_dt, g * kGran, n, 1.0f);
    };
    // grad_out and u of a granule of a row that has arrived
    auto read = [&](int v, int slot, uint32_t row, float mean, float rstd, int n, Cols& dy, Cols& u) {
        const int c0 = (v * gw + warp) * kSpan;
        const uint4* from = mine + slot * streams * V * kOne;
        Raw<T> r, q;
        span_read<kAligned>(r, from + v * kOne, row_at<const T>(a.grad.data, row, gs), c0, lane);
        span_read<kAligned>(q, from + (V + v) * kOne, row_at<const T>(a.hidden.data, row, hs), c0, lane);
        dy = widened(r);
        u = (widened(q) + all(-mean)) * all(rstd);
        if (!kAligned) {
            cut(dy, n);
            cut(u, n);
        }
    };
    auto sums = [&](uint32_t row, int slot, float mean, float rstd, float* to) {
        float2 s1 = both(0.0f), s2 = both(0.0f);
        if (row < rows)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int g = (v * gw + warp) * 32 + lane, n = granule_cols(g, cols);
                Cols dy, u;
                read(v, slot, row, mean, rstd, n, dy, u);
                if (kAligned && !n) continue;
                const Cols gr = dy * weight(v, g, n);
                sum_into(s1, gr);
                dot_into(s2, gr, u);
            }
        return pair_begin(s1.x + s1.y, s2.x + s2.y, lane, to);
    };

    uint32_t row = blockIdx.x * groups + group;
    for (int d = 0; d + 1 < depth; ++d) fetch(row + d * step, d);
    float mean = row < rows ? __ldg(a.mean + row) : 0.0f, rstd = row < rows ? __ldg(a.rstd + row) : 0.0f;
    // a row's mean and rstd are loaded a row ahead
    float next_mean = row + step < rows ? __ldg(a.mean + row + step) : 0.0f;
    float next_rstd = row + step < rows ? __ldg(a.rstd + row + step) : 0.0f;
    async_wait_but(depth - 2);
    __syncwarp();
    float sum = sums(row, 0, mean, rstd, &part[0][w * 32]);
    int slot = 0, side = 0;
    for (; row < rows; row += step) {
        __syncwarp();  // the last reads of the slot that is filled now
        fetch(row + (depth - 1) * step, slot == 0 ? depth - 1 : slot - 1);
        async_wait_but(depth - 2);
        if (groups == 1)
            __syncthreads();
        else if (gw > 1)  // the group's own barrier
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(gw * 32) : "memory");
        else
            __syncwarp();
        const float2 c = pair_end(sum, gw, lane, &part[side][group * gw * 32]);
        const int after = slot + 1 == depth ? 0 : slot + 1;
        float m = 0.0f, r = 0.0f;
        if (row + 2 * step < rows) {
            m = __ldg(a.mean + row + 2 * step);
            r = __ldg(a.rstd + row + 2 * step);
        }
        sum = sums(row + step, after, next_mean, next_rstd, &part[side ^ 1][w * 32]);
        const Cols k0 = all(rstd), k1 = all(-(c.x * inv)), k2 = all(-(c.y * inv));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int g = (v * gw + warp) * 32 + lane, c0 = (v * gw + warp) * kSpan, n = granule_cols(g, cols);
            Cols dy, u;
            read(v, slot, row, mean, rstd, n, dy, u);
            if (!kAligned || n) {
                db[v] = db[v] + dy;
                dw[v] = fma(dy, u, dw[v]);
            }
            Cols t = fma(u, k2, fma(dy, weight(v, g, n), k1));
            if (has<kMode>(kResidual, a.grad_hidden.data)) {
                Raw<T> q;
                span_read<kAligned>(q, mine + (slot * streams * V + 2 * V + v) * kOne, row_at<const T>(a.grad_hidden.data, row, as), c0, lane);
                t = fma(t, k0, widened(q));
            } else {
                t = t * k0;
            }
            store_grad<kAligned, kMode>(a, t, row, g, n, lane, row_at<T>(a.grad_res.data, row, rs), row_at<T>(a.grad_x.data, row, xs));
        }
        mean = next_mean;
        rstd = next_rstd;
        next_mean = m;
        next_rstd = r;
        slot = after;
        side ^= 1;
    }
    // the block's groups, added in turn
    float4* const box = reinterpret_cast<float4*>(ring);
    for (int k = 1; k < groups; ++k) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float4* q = box + ((v * 4 + i) * gw + warp) * 32 + lane;
                if (group == k) *q = make_float4(dw[v].p[i].x, dw[v].p[i].y, db[v].p[i].x, db[v].p[i].y);
            }
        __syncthreads();
        if (group == 0)
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 q = box[((v * 4 + i) * gw + warp) * 32 + lane];
                    dw[v].p[i] = __fadd2_rn(dw[v].p[i], make_float2(q.x, q.y));
                    db[v].p[i] = __fadd2_rn(db[v].p[i], make_float2(q.z, q.w));
                }
    }
    if (group != 0) return;
    float* const p = a.work + (int64_t)blockIdx.x * 2 * stride;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = ((v * gw + warp) * 32 + lane) * kGran;
        if (c >= cols) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            *reinterpret_cast<float2*>(p + c + 2 * i) = dw[v].p[i];
            *reinterpret_cast<float2*>(p + stride + c + 2 * i) = db[v].p[i];
        }
    }
}

// What a row's gradient needs at one granule, straight from memory.
template <typename T>
__device__ __forceinline__ void load_grad(const NormGradArgs& a, float mean, float rstd, int64_t row, int64_t g, int n,
                                          Cols& dy, Cols& u, Cols& gr) {
    Raw<T> r, q;
    load_granule(r, static_cast<const T*>(a.grad.data) + row * a.grad.stride, g * kGran, n);
    load_granule(q, static_cast<const T*>(a.hidden.data) + row * a.hidden.stride, g * kGran, n);
    dy = widened(r);
    u = (widened(q) + all(-mean)) * all(rstd);
    cut(u, n);
    gr = dy * load_param<false>(a.weight, a.param_dt, g * kGran, n, 1.0f);
}

// Rows too wide for registers, or too far apart for 32-bit strides: the rows'
// gradients, a block each ...
template <typename T>
__global__ void __launch_bounds__(kWideThreads) norm_grad_wide_kernel(NormGradArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gw = kWideThreads / 32;
    const int64_t row = blockIdx.x, end = (a.cols + kSpan - 1) / kSpan * 32;
    const float mean = __ldg(a.mean + row), rstd = __ldg(a.rstd + row);
    Cols dy, u, gr;
    float c[2] = {0.0f, 0.0f};
    for (int64_t g = threadIdx.x; g < end; g += kWideThreads) {
        load_grad<T>(a, mean, rstd, row, g, granule_cols(g, a.cols), dy, u, gr);
        float2 s1 = both(0.0f), s2 = both(0.0f);
        sum_into(s1, gr);
        dot_into(s2, gr, u);
        c[0] += s1.x + s1.y;
        c[1] += s2.x + s2.y;
    }
    group_sum(c, gw, 0, warp, lane, 0);
    const Cols k1 = all(-(c[0] / (float)a.cols)), k2 = all(-(c[1] / (float)a.cols));
    for (int64_t g = threadIdx.x; g < end; g += kWideThreads) {
        const int n = granule_cols(g, a.cols);
        load_grad<T>(a, mean, rstd, row, g, n, dy, u, gr);
        Cols t = fma(u, k2, gr + k1) * all(rstd);
        if (a.grad_hidden.data) {
            Raw<T> r;
            load_granule(r, static_cast<const T*>(a.grad_hidden.data) + row * a.grad_hidden.stride, g * kGran, n);
            t = t + widened(r);
        }
        store_grad<false, kEither>(a, t, row, g, n, lane, static_cast<T*>(a.grad_res.data) + row * a.grad_res.stride,
                                   static_cast<T*>(a.grad_x.data) + row * a.grad_x.stride);
    }
}
// ... and the weight's and bias's sums, a warp for a span of columns and a
// share of the rows.
template <typename T>
__global__ void __launch_bounds__(256) norm_param_kernel(NormGradArgs a, int64_t stride, int parts) {
    const int lane = threadIdx.x & 31, part = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int64_t g = (int64_t)blockIdx.x * 32 + lane, c = g * kGran;
    const int n = granule_cols(g, a.cols);
    if (part >= parts || n == 0) return;
    Cols dw = all(0.0f), db = all(0.0f);
    for (int64_t row = part; row < a.rows; row += parts) {
        Cols dy, u, gr;
        load_grad<T>(a, __ldg(a.mean + row), __ldg(a.rstd + row), row, g, n, dy, u, gr);
        db = db + dy;
        dw = fma(dy, u, dw);
    }
    float* p = a.work + (int64_t)part * 2 * stride + c;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        p[e] = dw.get(e);
        p[stride + e] = db.get(e);
    }
}

// Adds the parts' sums, 32 columns a block, a share of the parts for each of
// its warps: blockIdx.y 0 the weight's, 1 the bias's.
template <typename G>
__global__ void __launch_bounds__(1024)
    norm_join_kernel(const float* work, int64_t stride, int parts, int64_t cols, int accumulate, G* gw, G* gb) {
    __shared__ float sums[32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    G* out = blockIdx.y ? gb : gw;
    wait_for_previous();
    if (!out) return;
    float s = 0.0f;
    if (c < cols) {
        const float* from = work + blockIdx.y * stride + c;
#pragma unroll 8
        for (int p = parts * warp / warps; p < parts * (warp + 1) / warps; ++p) s += __ldcg(from + 2 * (int64_t)p * stride);
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || c >= cols) return;
    s = 0.0f;
    for (int q = 0; q < warps; ++q) s += sums[q][lane];
    if (accumulate) s += load_f32(out, c);
    store_f32(out, c, s);
}

// ----------------------------------------------------------------- launches

// Whether the rows' strides and numbers fit the 32-bit arithmetic of the
// kernels that keep rows in registers.
bool fits_32(const Mat& m, int es) { return m.stride < ((int64_t)1 << 32) / es; }

// What the blocks of an SM may take of shared memory together: the rest of
// its 256 KB is the L1 cache, where the parameters stay.
constexpr int64_t kSmemPerSm = 132 * 1024, kSmemMost = 200 * 1024;

// How a kernel is launched on rows of these columns: V granules a thread, gw
// warps a row, groups of them in a block, blocks of an SM, and the rows that
// its shared memory holds.
struct Shape {
    int v, gw, groups, per_sm, grid, depth;
    int64_t smem;
};

Shape norm_shape(int64_t rows, int64_t cols, int streams, int slot_bytes) {
    Shape f;
    const int64_t grans = (cols + kGran - 1) / kGran;
    // few warps a row make its two sums cheap: 16384 rows of bf16 with dropout
    // and residual take 31 us at 1024 columns with 2 granules a thread and 34
    // with 1, 91 at 4096 with 4 and 114 with 2, 166 at 8192 with 4 and 219
    // with 2. Rows that do not fill the GPU are done sooner by more warps (16
    // of 4096 columns: 3.4 us with 2 granules, 4.2 with 4).
    const int spans = (int)((cols + kSpan - 1) / kSpan);
    const bool few = rows <= 2 * (int64_t)sm_count();
    f.v = spans <= (few ? 4 : 1) ? 1 : (spans <= (few ? 16 : 8) ? 2 : 4);
    f.gw = (int)((grans + 32 * f.v - 1) / (32 * f.v));
    f.groups = f.gw >= 4 ? 1 : 4 / f.gw;
    const int block = 32 * f.gw * f.groups;
    f.per_sm = f.v <= 2 ? 1024 / block : (512 / block);
    const int64_t need = (rows + f.groups - 1) / f.groups;
    const int64_t most = (int64_t)sm_count() * f.per_sm;
    f.grid = (int)(need < most ? need : most);
    const int64_t stage = (int64_t)f.gw * f.groups * f.v * slot_bytes * streams;
    int64_t depth = kSmemPerSm / f.per_sm / stage;
    if (depth > 4) depth = 4;
    if (depth > (need + f.grid - 1) / f.grid) depth = (need + f.grid - 1) / f.grid;
    f.depth = (int)(depth > 1 ? depth : 1);
    f.smem = stage * f.depth;
    return f;
}

template <typename T, int V, bool kAligned, int kMode>
cudaError_t norm_rows(const NormArgs& a, const Shape& f, cudaStream_t s) {
    auto kernel = norm_kernel<T, V, kAligned, kMode>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), (int)kSmemMost, done);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)f.grid, 32 * f.gw * f.groups, f.smem, s>>>(a, f.gw, f.depth);
    return cudaGetLastError();
}
template <typename T, bool kAligned, int kMode>
cudaError_t norm_v(const NormArgs& a, const Shape& f, cudaStream_t s) {
    return f.v == 1 ? norm_rows<T, 1, kAligned, kMode>(a, f, s)
           : f.v == 2 ? norm_rows<T, 2, kAligned, kMode>(a, f, s) : norm_rows<T, 4, kAligned, kMode>(a, f, s);
}

template <typename T>
cudaError_t norm(const NormArgs& a, cudaStream_t s) {
    const int es = (int)sizeof(T);
    if (a.cols > kNormCols || !fits_32(a.x, es) || !fits_32(a.res, es) || !fits_32(a.hidden, es) || !fits_32(a.out, es)) {
        norm_wide_kernel<T><<<(unsigned)a.rows, kWideThreads, 0, s>>>(a);
        return cudaGetLastError();
    }
    const bool aligned = a.cols % kGran == 0 && on_grid(a.x, es) && on_grid(a.res, es) && on_grid(a.hidden, es) &&
                         on_grid(a.out, es) && on_grid(Mat{const_cast<void*>(a.weight), 0}, es) &&
                         on_grid(Mat{const_cast<void*>(a.bias), 0}, es);
    const int mode = (a.res.data ? kResidual : 0) | (a.mask.drops ? kDrops : 0);
    const Shape f = norm_shape(a.rows, a.cols, a.res.data ? 2 : 1, 16 * (aligned ? kSlot<true, T> : kSlot<false, T>));
    if (!aligned) return norm_v<T, false, kEither>(a, f, s);
    switch (mode) {
        case 0: return norm_v<T, true, 0>(a, f, s);
        case kResidual: return norm_v<T, true, kResidual>(a, f, s);
        case kDrops: return norm_v<T, true, kDrops>(a, f, s);
        default: return norm_v<T, true, kResidual | kDrops>(a, f, s);
    }
}

// cols <= kNormCols: a wider row would take more warps than a block has.
Shape grad_shape(int64_t rows, int64_t cols, int streams, int slot_bytes) {
    Shape f;
    // 2 granules a thread where they will do: with 3 or 4 the weight has to be
    // loaded again for every row (16384 rows of 6144 bf16: 135 us with 2, 12
    // warps and the fourth quarter of the SM's idle, 193 with 3 and all 16)
    const int spans = (int)((cols + kSpan - 1) / kSpan);
    f.v = spans <= 1 ? 1 : (spans <= 2 * kWarps ? 2 : (spans <= 3 * kWarps ? 3 : 4));
    f.gw = (spans + f.v - 1) / f.v;
    // a block takes as many rows at a time as it has warps for, and as there
    // are rows for all SMs: the fewer blocks, the fewer sums to add in the end
    const int64_t most_groups = kWarps / f.gw, share = (rows + sm_count() - 1) / sm_count();
    f.groups = (int)(share < most_groups ? share : most_groups);
    f.per_sm = f.v == 1 ? 2 : 1;
    const int64_t need = (rows + f.groups - 1) / f.groups;
    const int64_t most = (int64_t)sm_count() * f.per_sm;
    f.grid = (int)(need < most ? need : most);
    const int64_t stage = (int64_t)f.gw * f.groups * f.v * slot_bytes * streams;
    // two rows at least: a row's gradient beside the next one's sums
    int64_t depth = kSmemMost / f.per_sm / stage;
    if (depth > 4) depth = 4;
    if (depth > (need + f.grid - 1) / f.grid) depth = (need + f.grid - 1) / f.grid;
    f.depth = (int)(depth > 2 ? depth : 2);
    f.smem = stage * f.depth;
    const int64_t box = f.groups > 1 ? (int64_t)f.gw * f.v * 2048 : 0;  // where the groups meet
    if (f.smem < box) f.smem = box;
    return f;
}

template <typename T, int V, bool kAligned, int kMode>
cudaError_t grad_rows(const NormGradArgs& a, const Shape& f, int64_t stride, cudaStream_t s) {
    auto kernel = norm_grad_kernel<T, V, kAligned, kMode>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), (int)kSmemMost, done);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)f.grid, 32 * f.gw * f.groups, f.smem, s>>>(a, f.gw, f.depth, stride);
    return cudaGetLastError();
}
template <typename T, bool kAligned, int kMode>
cudaError_t grad_v(const NormGradArgs& a, const Shape& f, int64_t stride, cudaStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (f.v == 4) return grad_rows<T, 4, kAligned, kMode>(a, f, stride, s);
    } else {
        // rows of 4 granules a thread, 13 warps and more, are among the wide ones
        static_assert((int64_t)13 * 4 * 16 * kSlot<true, T> * 2 * 2 > kSmemMost, "two rows do not fit");
    }
    return f.v == 1 ? grad_rows<T, 1, kAligned, kMode>(a, f, stride, s)
           : f.v == 2 ? grad_rows<T, 2, kAligned, kMode>(a, f, stride, s) : grad_rows<T, 3, kAligned, kMode>(a, f, stride, s);
}

constexpr int kWideParts = 256;
int64_t grad_stride(int64_t cols) { return (cols + kGran - 1) / kGran * kGran; }

// The rows' gradients and the parts' sums; *parts is how many there are.
template <typename T>
cudaError_t norm_grad(const NormGradArgs& a, int* parts, cudaStream_t s) {
    const int es = (int)sizeof(T);
    const int64_t stride = grad_stride(a.cols);
    const bool aligned = a.cols % kGran == 0 && on_grid(a.grad, es) && on_grid(a.hidden, es) && on_grid(a.grad_hidden, es) &&
                         on_grid(a.grad_res, es) && on_grid(a.grad_x, es) && on_grid(Mat{const_cast<void*>(a.weight), 0}, es);
    const int mode = (a.grad_hidden.data ? kResidual : 0) | (a.mask.drops ? kDrops : 0);
    bool wide = a.cols > kNormCols || !fits_32(a.grad, es) || !fits_32(a.hidden, es) || !fits_32(a.grad_hidden, es) ||
                !fits_32(a.grad_res, es) || !fits_32(a.grad_x, es);
    Shape f = {};
    if (!wide) {
        f = grad_shape(a.rows, a.cols, a.grad_hidden.data ? 3 : 2, 16 * (aligned ? kSlot<true, T> : kSlot<false, T>));
        wide = f.smem > kSmemMost;  // fp32 rows of more than about 8192 columns do not fit shared memory twice
    }
    if (wide) {
        norm_grad_wide_kernel<T><<<(unsigned)a.rows, kWideThreads, 0, s>>>(a);
        count_launch();
        *parts = (int)(a.rows < kWideParts ? a.rows : kWideParts);
        norm_param_kernel<T><<<dim3((unsigned)((a.cols + kSpan - 1) / kSpan), (unsigned)((*parts + 7) / 8)), 256, 0, s>>>(a, stride, *parts);
        count_launch();
        return cudaGetLastError();
    }
    *parts = f.grid;
    count_launch();
    if (!aligned) return grad_v<T, false, kEither>(a, f, stride, s);
    switch (mode) {
        case 0: return grad_v<T, true, 0>(a, f, stride, s);
        case kResidual: return grad_v<T, true, kResidual>(a, f, stride, s);
        case kDrops: return grad_v<T, true, kDrops>(a, f, stride, s);
        default: return grad_v<T, true, kResidual | kDrops>(a, f, stride, s);
    }
}

}  // namespace

size_t norm_grad_bytes(int64_t rows, int64_t cols) {
    if (rows == 0 || cols == 0) return 0;
    // parts: a block's each, or the wide rows' shares
    int64_t parts = rows < kWideParts ? rows : kWideParts;
    if (cols <= kNormCols) {
        const int64_t grid = grad_shape(rows, cols, 2, 16).grid;
        if (grid > parts) parts = grid;
    }
    return (size_t)parts * 2 * grad_stride(cols) * 4;
}

cudaError_t launch_norm(int dt, const NormArgs& a, cudaStream_t s) {
    if (a.rows == 0 || a.cols == 0) return cudaSuccess;
    const cudaError_t e = dt == FSDP_F32 ? norm<float>(a, s) : norm<uint16_t>(a, s);
    count_launch();
    return e;
}

cudaError_t launch_norm_grad(int dt, int param_grad_dt, const NormGradArgs& a, cudaStream_t s) {
    if (a.cols == 0) return cudaSuccess;
    int parts = 0;
    if (a.rows > 0) {
        const cudaError_t e = dt == FSDP_F32 ? norm_grad<float>(a, &parts, s) : norm_grad<uint16_t>(a, &parts, s);
        if (e != cudaSuccess) return e;
    }
    if (!a.grad_weight && !a.grad_bias) return cudaSuccess;
    const dim3 grid((unsigned)((a.cols + 31) / 32), 2);
    const int block = grid.x < (unsigned)sm_count() ? 1024 : 512;  // many warps a block where there are few blocks
    const float* work = a.work;
    const int64_t stride = grad_stride(a.cols);
    count_launch();
    if (param_grad_dt == FSDP_F32)
        return launch_next(norm_join_kernel<float>, grid, block, 0, s, work, stride, parts, a.cols, a.accumulate,
                           static_cast<float*>(a.grad_weight), static_cast<float*>(a.grad_bias));
    return launch_next(norm_join_kernel<uint16_t>, grid, block, 0, s, work, stride, parts, a.cols, a.accumulate,
                       static_cast<uint16_t*>(a.grad_weight), static_cast<uint16_t*>(a.grad_bias));
}

}  // namespace fsdp
