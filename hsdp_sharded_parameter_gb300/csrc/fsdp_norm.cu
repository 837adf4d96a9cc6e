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
// the rows its group takes; a second kernel adds the groups' sums.
#include "fsdp_ops.cuh"

namespace fsdp {
namespace {

constexpr int kNormThreads = 512;  // largest block
constexpr int kMaxVec = 4;         // granules of a thread
constexpr int kNormCols = kNormThreads * kMaxVec * kGran;  // widest row kept in registers

// Sums two values over a row's group of gw warps; warp is the one inside the
// group. Every thread of the block takes part (groups of one warp need no
// barrier). slot alternates between calls, so one barrier a call is enough.
__device__ __forceinline__ float2 group_sum(float a, float b, int gw, int group, int warp, int lane, int slot) {
    __shared__ float2 part[2][kNormThreads / 32];
    a = warp_sum(a);
    b = warp_sum(b);
    if (gw == 1) return make_float2(a, b);
    float2* p = part[slot] + group * gw;
    if (lane == 0) p[warp] = make_float2(a, b);
    __syncthreads();
    float2 s = p[0];
    for (int i = 1; i < gw; ++i) {
        s.x += p[i].x;
        s.y += p[i].y;
    }
    return s;
}

template <typename P>
__device__ __forceinline__ void load_param(float (&x)[8], const void* p, int64_t c, int n, float none) {
    if (!p) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = none;
        return;
    }
    Raw<P> r;
    load_granule(r, static_cast<const P*>(p), c, n);
    widen(r, x);
}

// The n columns of granule g of h = residual + drop(x).
template <typename T>
__device__ __forceinline__ void load_hidden(float (&h)[8], const NormArgs& a, int64_t row, int64_t g, int n) {
    Raw<T> r, q;
    load_granule(r, static_cast<const T*>(a.x.data) + row * a.x.stride, g * kGran, n);
    if (a.res.data) load_granule(q, static_cast<const T*>(a.res.data) + row * a.res.stride, g * kGran, n);
    widen(r, h);
    if (a.mask.limit < 65536) drop(h, a.mask, row, (uint32_t)g);
    if (a.res.data) {
        float y[8];
        widen(q, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] += y[e];
    }
}

template <typename T, typename P>
__device__ __forceinline__ void store_norm(const NormArgs& a, float (&h)[8], float mean, float rstd, int64_t row,
                                           int64_t g, int n, int lane) {
    float w[8], b[8];
    load_param<P>(w, a.weight, g * kGran, n, 1.0f);
    load_param<P>(b, a.bias, g * kGran, n, 0.0f);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = __fmaf_rn((h[e] - mean) * rstd, w[e], b[e]);
    Raw<T> r;
    narrow(h, r);
    store_span(static_cast<T*>(a.out.data) + row * a.out.stride + g * kGran, r, n, lane);
}

// Rows in registers: V granules a thread, gw warps a row.
template <typename T, typename P, int V>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(NormArgs a, int gw) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, group = w / gw, warp = w % gw;
    const int groups = (blockDim.x >> 5) / gw;
    const int64_t row = (int64_t)blockIdx.x * groups + group;
    const bool on = row < a.rows;
    float h[V][8];
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t g = (v * gw + warp) * 32 + lane;
        const int n = on ? granule_cols(g, a.cols) : 0;
        if (on) load_hidden<T>(h[v], a, row, g, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += e < n ? h[v][e] : 0.0f;
    }
    const float mean = group_sum(s, 0.0f, gw, group, warp, lane, 0).x / (float)a.cols;
    s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int n = on ? granule_cols((v * gw + warp) * 32 + lane, a.cols) : 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) s = e < n ? __fmaf_rn(h[v][e] - mean, h[v][e] - mean, s) : s;
    }
    const float var = group_sum(s, 0.0f, gw, group, warp, lane, 1).x / (float)a.cols;
    if (!on) return;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (warp == 0 && lane == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t g = (v * gw + warp) * 32 + lane;
        const int n = granule_cols(g, a.cols);
        if (a.hidden.data) {
            Raw<T> r;
            narrow(h[v], r);
            store_span(static_cast<T*>(a.hidden.data) + row * a.hidden.stride + g * kGran, r, n, lane);
        }
        store_norm<T, P>(a, h[v], mean, rstd, row, g, n, lane);
    }
}

// Rows too wide for registers: a block reads the row's inputs once for each
// of the mean, the variance and the output.
template <typename T, typename P>
__global__ void __launch_bounds__(kNormThreads) norm_wide_kernel(NormArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gw = kNormThreads / 32;
    const int64_t row = blockIdx.x, end = (a.cols + kSpan - 1) / kSpan * 32;
    float h[8], s = 0.0f;
    for (int64_t g = threadIdx.x; g < end; g += kNormThreads) {
        const int n = granule_cols(g, a.cols);
        load_hidden<T>(h, a, row, g, n);
        float t = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) t += e < n ? h[e] : 0.0f;
        s += t;
    }
    const float mean = group_sum(s, 0.0f, gw, 0, warp, lane, 0).x / (float)a.cols;
    s = 0.0f;
    for (int64_t g = threadIdx.x; g < end; g += kNormThreads) {
        const int n = granule_cols(g, a.cols);
        load_hidden<T>(h, a, row, g, n);
        float t = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) t = e < n ? __fmaf_rn(h[e] - mean, h[e] - mean, t) : t;
        s += t;
    }
    const float var = group_sum(s, 0.0f, gw, 0, warp, lane, 1).x / (float)a.cols;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    for (int64_t g = threadIdx.x; g < end; g += kNormThreads) {
        const int n = granule_cols(g, a.cols);
        load_hidden<T>(h, a, row, g, n);
        if (a.hidden.data) {
            Raw<T> r;
            narrow(h, r);
            store_span(static_cast<T*>(a.hidden.data) + row * a.hidden.stride + g * kGran, r, n, lane);
        }
        store_norm<T, P>(a, h, mean, rstd, row, g, n, lane);
    }
}

template <typename T, typename P>
cudaError_t norm(const NormArgs& a, cudaStream_t s) {
    const int64_t grans = (a.cols + kGran - 1) / kGran;
    if (a.cols > kNormCols) {
        norm_wide_kernel<T, P><<<(unsigned)a.rows, kNormThreads, 0, s>>>(a);
    } else {
        const int v = grans <= 32 * 4 ? 1 : (grans <= 32 * 16 ? 2 : 4);
        const int gw = (int)((grans + 32 * v - 1) / (32 * v));
        const int groups = gw >= 4 ? 1 : 4 / gw;
        const unsigned grid = (unsigned)((a.rows + groups - 1) / groups);
        const int block = 32 * gw * groups;
        if (v == 1)
            norm_kernel<T, P, 1><<<grid, block, 0, s>>>(a, gw);
        else if (v == 2)
            norm_kernel<T, P, 2><<<grid, block, 0, s>>>(a, gw);
        else
            norm_kernel<T, P, 4><<<grid, block, 0, s>>>(a, gw);
    }
    count_launch();
    return cudaGetLastError();
}

// ----------------------------------------------------------------- gradient

// What a row's gradient needs at one granule: the gradients and u.
template <typename T, typename P>
__device__ __forceinline__ void load_grad(const NormGradArgs& a, float mean, float rstd, int64_t row, int64_t g, int n,
                                          float (&dy)[8], float (&u)[8], float (&gw)[8]) {
    Raw<T> r, q;
    load_granule(r, static_cast<const T*>(a.grad.data) + row * a.grad.stride, g * kGran, n);
    load_granule(q, static_cast<const T*>(a.hidden.data) + row * a.hidden.stride, g * kGran, n);
    float w[8];
    load_param<P>(w, a.weight, g * kGran, n, 1.0f);
    widen(r, dy);
    widen(q, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        u[e] = e < n ? (u[e] - mean) * rstd : 0.0f;
        gw[e] = dy[e] * w[e];
    }
}

template <typename T>
__device__ __forceinline__ void store_grad(const NormGradArgs& a, float rstd, float c1, float c2, int64_t row,
                                           int64_t g, int n, int lane, const float (&u)[8], const float (&gw)[8]) {
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = rstd * (gw[e] - c1 - u[e] * c2);
    Raw<T> r;
    if (a.grad_hidden.data) {
        float y[8];
        load_granule(r, static_cast<const T*>(a.grad_hidden.data) + row * a.grad_hidden.stride, g * kGran, n);
        widen(r, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] += y[e];
    }
    if (a.grad_res.data) {
        narrow(t, r);
        store_span(static_cast<T*>(a.grad_res.data) + row * a.grad_res.stride + g * kGran, r, n, lane);
    }
    if (a.mask.limit < 65536) drop(t, a.mask, row, (uint32_t)g);
    narrow(t, r);
    store_span(static_cast<T*>(a.grad_x.data) + row * a.grad_x.stride + g * kGran, r, n, lane);
}

// parts[part][0 weight, 1 bias][stride]: the sums of one group's rows.
template <typename T, typename P, int V>
__global__ void __launch_bounds__(kNormThreads) norm_grad_kernel(NormGradArgs a, int gw, int64_t stride) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, group = w / gw, warp = w % gw;
    const int groups = (blockDim.x >> 5) / gw;
    float dw[V][8] = {}, db[V][8] = {};
    int slot = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < a.rows; r0 += (int64_t)gridDim.x * groups) {
        const int64_t row = r0 + group;
        const bool on = row < a.rows;
        const float mean = on ? __ldg(a.mean + row) : 0.0f, rstd = on ? __ldg(a.rstd + row) : 0.0f;
        float u[V][8], g1[V][8];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t g = (v * gw + warp) * 32 + lane;
            const int n = on ? granule_cols(g, a.cols) : 0;
            float dy[8];
            if (on) {
                load_grad<T, P>(a, mean, rstd, row, g, n, dy, u[v], g1[v]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    db[v][e] += dy[e];
                    dw[v][e] = __fmaf_rn(dy[e], u[v][e], dw[v][e]);
                    if (e < n) {
                        s1 += g1[v][e];
                        s2 = __fmaf_rn(g1[v][e], u[v][e], s2);
                    }
                }
            }
        }
        const float2 c = group_sum(s1, s2, gw, group, warp, lane, slot);
        slot ^= 1;
        if (!on) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t g = (v * gw + warp) * 32 + lane;
            store_grad<T>(a, rstd, c.x / (float)a.cols, c.y / (float)a.cols, row, g, granule_cols(g, a.cols), lane,
                          u[v], g1[v]);
        }
    }
    float* p = a.work + ((int64_t)blockIdx.x * groups + group) * 2 * stride;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int64_t c = ((v * gw + warp) * 32 + lane) * (int64_t)kGran;
        if (c >= a.cols) continue;
        float4* q = reinterpret_cast<float4*>(p + c);
        q[0] = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
        q[1] = make_float4(dw[v][4], dw[v][5], dw[v][6], dw[v][7]);
        q = reinterpret_cast<float4*>(p + stride + c);
        q[0] = make_float4(db[v][0], db[v][1], db[v][2], db[v][3]);
        q[1] = make_float4(db[v][4], db[v][5], db[v][6], db[v][7]);
    }
}

// Rows too wide for registers: the rows' gradients, a block each ...
template <typename T, typename P>
__global__ void __launch_bounds__(kNormThreads) norm_grad_wide_kernel(NormGradArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gw = kNormThreads / 32;
    const int64_t row = blockIdx.x, end = (a.cols + kSpan - 1) / kSpan * 32;
    const float mean = __ldg(a.mean + row), rstd = __ldg(a.rstd + row);
    float dy[8], u[8], g1[8], s1 = 0.0f, s2 = 0.0f;
    for (int64_t g = threadIdx.x; g < end; g += kNormThreads) {
        const int n = granule_cols(g, a.cols);
        load_grad<T, P>(a, mean, rstd, row, g, n, dy, u, g1);
        float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) {
                t1 += g1[e];
                t2 = __fmaf_rn(g1[e], u[e], t2);
            }
        s1 += t1;
        s2 += t2;
    }
    const float2 c = group_sum(s1, s2, gw, 0, warp, lane, 0);
    for (int64_t g = threadIdx.x; g < end; g += kNormThreads) {
        const int n = granule_cols(g, a.cols);
        load_grad<T, P>(a, mean, rstd, row, g, n, dy, u, g1);
        store_grad<T>(a, rstd, c.x / (float)a.cols, c.y / (float)a.cols, row, g, n, lane, u, g1);
    }
}
// ... and the weight's and bias's sums, a warp for a span of columns and a
// share of the rows.
template <typename T, typename P>
__global__ void __launch_bounds__(256) norm_param_kernel(NormGradArgs a, int64_t stride, int parts) {
    const int lane = threadIdx.x & 31, part = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int64_t g = (int64_t)blockIdx.x * 32 + lane, c = g * kGran;
    const int n = granule_cols(g, a.cols);
    if (part >= parts || n == 0) return;
    float dw[8] = {}, db[8] = {};
    for (int64_t row = part; row < a.rows; row += parts) {
        float dy[8], u[8], g1[8];
        load_grad<T, P>(a, __ldg(a.mean + row), __ldg(a.rstd + row), row, g, n, dy, u, g1);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            db[e] += dy[e];
            dw[e] = __fmaf_rn(dy[e], u[e], dw[e]);
        }
    }
    float* p = a.work + (int64_t)part * 2 * stride + c;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        p[e] = dw[e];
        p[stride + e] = db[e];
    }
}

// Adds the parts' sums, 32 columns a block, a share of the parts for each of
// its 8 warps: blockIdx.y 0 the weight's, 1 the bias's.
template <typename G>
__global__ void __launch_bounds__(256)
    norm_join_kernel(const float* work, int64_t stride, int parts, int64_t cols, int accumulate, G* gw, G* gb) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    G* out = blockIdx.y ? gb : gw;
    if (!out) return;
    float s = 0.0f;
    if (c < cols)
        for (int p = parts * warp / 8; p < parts * (warp + 1) / 8; ++p) s += __ldcg(work + (2 * (int64_t)p + blockIdx.y) * stride + c);
    sums[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || c >= cols) return;
    s = 0.0f;
    for (int q = 0; q < 8; ++q) s += sums[q][lane];
    if (accumulate) s += load_f32(out, c);
    store_f32(out, c, s);
}

struct NormGradPlan {
    bool wide;
    int v, gw, groups, grid, parts;
    int64_t stride;
};

NormGradPlan grad_plan(int64_t rows, int64_t cols) {
    NormGradPlan p;
    const int64_t grans = (cols + kGran - 1) / kGran;
    p.stride = grans * kGran;
    p.wide = cols > kNormCols;
    if (p.wide) {
        p.v = p.gw = p.groups = p.grid = 0;
        p.parts = (int)(rows < 256 ? rows : 256);
        return p;
    }
    p.v = grans <= 32 * 8 ? 1 : (grans <= 32 * 16 ? 2 : 4);
    p.gw = (int)((grans + 32 * p.v - 1) / (32 * p.v));
    p.groups = p.gw >= 4 ? 1 : 4 / p.gw;
    const int64_t blocks = (rows + p.groups - 1) / p.groups;
    p.grid = (int)(blocks < 304 ? blocks : 304);
    p.parts = p.grid * p.groups;
    return p;
}

template <typename T, typename P>
cudaError_t norm_grad_rows(const NormGradArgs& a, const NormGradPlan& p, cudaStream_t s) {
    if (p.wide) {
        norm_grad_wide_kernel<T, P><<<(unsigned)a.rows, kNormThreads, 0, s>>>(a);
        count_launch();
        const dim3 grid((unsigned)((a.cols + kSpan - 1) / kSpan), (unsigned)((p.parts + 7) / 8));
        norm_param_kernel<T, P><<<grid, 256, 0, s>>>(a, p.stride, p.parts);
    } else if (p.v == 1) {
        norm_grad_kernel<T, P, 1><<<p.grid, 32 * p.gw * p.groups, 0, s>>>(a, p.gw, p.stride);
    } else if (p.v == 2) {
        norm_grad_kernel<T, P, 2><<<p.grid, 32 * p.gw * p.groups, 0, s>>>(a, p.gw, p.stride);
    } else {
        norm_grad_kernel<T, P, 4><<<p.grid, 32 * p.gw * p.groups, 0, s>>>(a, p.gw, p.stride);
    }
    count_launch();
    return cudaGetLastError();
}

}  // namespace

size_t norm_grad_bytes(int64_t rows, int64_t cols) {
    if (rows == 0 || cols == 0) return 0;
    const NormGradPlan p = grad_plan(rows, cols);
    return (size_t)p.parts * 2 * p.stride * 4;
}

cudaError_t launch_norm(int dt, int param_dt, const NormArgs& a, cudaStream_t s) {
    if (a.rows == 0 || a.cols == 0) return cudaSuccess;
    if (dt == FSDP_F32) return param_dt == FSDP_F32 ? norm<float, float>(a, s) : norm<float, uint16_t>(a, s);
    return param_dt == FSDP_F32 ? norm<uint16_t, float>(a, s) : norm<uint16_t, uint16_t>(a, s);
}

cudaError_t launch_norm_grad(int dt, int param_dt, int param_grad_dt, const NormGradArgs& a, cudaStream_t s) {
    if (a.cols == 0) return cudaSuccess;
    NormGradPlan p = {};
    if (a.rows > 0) {
        p = grad_plan(a.rows, a.cols);
        cudaError_t e;
        if (dt == FSDP_F32)
            e = param_dt == FSDP_F32 ? norm_grad_rows<float, float>(a, p, s) : norm_grad_rows<float, uint16_t>(a, p, s);
        else
            e = param_dt == FSDP_F32 ? norm_grad_rows<uint16_t, float>(a, p, s) : norm_grad_rows<uint16_t, uint16_t>(a, p, s);
        if (e != cudaSuccess) return e;
    }
    if (!a.grad_weight && !a.grad_bias) return cudaSuccess;
    const dim3 grid((unsigned)((a.cols + 31) / 32), 2);
    if (param_grad_dt == FSDP_F32)
        norm_join_kernel<float><<<grid, 256, 0, s>>>(a.work, p.stride, p.parts, a.cols, a.accumulate,
                                                     static_cast<float*>(a.grad_weight), static_cast<float*>(a.grad_bias));
    else
        norm_join_kernel<uint16_t><<<grid, 256, 0, s>>>(a.work, p.stride, p.parts, a.cols, a.accumulate,
                                                        static_cast<uint16_t*>(a.grad_weight), static_cast<uint16_t*>(a.grad_bias));
    count_launch();
    return cudaGetLastError();
}

}  // namespace fsdp
