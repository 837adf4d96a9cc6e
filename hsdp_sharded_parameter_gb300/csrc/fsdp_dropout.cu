// Dropout with a mask that is never stored, optionally added to a residual:
//   out = residual + keep(seed, draw, r, c) * x * 65536 / K.
// The backward pass is the same kernel on the gradient.
#include "fsdp_ops.cuh"

namespace fsdp {
namespace {

constexpr int kDropWarps = 8;
// Spans of a warp at a time.
template <typename T>
constexpr int kDropSpans = sizeof(T) == 4 ? 2 : 4;

// A warp takes kU neighbouring spans of 256 columns of a row at a time and
// starts all their loads before it draws the first mask: into registers, or,
// for rows off the 16-byte grid, whose granules are put together from two
// blocks each, into shared memory (kept in registers, they left room for half
// the loads in flight).
template <typename T, bool kAligned>
__global__ void __launch_bounds__(32 * kDropWarps, 4) dropout_kernel(DropoutArgs a, int64_t steps, int64_t items) {
    constexpr int kU = kDropSpans<T>;
    __shared__ uint4 staged[kAligned ? 1 : kDropWarps][kAligned ? 1 : 2 * kU][kAligned ? 1 : kSlot<false, T>];
    const int lane = threadIdx.x & 31;
    uint4(*const mine)[kAligned ? 1 : kSlot<false, T>] = staged[kAligned ? 0 : threadIdx.x >> 5];
    for (int64_t it = warp_id(); it < items; it += warp_count()) {
        const int64_t row = it / steps, g0 = (it - row * steps) * (kU * 32) + lane, c0 = (g0 - lane) * kGran;
        const T* x = static_cast<const T*>(a.x.data) + row * a.x.stride;
        const T* res = static_cast<const T*>(a.res.data) + row * a.res.stride;
        T* out = static_cast<T*>(a.out.data) + row * a.out.stride;
        const int left = (int)(a.cols - c0 < kU * kSpan ? a.cols - c0 : kU * kSpan);
        Raw<T> in[kU], add[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if constexpr (kAligned) {
                const int64_t g = g0 + u * 32;
                const int n = granule_cols(g, a.cols);
                load_cols<true>(in[u], x, g * kGran, n);
                if (a.res.data) load_cols<true>(add[u], res, g * kGran, n);
            } else {
                span_fetch<false>(mine[u], x + c0, u * kSpan, left, lane);
                if (a.res.data) span_fetch<false>(mine[kU + u], res + c0, u * kSpan, left, lane);
            }
        }
        if constexpr (!kAligned) {
            async_commit();
            async_wait<0>();
            __syncwarp();
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t g = g0 + u * 32;
            if constexpr (!kAligned) {
                if (u * kSpan >= left) break;
                span_read<false>(in[u], mine[u], x + c0, u * kSpan, lane);
                if (a.res.data) span_read<false>(add[u], mine[kU + u], res + c0, u * kSpan, lane);
            }
            const Cols v = widened(in[u]);
            Cols y = a.res.data ? widened(add[u]) : all(0.0f);
            if (a.mask.drops)
                add_dropped(y, v, a.mask, row, (uint32_t)g);
            else
                y = y + v;
            round_to(y, in[u]);
            store_cols<kAligned>(out + g * kGran, in[u], granule_cols(g, a.cols), lane);
        }
        if constexpr (!kAligned) __syncwarp();  // before the next spans come in
    }
}

// Narrow rows of grans granules, items granules in all.
template <typename T, bool kAligned>
__global__ void __launch_bounds__(32 * kDropWarps) dropout_narrow_kernel(DropoutArgs a, uint32_t grans, uint32_t items) {
    const uint32_t i0 = blockIdx.x * (kNarrow * blockDim.x) + threadIdx.x;
    Raw<T> in[kNarrow], add[kNarrow];
#pragma unroll
    for (int u = 0; u < kNarrow; ++u) {
        const uint32_t i = i0 + u * blockDim.x, row = i / grans, g = i - row * grans;
        const int n = i < items ? granule_cols((int64_t)g, a.cols) : 0;
        load_cols<kAligned>(in[u], static_cast<const T*>(a.x.data) + row * a.x.stride, g * kGran, n);
        if (a.res.data) load_cols<kAligned>(add[u], static_cast<const T*>(a.res.data) + row * a.res.stride, g * kGran, n);
    }
#pragma unroll
    for (int u = 0; u < kNarrow; ++u) {
        const uint32_t i = i0 + u * blockDim.x, row = i / grans, g = i - row * grans;
        if (i >= items) break;
        const Cols v = widened(in[u]);
        Cols y = a.res.data ? widened(add[u]) : all(0.0f);
        if (a.mask.drops)
            add_dropped(y, v, a.mask, row, g);
        else
            y = y + v;
        round_to(y, in[u]);
        store_granule(static_cast<T*>(a.out.data) + row * a.out.stride + g * kGran, in[u], granule_cols((int64_t)g, a.cols));
    }
}

template <typename T, bool kAligned>
void dropout(const DropoutArgs& a, cudaStream_t s) {
    if (narrow_rows(a.rows, a.cols, kAligned)) {
        const uint32_t grans = (uint32_t)((a.cols + kGran - 1) / kGran), items = (uint32_t)a.rows * grans;
        const uint32_t each = kNarrow * 32 * kDropWarps;
        dropout_narrow_kernel<T, kAligned><<<(items + each - 1) / each, 32 * kDropWarps, 0, s>>>(a, grans, items);
        return;
    }
    const int64_t span = kSpan * kDropSpans<T>, steps = (a.cols + span - 1) / span, items = steps * a.rows;
    const int64_t blocks = (items + kDropWarps - 1) / kDropWarps;
    const unsigned grid = (unsigned)(blocks < 0x7fffffff ? blocks : 0x7fffffff);
    dropout_kernel<T, kAligned><<<grid, 32 * kDropWarps, 0, s>>>(a, steps, items);
}

}  // namespace

cudaError_t launch_dropout(int dt, const DropoutArgs& a, cudaStream_t s) {
    if (a.rows == 0 || a.cols == 0) return cudaSuccess;
    const int es = dt == FSDP_F32 ? 4 : 2;
    const bool aligned = a.cols % kGran == 0 && on_grid(a.x, es) && on_grid(a.res, es) && on_grid(a.out, es);
    if (dt == FSDP_F32)
        aligned ? dropout<float, true>(a, s) : dropout<float, false>(a, s);
    else
        aligned ? dropout<uint16_t, true>(a, s) : dropout<uint16_t, false>(a, s);
    count_launch();
    return cudaGetLastError();
}

}  // namespace fsdp
