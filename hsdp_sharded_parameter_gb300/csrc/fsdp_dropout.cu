// Dropout with a mask that is never stored, optionally added to a residual:
//   out = residual + keep(seed, draw, r, c) * x * 65536 / K.
// The backward pass is the same kernel on the gradient.
#include "fsdp_ops.cuh"

namespace fsdp {
namespace {

constexpr int kDropWarps = 8;

// A warp takes a span of 256 columns of a row at a time, kGroup of them in
// flight.
template <typename T>
__global__ void __launch_bounds__(32 * kDropWarps) dropout_kernel(DropoutArgs a, int64_t spans, int64_t items) {
    const int lane = threadIdx.x & 31;
    for (int64_t it = warp_id(); it < items; it += warp_count()) {
        const int64_t row = it / spans, g = (it - row * spans) * 32 + lane, c = g * kGran;
        const int n = granule_cols(g, a.cols);
        Raw<T> in, out;
        float x[8], y[8];
        load_granule(in, static_cast<const T*>(a.x.data) + row * a.x.stride, c, n);
        if (a.res.data) load_granule(out, static_cast<const T*>(a.res.data) + row * a.res.stride, c, n);
        widen(in, x);
        drop(x, a.mask, row, (uint32_t)g);
        if (a.res.data) {
            widen(out, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += y[e];
        }
        narrow(x, out);
        store_span(static_cast<T*>(a.out.data) + row * a.out.stride + c, out, n, lane);
    }
}

}  // namespace

cudaError_t launch_dropout(int dt, const DropoutArgs& a, cudaStream_t s) {
    if (a.rows == 0 || a.cols == 0) return cudaSuccess;
    const int64_t spans = (a.cols + kSpan - 1) / kSpan, items = spans * a.rows;
    const int64_t blocks = (items + kDropWarps - 1) / kDropWarps;
    const unsigned grid = (unsigned)(blocks < 0x7fffffff ? blocks : 0x7fffffff);
    if (dt == FSDP_F32)
        dropout_kernel<float><<<grid, 32 * kDropWarps, 0, s>>>(a, spans, items);
    else
        dropout_kernel<uint16_t><<<grid, 32 * kDropWarps, 0, s>>>(a, spans, items);
    count_launch();
    return cudaGetLastError();
}

}  // namespace fsdp
