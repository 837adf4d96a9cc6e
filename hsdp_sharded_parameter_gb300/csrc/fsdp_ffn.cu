// The gated feed-forward block and its gradient.
#include "fsdp_gemm.cuh"

namespace fsdp {
namespace {

__device__ __forceinline__ uint16_t* at(const Mat& m, int64_t row, int64_t col) {
    return static_cast<uint16_t*>(m.data) + row * m.stride + col;
}

// ------------------------------------------------------------- activations

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.0f, 1.0f + expf(-z)); }
__device__ __forceinline__ float act_value(int act, float z) {
    if (act == FSDP_SILU) return z * sigmoid(z);
    if (act == FSDP_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    return z <= 0.0f ? 0.0f : z;
}
// The value, and the derivative in `slope`.
__device__ __forceinline__ float act_both(int act, float z, float& slope) {
    if (act == FSDP_SILU) {
        const float p = sigmoid(z), v = z * p;
        slope = __fmaf_rn(v, 1.0f - p, p);
        return v;
    }
    if (act == FSDP_GELU) {
        const float p = 0.5f + 0.5f * erff(z * 0.70710678118654752f);
        slope = __fmaf_rn(z * 0.39894228040143268f, expf(-0.5f * z * z), p);
        return z * p;
    }
    slope = z <= 0.0f ? 0.0f : 1.0f;
    return z <= 0.0f ? 0.0f : z;
}

// -------------------------------------------------------------- epilogues

__device__ __forceinline__ void put_bf16(const Mat& m, int64_t row, int64_t col, int n, const Cols& v) {
    Raw<uint16_t> r;
    round_to(v, r);
    store_granule(at(m, row, col), r, n);
}

// out = D, or out + D.
template <typename T>
struct Store {
    Mat out;
    int accumulate;
    __device__ __forceinline__ void operator()(int64_t row, int64_t col, int n, const Cols& v, const Cols&) const {
        T* p = static_cast<T*>(out.data) + row * out.stride + col;
        Raw<T> r;
        Cols sum = v;
        if (accumulate) {
            load_granule(r, p, 0, n);
            sum = sum + widened(r);
        }
        round_to(sum, r);
        store_granule(p, r, n);
    }
};

// h = act(gate) * up from the two projections, which are kept on request.
struct Gated {
    Mat h, gate, up;
    int act;
    __device__ __forceinline__ void operator()(int64_t row, int64_t col, int n, const Cols& g, const Cols& u) const {
        Cols v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v.set(e, act_value(act, g.get(e)) * u.get(e));
        put_bf16(h, row, col, n, v);
        if (gate.data) {
            put_bf16(gate, row, col, n, g);
            put_bf16(up, row, col, n, u);
        }
    }
};

// From the gradient d of h: those of gate and up, and h again.
struct GatedGrad {
    Mat gate, up, grad_gate, grad_up, h;
    int act;
    __device__ __forceinline__ void operator()(int64_t row, int64_t col, int n, const Cols& d, const Cols&) const {
        Raw<uint16_t> r;
        load_granule(r, at(gate, row, col), 0, n);
        const Cols g = widened(r);
        load_granule(r, at(up, row, col), 0, n);
        const Cols u = widened(r);
        Cols dg, du, v;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float slope;
            const float a = act_both(act, g.get(e), slope);
            v.set(e, a * u.get(e));
            du.set(e, d.get(e) * a);
            dg.set(e, d.get(e) * u.get(e) * slope);
        }
        put_bf16(grad_gate, row, col, n, dg);
        put_bf16(grad_up, row, col, n, du);
        put_bf16(h, row, col, n, v);
    }
};

int64_t padded(int64_t n) { return (n + 7) / 8 * 8; }
size_t room(int64_t rows, int64_t cols) { return (size_t)((rows * padded(cols) * 2 + 255) / 256 * 256); }

}  // namespace

size_t ffn_bytes(const FfnArgs& a) { return room(a.tokens, a.inner); }
size_t ffn_grad_bytes(const FfnGradArgs& a) { return 3 * room(a.tokens, a.inner); }
size_t ffn_most_bytes(int64_t tokens, int64_t, int64_t inner, bool) { return room(tokens, inner); }
size_t ffn_grad_most_bytes(int64_t tokens, int64_t, int64_t inner, bool) { return 3 * room(tokens, inner); }

cudaError_t launch_ffn(const FfnArgs& a, cudaStream_t s) {
    const Mat h = {a.work, padded(a.inner)};
    const Product in = {a.tokens, a.inner, 1, {a.hidden, 0}, {a.x, {}}, {a.w_gate, a.w_up}, 0, 0, 0, 1};
    const Product out = {a.tokens, a.hidden, 1, {a.inner, 0}, {h, {}}, {a.w_down, {}}, 0, 0, 0, 0};
    cudaError_t e = launch_product(in, Gated{h, a.gate, a.up, a.act}, s, true);
    if (e == cudaSuccess) e = launch_product(out, Store<uint16_t>{a.out, 0}, s, false);
    return e;
}

namespace {
template <typename T>
cudaError_t ffn_grad(const FfnGradArgs& a, cudaStream_t s) {
    const size_t each = room(a.tokens, a.inner);
    const int64_t ld = padded(a.inner);
    const Mat dg = {a.work, ld}, du = {a.work + each, ld}, h = {a.work + 2 * each, ld};
    const Product through = {a.tokens, a.inner, 1, {a.hidden, 0}, {a.grad, {}}, {a.w_down, {}}, 0, 1, 0, 0};
    const Product dx = {a.tokens, a.hidden, 2, {a.inner, a.inner}, {dg, du}, {a.w_gate, a.w_up}, 0, 1, 0, 0};
    const Product down = {a.hidden, a.inner, 1, {a.tokens, 0}, {a.grad, {}}, {h, {}}, 1, 1, 0, 0};
    Product side = {a.inner, a.hidden, 1, {a.tokens, 0}, {dg, {}}, {a.x, {}}, 1, 1, 0, 0};
    cudaError_t e = launch_product(through, GatedGrad{a.gate, a.up, dg, du, h, a.act}, s, true);
    if (e == cudaSuccess) e = launch_product(dx, Store<uint16_t>{a.grad_x, 0}, s, false);
    if (e == cudaSuccess) e = launch_product(down, Store<T>{a.grad_down, a.accumulate}, s, false);
    if (e == cudaSuccess) e = launch_product(side, Store<T>{a.grad_gate, a.accumulate}, s, false);
    side.a[0] = du;
    if (e == cudaSuccess) e = launch_product(side, Store<T>{a.grad_up, a.accumulate}, s, false);
    return e;
}
}  // namespace

cudaError_t launch_ffn_grad(int param_grad_dt, const FfnGradArgs& a, cudaStream_t s) {
    return param_grad_dt == FSDP_F32 ? ffn_grad<float>(a, s) : ffn_grad<uint16_t>(a, s);
}

cudaError_t ffn_gave_up(int* value, cudaStream_t s) { return take_gave_up(value, s); }

}  // namespace fsdp
