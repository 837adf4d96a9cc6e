// The gated feed-forward block and its gradient.
#include "fsdp_gemm.cuh"

namespace fsdp {
namespace {

__device__ __forceinline__ uint16_t* at(const Mat& m, int64_t row, int64_t col) {
    return static_cast<uint16_t*>(m.data) + row * m.stride + col;
}

// ------------------------------------------------------------- activations

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.0f, 1.0f + expf(-z)); }
// The normal distribution's integral up to z. (As (1 + erf) / 2 it has no digits
// left below z = -5. Out of line: eight of it in the epilogue cost the other
// activations too, 16384 x 4096 x 11008 with SiLU 2585 us and 2670.)
__device__ __noinline__ float normal_below(float z) { return 0.5f * erfcf(z * -0.70710678118654752f); }
__device__ __forceinline__ float act_value(int act, float z) {
    if (act == FSDP_SILU) return z * sigmoid(z);
    if (act == FSDP_GELU) return z * normal_below(z);
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
        const float p = normal_below(z);
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

// out = D, or out + D; each of a group's products has an out of its own.
template <typename T>
struct Store {
    static constexpr bool kMirror = false;
    struct Before {
        Raw<T> old;
    };
    struct Once {};
    Mat out[kMaxGroup];
    int accumulate;
    __device__ __forceinline__ Once once() const { return {}; }
    __device__ __forceinline__ T* place(int i, int64_t row, int64_t col) const {
        const Mat& o = i == 0 ? out[0] : (i == 1 ? out[1] : out[2]);
        return static_cast<T*>(o.data) + row * o.stride + col;
    }
    __device__ __forceinline__ void bring(int i, int64_t row, int64_t col, int n, Before& b) const {
        if (accumulate) load_granule(b.old, place(i, row, col), 0, n);
    }
    __device__ __forceinline__ void operator()(int i, int, int64_t row, int64_t col, int n, const Cols& v, const Cols&, const Before& b,
                                               Once, Raw<uint16_t>&) const {
        Raw<T> r;
        round_to(accumulate ? v + widened(b.old) : v, r);
        store_granule(place(i, row, col), r, n);
    }
};

// h = act(gate) * up from the two projections, which are kept on request.
struct Gated {
    static constexpr bool kMirror = false;
    struct Before {};
    struct Once {};
    Mat h, gate, up;
    int act;
    __device__ __forceinline__ Once once() const { return {}; }
    __device__ __forceinline__ void bring(int, int64_t, int64_t, int, Before&) const {}
    __device__ __forceinline__ void operator()(int, int, int64_t row, int64_t col, int n, const Cols& g, const Cols& u, const Before&,
                                               Once, Raw<uint16_t>&) const {
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
    static constexpr bool kMirror = false;
    struct Before {
        Raw<uint16_t> gate, up;
    };
    struct Once {};
    Mat gate, up, grad_gate, grad_up, h;
    int act;
    __device__ __forceinline__ Once once() const { return {}; }
    __device__ __forceinline__ void bring(int, int64_t row, int64_t col, int n, Before& b) const {
        load_granule(b.gate, at(gate, row, col), 0, n);
        load_granule(b.up, at(up, row, col), 0, n);
    }
    __device__ __forceinline__ void operator()(int, int, int64_t row, int64_t col, int n, const Cols& d, const Cols&, const Before& b,
                                               Once, Raw<uint16_t>&) const {
        const Cols g = widened(b.gate), u = widened(b.up);
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

// ------------------------------------------------------------ the products

Product gated_product(const FfnArgs& a) {
    return {a.tokens, a.inner, 1, {a.hidden, 0}, {a.x, {}}, {a.w_gate, a.w_up}, 0, 0, 0, 1, 0};
}
Product out_product(const FfnArgs& a, const Mat& h) {
    return {a.tokens, a.hidden, 1, {a.inner, 0}, {h, {}}, {a.w_down, {}}, 0, 0, 0, 0, 0};
}
Product through_product(const FfnGradArgs& a) {
    return {a.tokens, a.inner, 1, {a.hidden, 0}, {a.grad, {}}, {a.w_down, {}}, 0, 1, 0, 0, 0};
}
Product x_product(const FfnGradArgs& a, const Mat& dg, const Mat& du) {
    return {a.tokens, a.hidden, 2, {a.inner, a.inner}, {dg, du}, {a.w_gate, a.w_up}, 0, 1, 0, 0, 0};
}

// Room for the parts' sums of the larger of two products.
size_t sums_room(size_t a, size_t b) { return (std::max(a, b) + 255) / 256 * 256; }
size_t copy_room(const Mat& f, int64_t rows, int64_t cols) { return copies_read(f, rows, cols) ? 0 : aligned_room(rows, cols); }

}  // namespace

size_t ffn_bytes(const FfnArgs& a) {
    return aligned_room(a.tokens, a.inner) + sums_room(parts_bytes(gated_product(a)), parts_bytes(out_product(a, {}))) +
           copy_room(a.x, a.tokens, a.hidden) + copy_room(a.w_gate, a.inner, a.hidden) + copy_room(a.w_up, a.inner, a.hidden) +
           copy_room(a.w_down, a.hidden, a.inner);
}
size_t ffn_most_bytes(int64_t tokens, int64_t hidden, int64_t inner, bool aligned) {
    const size_t copies = aligned ? 0 : aligned_room(tokens, hidden) + 2 * aligned_room(inner, hidden) + aligned_room(hidden, inner);
    return aligned_room(tokens, inner) + sums_room(parts_most_bytes(tokens, inner, 2), parts_most_bytes(tokens, hidden, 1)) + copies;
}
size_t ffn_grad_bytes(const FfnGradArgs& a) {
    return 3 * aligned_room(a.tokens, a.inner) + sums_room(parts_bytes(through_product(a)), parts_bytes(x_product(a, {}, {}))) +
           copy_room(a.grad, a.tokens, a.hidden) + copy_room(a.x, a.tokens, a.hidden) + copy_room(a.w_gate, a.inner, a.hidden) +
           copy_room(a.w_up, a.inner, a.hidden) + copy_room(a.w_down, a.hidden, a.inner);
}
size_t ffn_grad_most_bytes(int64_t tokens, int64_t hidden, int64_t inner, bool aligned) {
    const size_t copies = aligned ? 0 : 2 * aligned_room(tokens, hidden) + 2 * aligned_room(inner, hidden) + aligned_room(hidden, inner);
    return 3 * aligned_room(tokens, inner) + sums_room(parts_most_bytes(tokens, inner, 1), parts_most_bytes(tokens, hidden, 1)) + copies;
}

cudaError_t launch_ffn(const FfnArgs& args, cudaStream_t s) {
    FfnArgs a = args;
    Copies c = {};
    char* room = a.work;
    const Mat h = {room, whole_granules(a.inner)};
    room += aligned_room(a.tokens, a.inner);
    float* sums = reinterpret_cast<float*>(room);
    room += sums_room(parts_bytes(gated_product(a)), parts_bytes(out_product(a, h)));
    a.x = readable(a.x, a.tokens, a.hidden, &c, &room);
    a.w_gate = readable(a.w_gate, a.inner, a.hidden, &c, &room);
    a.w_up = readable(a.w_up, a.inner, a.hidden, &c, &room);
    a.w_down = readable(a.w_down, a.hidden, a.inner, &c, &room);
    if (a.tokens == 0) return cudaSuccess;
    cudaError_t e = launch_copies(c, s);
    if (e == cudaSuccess) e = launch_product(gated_product(a), Gated{h, a.gate, a.up, a.act}, sums, s, c.n == 0);
    if (e == cudaSuccess) e = launch_product(out_product(a, h), Store<uint16_t>{{a.out, {}, {}}, 0}, sums, s, false);
    return e;
}

namespace {
template <typename T>
cudaError_t ffn_grad(const FfnGradArgs& args, cudaStream_t s) {
    FfnGradArgs a = args;
    Copies c = {};
    char* room = a.work;
    const size_t each = aligned_room(a.tokens, a.inner);
    const int64_t ld = whole_granules(a.inner);
    const Mat dg = {room, ld}, du = {room + each, ld}, h = {room + 2 * each, ld};
    room += 3 * each;
    float* sums = reinterpret_cast<float*>(room);
    room += sums_room(parts_bytes(through_product(a)), parts_bytes(x_product(a, dg, du)));
    a.grad = readable(a.grad, a.tokens, a.hidden, &c, &room);
    a.x = readable(a.x, a.tokens, a.hidden, &c, &room);
    a.w_gate = readable(a.w_gate, a.inner, a.hidden, &c, &room);
    a.w_up = readable(a.w_up, a.inner, a.hidden, &c, &room);
    a.w_down = readable(a.w_down, a.hidden, a.inner, &c, &room);
    const Product weights[3] = {{a.inner, a.hidden, 1, {a.tokens, 0}, {dg, {}}, {a.x, {}}, 1, 1, 0, 0, 0},
                                {a.inner, a.hidden, 1, {a.tokens, 0}, {du, {}}, {a.x, {}}, 1, 1, 0, 0, 0},
                                {a.hidden, a.inner, 1, {a.tokens, 0}, {a.grad, {}}, {h, {}}, 1, 1, 0, 0, 0}};
    const Store<T> store = {{a.grad_gate, a.grad_up, a.grad_down}, a.accumulate};
    if (a.tokens == 0) {
        // sums over nothing
        for (int i = 0; i < 3; ++i) {
            const cudaError_t e = launch_product(weights[i], Store<T>{{store.out[i], {}, {}}, a.accumulate}, nullptr, s, true);
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    }
    cudaError_t e = launch_copies(c, s);
    if (e == cudaSuccess) e = launch_product(through_product(a), GatedGrad{a.gate, a.up, dg, du, h, a.act}, sums, s, c.n == 0);
    if (e == cudaSuccess) e = launch_product(x_product(a, dg, du), Store<uint16_t>{{a.grad_x, {}, {}}, 0}, sums, s, false);
    if (e == cudaSuccess && a.inner > 0 && a.hidden > 0) e = launch_group(weights, 3, store, cut_of(weights[0], false), s, false);
    return e;
}
}  // namespace

cudaError_t launch_ffn_grad(int param_grad_dt, const FfnGradArgs& a, cudaStream_t s) {
    return param_grad_dt == FSDP_F32 ? ffn_grad<float>(a, s) : ffn_grad<uint16_t>(a, s);
}

cudaError_t ffn_gave_up(int* value, cudaStream_t s) { return take_gave_up(value, s); }

}  // namespace fsdp
