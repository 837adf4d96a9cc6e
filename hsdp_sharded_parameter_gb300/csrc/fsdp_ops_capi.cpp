// C-ABI entry points of the training operators: argument checks and the
// hand-over to the kernels (fsdp_embedding.cu, fsdp_dropout.cu, fsdp_norm.cu).
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <string>

#include "fsdp_internal.h"
#include "fsdp_ops.h"

namespace fsdp {

int sm_count() {
    static std::atomic<int> known[64];  // by device, 0: not asked yet
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64) {
        n = known[dev].load(std::memory_order_relaxed);
        if (n > 0) return n;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0) {
            known[dev].store(n, std::memory_order_relaxed);
            return n;
        }
    }
    (void)cudaGetLastError();
    return 1;
}

cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

namespace {

int bad(const char* what, const std::string& why) { return set_error(FSDP_ERR_INVALID_ARG, std::string(what) + ": " + why); }

// A matrix argument as the checks see it.
struct Operand {
    const char* name;
    const void* data;
    int64_t stride;
    int dt;
    int64_t rows;
    bool output, optional;
};

constexpr int64_t kMaxSide = (int64_t)1 << 40;

int check_size(const char* what, int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || rows > kMaxSide || cols > kMaxSide) return bad(what, "a size is negative or too large");
    return FSDP_OK;
}

int check_operands(const char* what, int64_t cols, std::initializer_list<Operand> ops) {
    for (const Operand& o : ops) {
        const std::string name = o.name;
        const int es = elem_size(o.dt);
        if (es == 0) return bad(what, name + ": unknown dtype");
        if (!o.data) {
            if (!o.optional && o.rows > 0 && cols > 0) return bad(what, name + " is NULL");
            continue;
        }
        if (reinterpret_cast<uintptr_t>(o.data) % es) return bad(what, name + " is not aligned to its element size");
        if (o.stride < 0 || o.stride > kMaxSide) return bad(what, name + ": stride out of range");
        if (o.output && o.rows > 1 && o.stride < cols) return bad(what, name + ": rows of an output overlap (stride below its columns)");
        // the last element's offset has to fit 62 bits
        if (o.rows > 0 && o.stride > 0 && o.rows > ((int64_t)1 << 59) / o.stride) return bad(what, name + " is too large");
    }
    return FSDP_OK;
}

int check_ids(const char* what, int index_type, const void* ids, int64_t n, int64_t vocab, int64_t cols,
              int64_t most = INT32_MAX - 1) {
    if (cols > INT32_MAX) return bad(what, "too many columns");
    if (index_type != FSDP_I32 && index_type != FSDP_I64) return bad(what, "unknown index type");
    if (n < 0 || n > most) return bad(what, "n_ids out of range");
    if (vocab < 0 || vocab >= INT32_MAX) return bad(what, "vocab out of range");
    if (n > 0 && !ids) return bad(what, "ids is NULL");
    if (reinterpret_cast<uintptr_t>(ids) % (index_type == FSDP_I64 ? 8 : 4)) return bad(what, "ids is not aligned to its element size");
    return FSDP_OK;
}

int check_work(const char* what, const void* work, size_t have, size_t need) {
    if (have < need) return bad(what, "workspace holds " + std::to_string(have) + " bytes, needs " + std::to_string(need));
    if (need > 0 && !work) return bad(what, "workspace is NULL");
    if (reinterpret_cast<uintptr_t>(work) % 16) return bad(what, "workspace is not 16-byte aligned");
    return FSDP_OK;
}

int make_mask(const char* what, double p, uint64_t seed, uint32_t draw, int64_t cols, Mask& m) {
    if (!(p >= 0.0 && p <= 1.0)) return bad(what, "p is not in [0, 1]");
    if (cols > (int64_t)1 << 34) return bad(what, "too many columns");
    const int kept = (int)std::nearbyint((1.0 - p) * 65536.0);  // K of the header
    for (uint32_t i = 0; i < 10; ++i) {
        m.key[2 * i] = (uint32_t)seed + i * 0x9E3779B9u;
        m.key[2 * i + 1] = (uint32_t)(seed >> 32) + i * 0xBB67AE85u;
    }
    m.draw = draw;
    m.drops = kept < 65536;
    m.limit = (uint32_t)kept << 16;
    m.scale = kept ? (float)(65536.0 / kept) : 1.0f;
    return FSDP_OK;
}

int check_float(const char* what, const char* name, double v) {
    return std::isfinite((float)v) ? FSDP_OK : bad(what, std::string(name) + " is not finite in binary32");
}

int check_aligned(const char* what, const char* name, const void* p, int es) {
    return reinterpret_cast<uintptr_t>(p) % es ? bad(what, std::string(name) + " is not aligned to its element size") : FSDP_OK;
}

int launched(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return FSDP_OK;
    (void)cudaGetLastError();  // reported here, not by the caller's next call
    return set_error(FSDP_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

Mat mat(const void* data, int64_t stride) { return Mat{const_cast<void*>(data), stride}; }

}  // namespace
}  // namespace fsdp

using namespace fsdp;

#define FSDP_TRY(call)               \
    do {                             \
        if (int rc_ = (call)) return rc_; \
    } while (0)

extern "C" {

int fsdp_embedding(int table_dt, const void* table, int64_t table_stride, int64_t vocab, int64_t cols,
                   int index_type, const void* ids, int64_t n_ids, int64_t first_row, double scale, int out_dt,
                   void* out, int64_t out_stride, fsdp_stream_t stream) {
    const char* what = "embedding";
    clear_error();
    FSDP_TRY(check_ids(what, index_type, ids, n_ids, vocab, cols));
    FSDP_TRY(check_size(what, n_ids, cols));
    FSDP_TRY(check_operands(what, cols, {{"table", table, table_stride, table_dt, vocab, false, n_ids == 0},
                                         {"out", out, out_stride, out_dt, n_ids, true, false}}));
    FSDP_TRY(check_float(what, "scale", scale));
    const EmbeddingArgs a = {mat(table, table_stride), mat(out, out_stride), ids, vocab, cols, n_ids, first_row,
                             index_type == FSDP_I64, (float)scale};
    return launched(launch_embedding(table_dt, out_dt, a, stream), what);
}

int fsdp_embedding_grad_workspace(int64_t n_ids, int64_t vocab, int64_t cols, size_t* bytes) {
    const char* what = "embedding_grad_workspace";
    clear_error();
    if (!bytes) return bad(what, "bytes is NULL");
    FSDP_TRY(check_ids(what, FSDP_I64, n_ids > 0 ? &n_ids : nullptr, n_ids, vocab, cols, kMaxGradTokens));
    FSDP_TRY(check_size(what, n_ids, cols));
    *bytes = embedding_grad_most_bytes(n_ids, vocab, cols);
    return FSDP_OK;
}

int fsdp_embedding_grad(int grad_dt, const void* grad_out, int64_t grad_out_stride, int index_type, const void* ids,
                        int64_t n_ids, int64_t first_row, double scale, int accumulate, int table_dt,
                        void* grad_table, int64_t grad_table_stride, int64_t vocab, int64_t cols, void* workspace,
                        size_t workspace_bytes, fsdp_stream_t stream) {
    const char* what = "embedding_grad";
    clear_error();
    FSDP_TRY(check_ids(what, index_type, ids, n_ids, vocab, cols, kMaxGradTokens));
    FSDP_TRY(check_size(what, n_ids, cols));
    FSDP_TRY(check_operands(what, cols, {{"grad_out", grad_out, grad_out_stride, grad_dt, n_ids, false, false},
                                         {"grad_table", grad_table, grad_table_stride, table_dt, vocab, true, false}}));
    FSDP_TRY(check_float(what, "scale", scale));
    FSDP_TRY(check_work(what, workspace, workspace_bytes, embedding_grad_bytes(n_ids, vocab, cols)));
    const EmbeddingGradArgs a = {mat(grad_out, grad_out_stride), mat(grad_table, grad_table_stride), ids, vocab, cols,
                                 n_ids, first_row, index_type == FSDP_I64, accumulate ? 1 : 0, (float)scale, workspace};
    return launched(launch_embedding_grad(grad_dt, table_dt, a, stream), what);
}

int fsdp_dropout(int64_t rows, int64_t cols, int dt, const void* x, int64_t x_stride, const void* residual,
                 int64_t residual_stride, double p, uint64_t seed, uint32_t draw, void* out, int64_t out_stride,
                 fsdp_stream_t stream) {
    const char* what = "dropout";
    clear_error();
    FSDP_TRY(check_size(what, rows, cols));
    FSDP_TRY(check_operands(what, cols, {{"x", x, x_stride, dt, rows, false, false},
                                         {"residual", residual, residual_stride, dt, rows, false, true},
                                         {"out", out, out_stride, dt, rows, true, false}}));
    if (out && rows > 1 && ((out == x && out_stride != x_stride) || (out == residual && out_stride != residual_stride)))
        return bad(what, "out is an input with another stride");
    DropoutArgs a = {rows, cols, mat(x, x_stride), mat(residual, residual_stride), mat(out, out_stride), {}};
    FSDP_TRY(make_mask(what, p, seed, draw, cols, a.mask));
    return launched(launch_dropout(dt, a, stream), what);
}

int fsdp_layer_norm(int64_t rows, int64_t cols, int dt, const void* x, int64_t x_stride, const void* residual,
                    int64_t residual_stride, double p, uint64_t seed, uint32_t draw, int param_dt, const void* weight,
                    const void* bias, double eps, void* hidden, int64_t hidden_stride, void* out, int64_t out_stride,
                    float* mean, float* rstd, fsdp_stream_t stream) {
    const char* what = "layer_norm";
    clear_error();
    FSDP_TRY(check_size(what, rows, cols));
    if (rows >= INT32_MAX) return bad(what, "too many rows");
    FSDP_TRY(check_operands(what, cols, {{"x", x, x_stride, dt, rows, false, false},
                                         {"residual", residual, residual_stride, dt, rows, false, true},
                                         {"weight", weight, 0, param_dt, 1, false, true},
                                         {"bias", bias, 0, param_dt, 1, false, true},
                                         {"hidden", hidden, hidden_stride, dt, rows, true, true},
                                         {"out", out, out_stride, dt, rows, true, false}}));
    if (out && (out == x || out == residual || out == hidden)) return bad(what, "out is another operand's memory");
    if (hidden && (hidden == x || hidden == residual)) return bad(what, "hidden is an input's memory");
    FSDP_TRY(check_aligned(what, "mean", mean, 4));
    FSDP_TRY(check_aligned(what, "rstd", rstd, 4));
    FSDP_TRY(check_float(what, "eps", eps));
    if (eps < 0) return bad(what, "eps is negative");
    NormArgs a = {rows, cols, mat(x, x_stride), mat(residual, residual_stride), mat(hidden, hidden_stride),
                  mat(out, out_stride), param_dt, weight, bias, mean, rstd, (float)eps, {}};
    FSDP_TRY(make_mask(what, p, seed, draw, cols, a.mask));
    return launched(launch_norm(dt, a, stream), what);
}

int fsdp_layer_norm_grad_workspace(int64_t rows, int64_t cols, size_t* bytes) {
    const char* what = "layer_norm_grad_workspace";
    clear_error();
    if (!bytes) return bad(what, "bytes is NULL");
    FSDP_TRY(check_size(what, rows, cols));
    if (rows >= INT32_MAX) return bad(what, "too many rows");
    *bytes = norm_grad_bytes(rows, cols);
    return FSDP_OK;
}

int fsdp_layer_norm_grad(int64_t rows, int64_t cols, int dt, const void* grad_out, int64_t grad_out_stride,
                         const void* grad_hidden, int64_t grad_hidden_stride, const void* hidden,
                         int64_t hidden_stride, const float* mean, const float* rstd, int param_dt, const void* weight,
                         double p, uint64_t seed, uint32_t draw, int accumulate, void* grad_residual,
                         int64_t grad_residual_stride, void* grad_x, int64_t grad_x_stride, int param_grad_dt,
                         void* grad_weight, void* grad_bias, void* workspace, size_t workspace_bytes,
                         fsdp_stream_t stream) {
    const char* what = "layer_norm_grad";
    clear_error();
    FSDP_TRY(check_size(what, rows, cols));
    if (rows >= INT32_MAX) return bad(what, "too many rows");
    FSDP_TRY(check_operands(what, cols, {{"grad_out", grad_out, grad_out_stride, dt, rows, false, false},
                                         {"grad_hidden", grad_hidden, grad_hidden_stride, dt, rows, false, true},
                                         {"hidden", hidden, hidden_stride, dt, rows, false, false},
                                         {"weight", weight, 0, param_dt, 1, false, true},
                                         {"grad_residual", grad_residual, grad_residual_stride, dt, rows, true, true},
                                         {"grad_x", grad_x, grad_x_stride, dt, rows, true, false},
                                         {"grad_weight", grad_weight, 0, param_grad_dt, 1, true, true},
                                         {"grad_bias", grad_bias, 0, param_grad_dt, 1, true, true}}));
    if (grad_x && (grad_x == grad_out || grad_x == hidden || grad_x == grad_hidden || grad_x == grad_residual))
        return bad(what, "grad_x is another operand's memory");
    if (grad_residual && (grad_residual == grad_out || grad_residual == hidden || grad_residual == grad_hidden))
        return bad(what, "grad_residual is an input's memory");
    if (rows > 0 && cols > 0 && (!mean || !rstd)) return bad(what, "mean or rstd is NULL");
    FSDP_TRY(check_aligned(what, "mean", mean, 4));
    FSDP_TRY(check_aligned(what, "rstd", rstd, 4));
    FSDP_TRY(check_work(what, workspace, workspace_bytes, norm_grad_bytes(rows, cols)));
    NormGradArgs a = {rows, cols, mat(grad_out, grad_out_stride), mat(grad_hidden, grad_hidden_stride),
                      mat(hidden, hidden_stride), mat(grad_residual, grad_residual_stride), mat(grad_x, grad_x_stride),
                      mean, rstd, param_dt, weight, grad_weight, grad_bias, accumulate ? 1 : 0, static_cast<float*>(workspace), {}};
    FSDP_TRY(make_mask(what, p, seed, draw, cols, a.mask));
    return launched(launch_norm_grad(dt, param_grad_dt, a, stream), what);
}

}  // extern "C"
