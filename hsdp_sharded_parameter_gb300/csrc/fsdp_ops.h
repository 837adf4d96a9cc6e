// Launch interface of the training operators (embedding, dropout, layer norm,
// gated feed-forward, orthogonalised updates): what the C-ABI entry points (fsdp_ops_capi.cpp) hand to the kernels
// once the arguments are checked. Not installed.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "hsdp_fsdp.h"

namespace fsdp {

// A matrix in device memory: element (r, c) at data[r * stride + c].
struct Mat {
    void* data;
    int64_t stride;
};

// Whether a matrix's rows all start on the 16-byte grid.
inline bool on_grid(const Mat& m, int es) {
    return reinterpret_cast<uintptr_t>(m.data) % 16 == 0 && m.stride * es % 16 == 0;
}

// The mask of a dropout: the generator's round keys (ten pairs, worked out
// once on the host: as kernel arguments they are operands of the rounds'
// instructions), and whether a 16-bit half is kept: half << 16 < limit.
struct Mask {
    uint32_t key[20];
    uint32_t draw, limit;
    int drops;    // 0: everything is kept as it is
    float scale;  // of what is kept
};

struct EmbeddingArgs {
    Mat table, out;
    const void* ids;
    int64_t vocab, cols, n, first;
    int wide_ids;  // 1: 64-bit ids
    float scale;
};

struct EmbeddingGradArgs {
    Mat grad, table;
    const void* ids;
    int64_t vocab, cols, n, first;
    int wide_ids, accumulate;
    float scale;
    void* work;
};

struct DropoutArgs {
    int64_t rows, cols;
    Mat x, res, out;  // res.data may be nullptr
    Mask mask;
};

struct NormArgs {
    int64_t rows, cols;
    Mat x, res, hidden, out;  // res.data, hidden.data may be nullptr
    int param_dt;
    const void *weight, *bias;
    float *mean, *rstd;
    float eps;
    Mask mask;
};

struct NormGradArgs {
    int64_t rows, cols;
    Mat grad, grad_hidden, hidden, grad_res, grad_x;
    const float *mean, *rstd;
    int param_dt;
    const void* weight;
    void *grad_weight, *grad_bias;
    int accumulate;
    float* work;
    Mask mask;
};

struct FfnArgs {
    int64_t tokens, hidden, inner;
    int act;
    Mat x, w_gate, w_up, w_down, gate, up, out;  // gate.data, up.data may both be nullptr
    char* work;
};

struct FfnGradArgs {
    int64_t tokens, hidden, inner;
    int act, accumulate;
    Mat grad, x, w_gate, w_up, w_down, gate, up, grad_x, grad_gate, grad_up, grad_down;
    char* work;
};

struct OrthoArgs {
    int64_t rows, cols;
    Mat x, out;
    int steps;
    float a, b, c, scale;
    double eps;
    char* work;
};

// SMs of the current device.
int sm_count();
// Lets a kernel take up to `bytes` of dynamic shared memory on the current
// device; `done` remembers the devices it was said for.
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done);

// The gradient's sort numbers tokens in 32 bits and steps past the last one by
// up to a tile.
constexpr int64_t kMaxGradTokens = ((int64_t)1 << 31) - (1 << 14) - 1;
// Workspace of a call, and one that serves every call of up to n tokens.
size_t embedding_grad_bytes(int64_t n, int64_t vocab, int64_t cols);
size_t embedding_grad_most_bytes(int64_t n, int64_t vocab, int64_t cols);
size_t norm_grad_bytes(int64_t rows, int64_t cols);

size_t ffn_bytes(const FfnArgs& a);
size_t ffn_most_bytes(int64_t tokens, int64_t hidden, int64_t inner, bool aligned);
size_t ffn_grad_bytes(const FfnGradArgs& a);
size_t ffn_grad_most_bytes(int64_t tokens, int64_t hidden, int64_t inner, bool aligned);
size_t ortho_bytes(int64_t rows, int64_t cols);
// The largest singular value that any of the steps may start from, those of the
// first iterate being at most 1; the scales allow for kMostReach.
double ortho_reach(int steps, double a, double b, double c);
constexpr double kMostReach = 8.0;

// Each enqueues its kernels (counting them) and returns the launches' error.
cudaError_t launch_embedding(int table_dt, int out_dt, const EmbeddingArgs& a, cudaStream_t s);
cudaError_t launch_embedding_grad(int grad_dt, int table_dt, const EmbeddingGradArgs& a, cudaStream_t s);
cudaError_t launch_dropout(int dt, const DropoutArgs& a, cudaStream_t s);
cudaError_t launch_norm(int dt, const NormArgs& a, cudaStream_t s);
cudaError_t launch_norm_grad(int dt, int param_grad_dt, const NormGradArgs& a, cudaStream_t s);
cudaError_t launch_ffn(const FfnArgs& a, cudaStream_t s);
cudaError_t launch_ffn_grad(int param_grad_dt, const FfnGradArgs& a, cudaStream_t s);
cudaError_t launch_ortho(int dt, const OrthoArgs& a, cudaStream_t s);
// Whether a wait inside an operator's kernel has run out since the last
// question, after what the stream holds.
cudaError_t ffn_gave_up(int* value, cudaStream_t s);
cudaError_t ortho_gave_up(int* value, cudaStream_t s);

}  // namespace fsdp
