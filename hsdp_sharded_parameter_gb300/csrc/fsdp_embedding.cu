// Embedding lookup with a scale, and its gradient by sorted tokens.
//
// Forward: out[t] = scale * table[ids[t] - first], zeros where the id names
// no row.
//
// Gradient: grad_table[v] = scale * sum of grad_out[t] over the tokens t of
// row v. Three kernels:
//   1. a stable radix sort of (row, token) by one cluster of blocks, while
//      the other blocks write the zeros of the rows no token names;
//   2. sums over chunks of sorted tokens: a warp adds up the gradients of a
//      chunk for a span of 256 columns, writes the rows that lie inside the
//      chunk and leaves the sums of rows that cross its ends;
//   3. the rows that cross chunks: their partial sums added in order.
#include "fsdp_ops.cuh"

namespace fsdp {
namespace {

constexpr int kEmbWarps = 8;

__device__ __forceinline__ int64_t read_id(const void* ids, int wide, int64_t t) {
    return wide ? __ldg(static_cast<const long long*>(ids) + t) : (int64_t)__ldg(static_cast<const int*>(ids) + t);
}

// The row an id names in a table of vocab rows, vocab where it names none.
__device__ __forceinline__ int row_of(int64_t id, int64_t first, int64_t vocab) {
    const uint64_t v = (uint64_t)id - (uint64_t)first;
    return (int)(v < (uint64_t)vocab ? v : (uint64_t)vocab);
}

// ------------------------------------------------------------------ forward

template <typename S, typename D>
__global__ void __launch_bounds__(32 * kEmbWarps) embedding_kernel(EmbeddingArgs a, int64_t spans, int64_t items) {
    const int lane = threadIdx.x & 31;
    for (int64_t it = warp_id(); it < items; it += warp_count()) {
        const int64_t t = it / spans, g = (it - t * spans) * 32 + lane, c = g * kGran;
        const int n = granule_cols(g, a.cols);
        const int64_t row = row_of(read_id(a.ids, a.wide_ids, t), a.first, a.vocab);
        Raw<S> in;
        Raw<D> out;
        zero_raw(in);
        if (row < a.vocab) load_granule(in, static_cast<const S*>(a.table.data) + row * a.table.stride, c, n);
        round_to(row < a.vocab ? widened(in) * all(a.scale) : all(0.0f), out);
        store_span(static_cast<D*>(a.out.data) + t * a.out.stride + c, out, n, lane);
    }
}

// ------------------------------------------------- gradient: sort and zeros

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kMaxBins = 256;
constexpr int kSortCluster = 8;

// Workspace: the number of tokens that name a row, two buffers of sorted rows
// and tokens, and the partial sums of rows that cross chunks ([chunk] for one
// that began in an earlier chunk, [nchunks + chunk] for one that begins in
// it), stride columns each.
struct GradWork {
    int* count;
    int *rows[2], *toks[2];
    float* part;
    int64_t stride;
    int chunk, nchunks;
};

int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

// Tokens of a chunk.
int chunk_tokens(int64_t) { return 32; }

GradWork grad_work(void* work, int64_t n, int64_t cols, size_t* bytes) {
    GradWork w;
    char* p = static_cast<char*>(work);
    size_t at = 256;
    w.count = reinterpret_cast<int*>(p);
    for (int i = 0; i < 2; ++i) {
        w.rows[i] = reinterpret_cast<int*>(p + at);
        at += up(n * 4, 256);
        w.toks[i] = reinterpret_cast<int*>(p + at);
        at += up(n * 4, 256);
    }
    w.chunk = chunk_tokens(n);
    w.nchunks = (int)((n + w.chunk - 1) / w.chunk);
    w.stride = up(cols, kGran);
    w.part = reinterpret_cast<float*>(p + at);
    at += (size_t)2 * w.nchunks * w.stride * 4;
    if (bytes) *bytes = at;
    return w;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_read(const uint32_t* p, int rank) {
    uint32_t a = (uint32_t)__cvta_generic_to_shared(p), v;
    asm volatile("{\n.reg .u32 r;\nmapa.shared::cluster.u32 r, %1, %2;\nld.shared::cluster.u32 %0, [r];\n}"
                 : "=r"(v)
                 : "r"(a), "r"(rank)
                 : "memory");
    return v;
}

struct SortSmem {
    uint32_t hist[kSortWarps][kMaxBins];
    uint32_t total[kMaxBins + 1];  // of this block; [kMaxBins]: tokens that name a row
    uint32_t base[kMaxBins];
    uint32_t scan[kMaxBins / 32];
};

// One pass over this block's part of the tokens: their digit's counts, the
// places the counts of all blocks give them, and the move. Tokens keep their
// order within a digit: a warp's tokens are consecutive and it ranks 32 of
// them at a time by the lanes that hold the same digit.
template <typename Read>
__device__ void sort_pass(SortSmem& sm, int64_t n, int blocks, int rank, int shift, int bits, bool first,
                          int64_t vocab, Read read, int* rows_out, int* toks_out) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bins = 1 << bits;
    const int64_t per = ((n + blocks - 1) / blocks + kSortWarps * 32 - 1) / (kSortWarps * 32) * 32;  // of a warp
    const int64_t lo = (rank * (int64_t)kSortWarps + warp) * per;
    const int64_t hi = lo + per < n ? lo + per : n;
    for (int i = lane; i < bins; i += 32) sm.hist[warp][i] = 0;
    if (first && tid == 0) sm.total[kMaxBins] = 0;
    __syncthreads();
    int named = 0;
    for (int64_t i = lo; i < hi; i += 32) {
        int row = 0, tok;
        const bool on = i + lane < hi;
        if (on) read(i + lane, row, tok);
        const int d = on ? (row >> shift) & (bins - 1) : bins;
        const unsigned peers = __match_any_sync(kFull, d);
        if (on && lane == __ffs(peers) - 1) sm.hist[warp][d] += __popc(peers);
        if (first) named += __popc(__ballot_sync(kFull, on && row < vocab));
        __syncwarp();
    }
    if (first && lane == 0 && named) atomicAdd(&sm.total[kMaxBins], (uint32_t)named);
    __syncthreads();
    if (tid < bins) {
        uint32_t s = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t t = sm.hist[w][tid];
            sm.hist[w][tid] = s;
            s += t;
        }
        sm.total[tid] = s;
    }
    cluster_sync();
    uint32_t before = 0, all = 0, incl = 0;
    if (tid < kMaxBins) {
        if (tid < bins)
            for (int r = 0; r < blocks; ++r) {
                const uint32_t t = cluster_read(&sm.total[tid], r);
                if (r < rank) before += t;
                all += t;
            }
        incl = all;
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t t = __shfl_up_sync(kFull, incl, d);
            if (lane >= d) incl += t;
        }
        if (lane == 31) sm.scan[warp] = incl;
    }
    __syncthreads();
    if (tid < kMaxBins) {
        for (int w = 0; w < warp; ++w) incl += sm.scan[w];
        sm.base[tid] = incl - all + before;
    }
    __syncthreads();
    for (int64_t i = lo; i < hi; i += 32) {
        int row = 0, tok = 0;
        const bool on = i + lane < hi;
        if (on) read(i + lane, row, tok);
        const int d = on ? (row >> shift) & (bins - 1) : bins;
        const unsigned peers = __match_any_sync(kFull, d);
        if (on) {
            const uint32_t at = sm.base[d] + sm.hist[warp][d] + __popc(peers & ((1u << lane) - 1));
            rows_out[at] = row;
            toks_out[at] = tok;
        }
        __syncwarp();
        if (on && lane == __ffs(peers) - 1) sm.hist[warp][d] += __popc(peers);
        __syncwarp();
    }
    // the moved tokens reach the cluster's other blocks, and the totals may go
    cluster_sync();
}

// Blocks 0 .. blocks-1, one cluster, sort; the others write the zeros of the
// rows that no token names, each for a range of rows whose tokens it looks
// for among all ids.
template <typename D>
__global__ void __launch_bounds__(kSortThreads)
    embedding_sort_kernel(EmbeddingGradArgs a, GradWork w, int blocks, int passes, int bits) {
    extern __shared__ uint32_t raw_smem[];
    if ((int)blockIdx.x < blocks) {
        SortSmem& sm = *reinterpret_cast<SortSmem*>(raw_smem);
        const int rank = blockIdx.x;
        for (int p = 0; p < passes; ++p) {
            int *ro = w.rows[p & 1], *to = w.toks[p & 1];
            if (p == 0) {
                sort_pass(sm, a.n, blocks, rank, 0, bits, true, a.vocab,
                          [&](int64_t i, int& row, int& tok) {
                              row = row_of(read_id(a.ids, a.wide_ids, i), a.first, a.vocab);
                              tok = (int)i;
                          },
                          ro, to);
                if (rank == 0 && threadIdx.x == 0) {
                    uint32_t c = 0;
                    for (int r = 0; r < blocks; ++r) c += cluster_read(&sm.total[kMaxBins], r);
                    *w.count = (int)c;
                }
            } else {
                const int *ri = w.rows[(p & 1) ^ 1], *ti = w.toks[(p & 1) ^ 1];
                sort_pass(sm, a.n, blocks, rank, p * bits, bits, false, a.vocab,
                          [&](int64_t i, int& row, int& tok) {
                              row = __ldcg(ri + i);
                              tok = __ldcg(ti + i);
                          },
                          ro, to);
            }
        }
        cluster_sync();  // no block leaves while another reads its counts
        return;
    }
    // zeros
    const int64_t nz = gridDim.x - blocks, z = blockIdx.x - blocks;
    const int64_t r0 = a.vocab * z / nz, r1 = a.vocab * (z + 1) / nz;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int64_t kRows = 32 * 4096;  // rows whose bits fit the block's shared memory
    for (int64_t b = r0; b < r1; b += kRows) {
        const int64_t e = b + kRows < r1 ? b + kRows : r1;
        for (int i = tid; i < (e - b + 31) / 32; i += kSortThreads) raw_smem[i] = 0;
        __syncthreads();
        for (int64_t i = tid; i < a.n; i += kSortThreads) {
            const int64_t v = row_of(read_id(a.ids, a.wide_ids, i), a.first, a.vocab);
            if (v >= b && v < e) atomicOr(&raw_smem[(v - b) >> 5], 1u << ((v - b) & 31));
        }
        __syncthreads();
        const Raw<D> none = {};
        const int64_t spans = (a.cols + kSpan - 1) / kSpan;
        for (int64_t it = warp; it < (e - b) * spans; it += kSortWarps) {
            const int64_t r = it / spans, g = (it - r * spans) * 32 + lane;
            if (raw_smem[r >> 5] >> (r & 31) & 1) continue;
            store_span(static_cast<D*>(a.table.data) + (b + r) * a.table.stride + g * kGran, none,
                       granule_cols(g, a.cols), lane);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------ gradient: sums

// Scales a row's sums, adds what the table holds where the caller wants it,
// rounds and stores them.
template <typename D>
__device__ __forceinline__ void store_row(const EmbeddingGradArgs& a, int row, int64_t g, Cols x, int lane) {
    const int n = granule_cols(g, a.cols);
    D* p = static_cast<D*>(a.table.data) + row * a.table.stride + g * kGran;
    Raw<D> r;
    x = x * all(a.scale);
    if (a.accumulate) {
        load_granule(r, p - g * kGran, g * kGran, n);
        x = x + widened(r);
        __syncwarp();  // a shifted load reads its neighbours' blocks
    }
    round_to(x, r);
    store_span(p, r, n, lane);
}

__device__ __forceinline__ void store_part(float* p, const Cols& x) {
    float4* q = reinterpret_cast<float4*>(p);
    q[0] = make_float4(x.p[0].x, x.p[0].y, x.p[1].x, x.p[1].y);
    q[1] = make_float4(x.p[2].x, x.p[2].y, x.p[3].x, x.p[3].y);
}
__device__ __forceinline__ Cols load_part(const float* p) {
    const float4 u = __ldcg(reinterpret_cast<const float4*>(p)), v = __ldcg(reinterpret_cast<const float4*>(p) + 1);
    return {{make_float2(u.x, u.y), make_float2(u.z, u.w), make_float2(v.x, v.y), make_float2(v.z, v.w)}};
}

template <typename S, typename D>
__global__ void __launch_bounds__(32 * kEmbWarps)
    embedding_sum_kernel(EmbeddingGradArgs a, GradWork w, const int* rows, const int* toks, int64_t spans) {
    constexpr int kU = 4;
    const int lane = threadIdx.x & 31;
    const int64_t it = warp_id();
    const int64_t chunk = it / spans, span = it - chunk * spans;
    const int count = __ldg(w.count);
    const int64_t lo = chunk * w.chunk;
    if (lo >= count) return;
    const int hi = (int)(lo + w.chunk < count ? lo + w.chunk : count);
    const int64_t g = span * 32 + lane, c = g * kGran;
    const int n = granule_cols(g, a.cols);
    const int prev = lo > 0 ? __ldg(rows + lo - 1) : -1;
    const int next = hi < count ? __ldg(rows + hi) : -1;
    Cols acc = all(0.0f);
    int cur = -1;
    bool open = false;  // cur began in an earlier chunk
    for (int b = (int)lo; b < hi; b += 32) {
        const int m = hi - b < 32 ? hi - b : 32;
        const int my_row = lane < m ? __ldg(rows + b + lane) : -1, my_tok = lane < m ? __ldg(toks + b + lane) : 0;
        for (int j = 0; j < m; j += kU) {
            Raw<S> in[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int64_t t = __shfl_sync(kFull, my_tok, (j + u) & 31);
                if (j + u < m) load_granule(in[u], static_cast<const S*>(a.grad.data) + t * a.grad.stride, c, n);
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (j + u >= m) break;
                const int row = __shfl_sync(kFull, my_row, (j + u) & 31);
                const Cols x = widened(in[u]);
                if (row != cur) {
                    if (cur >= 0) {
                        if (!open)
                            store_row<D>(a, cur, g, acc, lane);
                        else if (n)
                            store_part(w.part + chunk * w.stride + c, acc);
                    }
                    open = cur < 0 && row == prev;
                    cur = row;
                    acc = x;
                } else {
                    acc = acc + x;
                }
            }
        }
    }
    if (open) {
        if (n) store_part(w.part + chunk * w.stride + c, acc);
    } else if (cur == next) {
        if (n) store_part(w.part + (w.nchunks + chunk) * w.stride + c, acc);
    } else {
        store_row<D>(a, cur, g, acc, lane);
    }
}

// Block (span, y): the rows that cross chunk ends y + 1, y + 1 + gridDim.y,
// ... and began in the chunk before that end.
template <typename D>
__global__ void __launch_bounds__(32 * kEmbWarps)
    embedding_join_kernel(EmbeddingGradArgs a, GradWork w, const int* rows) {
    __shared__ float part[kEmbWarps][kSpan];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t g = (int64_t)blockIdx.x * 32 + lane, c = g * kGran;
    const int n = granule_cols(g, a.cols);
    const int count = __ldg(w.count);
    for (int64_t b = blockIdx.y + 1; b * w.chunk < count; b += gridDim.y) {
        const int row = __ldg(rows + b * w.chunk);
        if (__ldg(rows + b * w.chunk - 1) != row) continue;
        if (b > 1 && __ldg(rows + (b - 1) * w.chunk - 1) == row) continue;
        int lo = (int)(b * w.chunk), hi = count;  // the row's last token: rows[lo] == row, rows[hi] > row
        while (hi - lo > 1) {
            const int mid = lo + (hi - lo) / 2;
            if (__ldg(rows + mid) == row)
                lo = mid;
            else
                hi = mid;
        }
        // partial sums b - 1 (its tail), b, ..., last, a share for each warp
        const int64_t last = lo / w.chunk, parts = last - b + 2;
        const int64_t p0 = parts * warp / kEmbWarps, p1 = parts * (warp + 1) / kEmbWarps;
        Cols acc = all(0.0f);
        if (n)
            for (int64_t p = p0; p < p1; ++p)
                acc = acc + load_part(w.part + (p == 0 ? w.nchunks + b - 1 : b - 1 + p) * w.stride + c);
        store_part(&part[warp][lane * kGran], acc);
        __syncthreads();
        if (warp == 0) {
            for (int q = 1; q < kEmbWarps; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc.set(e, acc.get(e) + part[q][lane * kGran + e]);
            store_row<D>(a, row, g, acc, lane);
        }
        __syncthreads();
    }
}

template <typename S, typename D>
cudaError_t embedding_grad(const EmbeddingGradArgs& a, cudaStream_t s) {
    const GradWork w = grad_work(a.work, a.n, a.cols, nullptr);
    int need = 1;
    while (((int64_t)1 << need) <= a.vocab) ++need;  // bits of the values 0 .. vocab
    const int passes = (need + 7) / 8, bits = (need + passes - 1) / passes;
    const int blocks = a.n <= 8192 ? 1 : kSortCluster;
    const int64_t spans = (a.cols + kSpan - 1) / kSpan;
    // one block of zeros per SM beside the sort
    const int zeros = a.accumulate ? 0 : sm_count();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks + (zeros + blocks - 1) / blocks * blocks);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = sizeof(SortSmem);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = blocks;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, embedding_sort_kernel<D>, a, w, blocks, passes, bits);
    if (e != cudaSuccess) return e;
    count_launch();
    if (a.n == 0) return cudaSuccess;
    const int *rows = w.rows[(passes - 1) & 1], *toks = w.toks[(passes - 1) & 1];
    const int64_t items = w.nchunks * spans;
    embedding_sum_kernel<S, D><<<(unsigned)((items + kEmbWarps - 1) / kEmbWarps), 32 * kEmbWarps, 0, s>>>(a, w, rows, toks, spans);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (w.nchunks > 1) {
        const int64_t y = w.nchunks - 1 < 64 ? w.nchunks - 1 : 64;
        embedding_join_kernel<D><<<dim3((unsigned)spans, (unsigned)y), 32 * kEmbWarps, 0, s>>>(a, w, rows);
        count_launch();
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace

size_t embedding_grad_bytes(int64_t n, int64_t vocab, int64_t cols) {
    size_t bytes = 0;
    grad_work(nullptr, n, cols, &bytes);
    return bytes;
}

cudaError_t launch_embedding(int table_dt, int out_dt, const EmbeddingArgs& a, cudaStream_t s) {
    if (a.n == 0 || a.cols == 0) return cudaSuccess;
    const int64_t spans = (a.cols + kSpan - 1) / kSpan, items = spans * a.n;
    const int64_t blocks = (items + kEmbWarps - 1) / kEmbWarps;
    const unsigned grid = (unsigned)(blocks < 0x7fffffff ? blocks : 0x7fffffff);
    const int block = 32 * kEmbWarps;
    if (table_dt == FSDP_F32 && out_dt == FSDP_F32)
        embedding_kernel<float, float><<<grid, block, 0, s>>>(a, spans, items);
    else if (table_dt == FSDP_F32)
        embedding_kernel<float, uint16_t><<<grid, block, 0, s>>>(a, spans, items);
    else if (out_dt == FSDP_F32)
        embedding_kernel<uint16_t, float><<<grid, block, 0, s>>>(a, spans, items);
    else
        embedding_kernel<uint16_t, uint16_t><<<grid, block, 0, s>>>(a, spans, items);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_embedding_grad(int grad_dt, int table_dt, const EmbeddingGradArgs& a, cudaStream_t s) {
    if (a.vocab == 0 || a.cols == 0) return cudaSuccess;
    if (a.accumulate && a.n == 0) return cudaSuccess;
    if (grad_dt == FSDP_F32) return table_dt == FSDP_F32 ? embedding_grad<float, float>(a, s) : embedding_grad<float, uint16_t>(a, s);
    return table_dt == FSDP_F32 ? embedding_grad<uint16_t, float>(a, s) : embedding_grad<uint16_t, uint16_t>(a, s);
}

}  // namespace fsdp
