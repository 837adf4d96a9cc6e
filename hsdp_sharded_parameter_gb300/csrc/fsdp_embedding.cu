// Embedding lookup with a scale, and its gradient by sorted tokens.
//
// Forward: out[t] = scale * table[ids[t] - first], zeros where the id names
// no row.
//
// Gradient: grad_table[v] = scale * sum of grad_out[t] over the tokens t of
// row v. One kernel for few tokens (below); else three, each launched while the
// one before it runs:
//   1. a stable radix sort of (row, token) by one cluster of blocks;
//   2. sums: a warp adds up the gradients of a chunk of sorted tokens for a
//      span of 256 columns, writes the rows that lie inside the chunk, leaves
//      partial sums of those that cross its ends, and lists these; it also
//      marks the rows that a token names;
//   3. the partial sums of the listed rows, added in order, and beside them
//      the zeros of the rows that are not marked.
#include <algorithm>

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

// The table's columns of a granule of an aligned row. Rows are looked up again,
// so they are not marked for early eviction as streams are.
template <typename T>
__device__ __forceinline__ void load_table(Raw<T>& r, const T* row, int64_t c, int n) {
    if (n == 0) return;
    const uint4* q = reinterpret_cast<const uint4*>(row + c);
#pragma unroll
    for (int v = 0; v < Raw<T>::kVec; ++v) put(r.w + 4 * v, ld_reuse(q + v));
}

// A warp takes up to kEmbSpans neighbouring spans of 256 columns of a token:
// 32768 tokens of 8192 bf16 take 116 us with 8, 121 with 4 and 141 with 2; to
// fp32 268, 250 and 225.
template <typename S, typename D>
constexpr int kEmbSpans = sizeof(D) == 4 ? 2 : (sizeof(S) == 4 ? 4 : 8);

template <typename S, typename D, bool kAligned>
__global__ void __launch_bounds__(32 * kEmbWarps) embedding_kernel(EmbeddingArgs a, int64_t steps, int per, int64_t items) {
    // rows off the 16-byte grid come in through shared memory
    __shared__ uint4 staged[kAligned ? 1 : kEmbWarps][kAligned ? 1 : kEmbSpans<S, D>][kAligned ? 1 : kSlot<false, S>];
    const int lane = threadIdx.x & 31;
    uint4(*const mine)[kAligned ? 1 : kSlot<false, S>] = staged[kAligned ? 0 : threadIdx.x >> 5];
    for (int64_t it = warp_id(); it < items; it += warp_count()) {
        const int64_t t = it / steps, g0 = (it - t * steps) * (per * 32) + lane, c0 = (g0 - lane) * kGran;
        const int64_t row = row_of(read_id(a.ids, a.wide_ids, t), a.first, a.vocab);
        const bool named = row < a.vocab;
        const S* from = static_cast<const S*>(a.table.data) + row * a.table.stride;
        D* to = static_cast<D*>(a.out.data) + t * a.out.stride;
        const int left = (int)(a.cols - c0 < per * kSpan ? a.cols - c0 : per * kSpan);
        Raw<S> in[kEmbSpans<S, D>];
#pragma unroll
        for (int u = 0; u < kEmbSpans<S, D>; ++u) {
            if (!named || u >= per) break;
            if constexpr (kAligned)
                load_table(in[u], from, (g0 + u * 32) * kGran, granule_cols(g0 + u * 32, a.cols));
            else
                span_fetch<false, true>(mine[u], from + c0, u * kSpan, left, lane);  // rows are looked up again
        }
        if constexpr (!kAligned) {
            async_commit();
            async_wait<0>();
            __syncwarp();
        }
#pragma unroll
        for (int u = 0; u < kEmbSpans<S, D>; ++u) {
            if (u * kSpan >= left) break;
            const int64_t g = g0 + u * 32;
            if constexpr (!kAligned)
                if (named) span_read<false>(in[u], mine[u], from + c0, u * kSpan, lane);
            Raw<D> r;
            round_to(named ? widened(in[u]) * all(a.scale) : all(0.0f), r);
            store_cols<kAligned>(to + g * kGran, r, granule_cols(g, a.cols), lane);
        }
        if constexpr (!kAligned) __syncwarp();  // before the next spans come in
    }
}

// Narrow rows of grans granules, items granules in all.
template <typename S, typename D, bool kAligned>
__global__ void __launch_bounds__(32 * kEmbWarps) embedding_narrow_kernel(EmbeddingArgs a, uint32_t grans, uint32_t items) {
    const uint32_t i0 = blockIdx.x * (kNarrow * blockDim.x) + threadIdx.x;
    Raw<S> in[kNarrow];
    bool named[kNarrow];
#pragma unroll
    for (int u = 0; u < kNarrow; ++u) {
        const uint32_t i = i0 + u * blockDim.x, t = i / grans, g = i - t * grans;
        const int64_t row = i < items ? row_of(read_id(a.ids, a.wide_ids, t), a.first, a.vocab) : a.vocab;
        named[u] = row < a.vocab;
        if (named[u])
            load_cols<kAligned>(in[u], static_cast<const S*>(a.table.data) + row * a.table.stride, g * kGran, granule_cols((int64_t)g, a.cols));
    }
#pragma unroll
    for (int u = 0; u < kNarrow; ++u) {
        const uint32_t i = i0 + u * blockDim.x, t = i / grans, g = i - t * grans;
        if (i >= items) break;
        Raw<D> r;
        round_to(named[u] ? widened(in[u]) * all(a.scale) : all(0.0f), r);
        store_granule(static_cast<D*>(a.out.data) + t * a.out.stride + g * kGran, r, granule_cols((int64_t)g, a.cols));
    }
}

// ------------------------------------------------- gradient: the sort

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kMaxBits = 9;      // of a digit: the counts of 32 warps take half the shared memory
constexpr int kSortCluster = 8;
constexpr int kKeep = 8;         // tokens of a lane at a time
constexpr int kTile = kSortThreads * kKeep;
static_assert(kMaxGradTokens + 2 * kTile <= INT32_MAX, "a token's number and a tile fit an int");
constexpr int kFewTokens = 512;  // summed without a sort

// A row whose tokens lie in chunks first, first + 1, ..., first + more.
struct Crossing {
    int row, first, more, unused;
};

// Workspace: how many tokens name a row and how many rows cross chunks, two
// buffers of sorted tokens, the marked rows, the rows that cross, and their partial
// sums ([chunk] for a row that began in an earlier chunk, [nchunks + chunk]
// for one that begins in it), stride columns each.
struct GradWork {
    int *count, *crossings;
    int2* sorted[2];  // (row, token)
    uint32_t* marks;  // a bit for each row
    Crossing* cross;
    float* part;
    int64_t stride;
    int chunk, nchunks;
};

int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

// Tokens of a chunk: few while that gives no more warps than the GPU holds at
// once (the fewer, the sooner the longest is done) and no long lists of parts
// for rows of many tokens (57970 tokens, most in three rows of 16 columns: 42 us
// with chunks of 8, 37 with 32), else 32.
struct ChunkRule {
    int64_t most8, most16;  // tokens up to which a chunk has 8 and 16
};
ChunkRule chunk_rule(int64_t cols) {
    const int64_t spans = (cols + kSpan - 1) / kSpan, warps = 64 * (int64_t)sm_count();
    if (spans == 0) return {4096, 16384};
    return {std::min<int64_t>(4096, 8 * warps / spans), std::min<int64_t>(16384, 16 * warps / spans)};
}
int chunk_tokens(int64_t n, int64_t cols) {
    const ChunkRule r = chunk_rule(cols);
    return n <= r.most8 ? 8 : (n <= r.most16 ? 16 : 32);
}

GradWork grad_work(void* work, int64_t n, int64_t vocab, int64_t cols, size_t* bytes) {
    GradWork w;
    char* p = static_cast<char*>(work);
    size_t at = 256;
    w.count = reinterpret_cast<int*>(p);
    w.crossings = w.count + 1;
    for (int i = 0; i < 2; ++i) {
        w.sorted[i] = reinterpret_cast<int2*>(p + at);
        at += up(n * 8, 256);
    }
    w.marks = reinterpret_cast<uint32_t*>(p + at);
    at += up((vocab + 31) / 32 * 4, 256);
    w.chunk = chunk_tokens(n, cols);
    w.nchunks = (int)((n + w.chunk - 1) / w.chunk);
    w.cross = reinterpret_cast<Crossing*>(p + at);
    at += up((int64_t)w.nchunks * sizeof(Crossing), 256);
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

// Shared memory of the sort: a tile of tokens in their new order, each warp's
// count of each digit and the lanes that hold it (rows of an odd length, so
// that warps and digits spread over the banks), the block's counts, where each
// digit's tokens of this block go, and where they begin in the tile.
struct SortSmem {
    int2* tile;
    uint32_t *hist, *lanes, *total, *base, *start, *scan;
    int pitch;
    __device__ SortSmem(void* p, int bins) : pitch(bins | 1) {
        tile = static_cast<int2*>(p);
        hist = reinterpret_cast<uint32_t*>(tile + kTile);
        lanes = hist + kSortWarps * pitch;
        total = lanes + kSortWarps * pitch;
        base = total + bins + 1;  // total[bins]: the block's tokens that name a row
        start = base + bins;
        scan = start + bins;
    }
    static size_t bytes(int bins) {
        return 8 * kTile + 4 * (size_t)(2 * kSortWarps * (bins | 1) + 3 * bins + 1 + 2 * kSortWarps);
    }
};

// The sums of the block's threads' two values before this one.
__device__ __forceinline__ uint2 block_scan(const SortSmem& sm, uint2 v, int lane, int warp) {
    uint2 incl = v;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const uint32_t x = __shfl_up_sync(kFull, incl.x, s), y = __shfl_up_sync(kFull, incl.y, s);
        if (lane >= s) {
            incl.x += x;
            incl.y += y;
        }
    }
    if (lane == 31) {
        sm.scan[2 * warp] = incl.x;
        sm.scan[2 * warp + 1] = incl.y;
    }
    __syncthreads();
    const uint32_t x = __reduce_add_sync(kFull, lane < warp ? sm.scan[2 * lane] : 0);
    const uint32_t y = __reduce_add_sync(kFull, lane < warp ? sm.scan[2 * lane + 1] : 0);
    return make_uint2(x + incl.x - v.x, y + incl.y - v.y);
}

// A digit's counts before each warp, and their total: a thread adds down a
// column.
__device__ __forceinline__ uint32_t column_sums(const SortSmem& sm, int d) {
    uint32_t sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = sm.hist[w * sm.pitch + d];
        sm.hist[w * sm.pitch + d] = sum;
        sum += c;
    }
    return sum;
}

// One pass over this block's part of the tokens: its digits' counts, the
// places that the counts of all blocks give them, and the move. Tokens keep
// their order within a digit: a warp's tokens of a tile are consecutive, and
// it ranks 32 of them at a time by the lanes that hold the same digit, which
// meet in a word of shared memory (a vote for each bit, or a match over the
// warp, is 1400 cycles and more for a step of 32 warps). A tile is put in order in shared
// memory and written from there, neighbours to neighbouring places.
__device__ __forceinline__ void sort_pass(const EmbeddingGradArgs& a, const SortSmem& sm, int blocks, int rank, int shift,
                                          int bits, const int2* in, int2* out) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bins = 1 << bits, n = (int)a.n, per = (n + blocks - 1) / blocks;
    const int64_t from = (int64_t)rank * per;
    const int lo = (int)(from < n ? from : n), hi = from + per < n ? (int)(from + per) : n;
    const bool one = hi - lo <= kTile;
    uint32_t* const hist = sm.hist + warp * sm.pitch;
    uint32_t* const lanes = sm.lanes + warp * sm.pitch;
    int2 tok[kKeep];
    uint32_t before[kKeep];  // the warp's tokens of the same digit before this one
    int steps = 0;           // of 32 tokens, for each warp
    // a lane's tokens of the tile at b, -1 where there is none
    auto load = [&](int b) {
        steps = hi - b < kTile ? (hi - b + kSortThreads - 1) / kSortThreads : kKeep;
#pragma unroll
        for (int k = 0; k < kKeep; ++k) {
            const int i = b + (warp * steps + k) * 32 + lane;
            tok[k] = make_int2(-1, i);
            if (k < steps && i < hi) {
                if (in)
                    tok[k] = __ldcg(in + i);
                else
                    tok[k].x = row_of(read_id(a.ids, a.wide_ids, i), a.first, a.vocab);
            }
        }
    };
    auto clear = [&] {
        for (int i = tid; i < kSortWarps * sm.pitch; i += kSortThreads) sm.hist[i] = sm.lanes[i] = 0;
        __syncthreads();
    };
    auto count = [&] {
        int named = 0;
#pragma unroll
        for (int k = 0; k < kKeep; ++k)
            if (k < steps) {
                const bool on = tok[k].x >= 0;
                const int d = (tok[k].x >> shift) & (bins - 1);
                if (on) atomicOr(lanes + d, 1u << lane);
                __syncwarp();
                const uint32_t peers = on ? lanes[d] : 0, seen = on ? hist[d] : 0;
                __syncwarp();
                if (on && lane == __ffs(peers) - 1) {
                    hist[d] = seen + __popc(peers);
                    lanes[d] = 0;
                }
                __syncwarp();
                before[k] = seen + __popc(peers & ((1u << lane) - 1));
                named += on && tok[k].x < a.vocab;
            }
        return named;
    };

    if (one) load(lo);
    if (tid == 0) sm.total[bins] = 0;
    clear();
    int named = 0;
#pragma unroll 1
    for (int b = lo; b < hi; b += kTile) {
        if (!one) load(b);
        named += count();
    }
    named = __reduce_add_sync(kFull, named);
    if (lane == 0 && named) atomicAdd(&sm.total[bins], (uint32_t)named);
    __syncthreads();
    uint32_t mine = 0;  // the digit's tokens in the tile at hand
    if (tid < bins) sm.total[tid] = mine = column_sums(sm, tid);
    cluster_sync();
    // the digit's tokens in all blocks and in those before this one, and the scan over digits
    uint32_t below = 0, sum = 0;
    if (tid < bins)
#pragma unroll
        for (int r = 0; r < kSortCluster; ++r) {
            const uint32_t t = r < blocks ? cluster_read(&sm.total[tid], r) : 0;
            if (r < rank) below += t;
            sum += t;
        }
    const uint2 at = block_scan(sm, make_uint2(sum, mine), lane, warp);
    if (tid < bins) {
        sm.base[tid] = at.x + below;
        sm.start[tid] = at.y;
    }
    __syncthreads();
#pragma unroll 1
    for (int b = lo; b < hi; b += kTile) {
        if (!one) {
            load(b);
            clear();
            count();
            __syncthreads();
            if (tid < bins) mine = column_sums(sm, tid);
            const uint32_t begin = block_scan(sm, make_uint2(0, mine), lane, warp).y;
            if (tid < bins) sm.start[tid] = begin;
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < kKeep; ++k)
            if (k < steps && tok[k].x >= 0) {
                const int d = (tok[k].x >> shift) & (bins - 1);
                sm.tile[sm.start[d] + hist[d] + before[k]] = tok[k];
            }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kKeep; ++k) {
            const int i = k * kSortThreads + tid;
            if (i < hi - b) {
                const int2 x = sm.tile[i];
                const int d = (x.x >> shift) & (bins - 1);
                const uint32_t at = sm.base[d] + i - sm.start[d];
                if (at < (uint32_t)n) out[at] = x;  // always, but in a workspace that another call shares
            }
        }
        if (one) break;
        __syncthreads();
        if (tid < bins) sm.base[tid] += mine;
    }
    // the moved tokens reach the cluster's other blocks, and the totals may go
    cluster_sync();
}

// The blocks, one cluster, sort the tokens by row.
__global__ void __launch_bounds__(kSortThreads)
    embedding_sort_kernel(EmbeddingGradArgs a, GradWork w, int passes, int bits) {
    extern __shared__ uint4 raw_smem[];
    allow_next();
    const int blocks = gridDim.x, rank = blockIdx.x, tid = threadIdx.x;
    const SortSmem sm(raw_smem, 1 << bits);
    if (rank == 0 && tid == 0) *w.crossings = 0;
    if (!a.accumulate)
        for (int64_t i = rank * kSortThreads + tid; i < (a.vocab + 31) / 32; i += blocks * kSortThreads) w.marks[i] = 0;
#pragma unroll 1
    for (int p = 0; p < passes; ++p)
        sort_pass(a, sm, blocks, rank, p * bits, bits, p ? w.sorted[(p & 1) ^ 1] : nullptr, w.sorted[p & 1]);
    if (rank == 0 && tid == 0) {
        int count = 0;
#pragma unroll
        for (int r = 0; r < kSortCluster; ++r)
            if (r < blocks) count += (int)cluster_read(&sm.total[1 << bits], r);
        *w.count = count;
    }
    cluster_sync();  // no block leaves while another reads its counts
}

// ------------------------------------------------------------ gradient: zeros and sums

// Scales a row's sums, adds what the table holds where the caller wants it,
// rounds and stores them.
template <typename D, bool kAligned>
__device__ __forceinline__ void store_row(const EmbeddingGradArgs& a, int row, int64_t g, Cols x, int lane) {
    const int n = granule_cols(g, a.cols);
    D* p = static_cast<D*>(a.table.data) + row * a.table.stride + g * kGran;
    Raw<D> r;
    x = x * all(a.scale);
    if (a.accumulate) {
        load_cols<kAligned>(r, p - g * kGran, g * kGran, n);
        x = x + widened(r);
        __syncwarp();  // a shifted load reads its neighbours' blocks
    }
    round_to(x, r);
    store_cols<kAligned>(p, r, n, lane);
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

// Lists a row that begins in a chunk and reaches further ones: the last is
// found among the chunks' first tokens, 32 probes at a time.
__device__ __forceinline__ void list_crossing(const GradWork& w, const int2* sorted, int count, int row, int chunk, int lane) {
    int lo = chunk + 1, hi = (count + w.chunk - 1) / w.chunk;  // chunk lo begins with the row, chunk hi does not
    while (hi - lo > 1) {
        const int gap = (hi - lo + 32) / 33, at = lo + (lane + 1) * gap;
        const unsigned more = __popc(__ballot_sync(kFull, at < hi && __ldcg(&sorted[at * w.chunk].x) == row));
        hi = lo + (int)(more + 1) * gap < hi ? lo + (int)(more + 1) * gap : hi;
        lo += (int)more * gap;
    }
    if (lane == 0) {
        const int at = atomicAdd(w.crossings, 1);
        if (at < w.nchunks) w.cross[at] = Crossing{row, chunk, lo - chunk, 0};
    }
}

// Zeros for a row of n elements, by one warp.
template <typename D>
__device__ __forceinline__ void zero_row(D* row, int64_t n, int lane) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(row), end = reinterpret_cast<uintptr_t>(row + n);
    const uintptr_t body = (p + 15) & ~(uintptr_t)15, tail = end & ~(uintptr_t)15;
    if (body >= tail) {
        for (int64_t i = lane; i < n; i += 32) row[i] = D(0);
        return;
    }
    if (p + lane * sizeof(D) < body) row[lane] = D(0);
    if (tail + lane * sizeof(D) < end) reinterpret_cast<D*>(tail)[lane] = D(0);
#pragma unroll 4
    for (uintptr_t q = body + lane * 16; q < tail; q += 512) st_stream(reinterpret_cast<uint4*>(q), make_uint4(0, 0, 0, 0));
}

// Zeros for the columns from first on (width of them) of those of count rows
// from r0 on that have no bit in named. Neighbouring rows without a gap between
// them are one stretch.
template <typename D>
__device__ __forceinline__ void zero_rows(const EmbeddingGradArgs& a, int64_t r0, int count, uint32_t named, int64_t first,
                                          int64_t width, int lane) {
    uint32_t todo = ~named & (count < 32 ? (1u << count) - 1 : ~0u);
    while (todo) {
        const int i = __ffs(todo) - 1;
        const uint32_t past = ~(todo >> i);
        const int run = a.table.stride == width && past ? __ffs(past) - 1 : (a.table.stride == width ? 32 - i : 1);
        zero_row(static_cast<D*>(a.table.data) + (r0 + i) * a.table.stride + first, run * width, lane);
        todo &= run < 32 ? ~(((1u << run) - 1) << i) : 0u;
    }
}

// Block z writes the zeros of its rows, per for each warp (a power of two up to
// 32, so that their marks lie in one word), that are not marked. Many short
// blocks: 131072 rows of 32 KB take 575 us in blocks of 8 rows and 656 in two
// blocks an SM that each take a long range.
template <typename D>
__device__ __forceinline__ void write_zeros(const EmbeddingGradArgs& a, const uint32_t* marks, int64_t z, int per) {
    const int64_t r0 = (z * kEmbWarps + (threadIdx.x >> 5)) * per;
    if (r0 >= a.vocab) return;
    const uint32_t named = __ldcg(marks + (r0 >> 5)) >> (r0 & 31);
    zero_rows<D>(a, r0, (int)(a.vocab - r0 < per ? a.vocab - r0 : per), named, 0, a.cols, threadIdx.x & 31);
}

// Tokens whose gradients a warp has in flight, in shared memory.
constexpr int kFlight = 8;

template <typename S, typename D, bool kAligned>
__global__ void __launch_bounds__(32 * kEmbWarps, sizeof(S) == 4 ? 3 : 5)
    embedding_sum_kernel(EmbeddingGradArgs a, GradWork w, const int2* sorted, int spans) {
    extern __shared__ uint4 flight[];
    constexpr int kOne = kSlot<kAligned, S>;
    uint4* const slots = flight + (threadIdx.x >> 5) * kFlight * kOne;
    const int lane = threadIdx.x & 31;
    const int64_t it = warp_id();
    const int64_t chunk = it / spans;
    const int g = (int)(it - chunk * spans) * 32 + lane, n = granule_cols((int64_t)g, a.cols);
    const int64_t c = (int64_t)g * kGran, c0 = c - lane * kGran;
    const int left = (int)(a.cols - c0 < kSpan ? a.cols - c0 : kSpan);
    allow_next();
    wait_for_previous();
    const int count = min(__ldcg(w.count), (int)a.n);
    if (chunk * w.chunk >= count) return;
    const int lo = (int)chunk * w.chunk, m = count - lo < w.chunk ? count - lo : w.chunk;
    // (calls that shared a workspace in spite of the header would leave any
    // numbers there: no gradient, row or part outside its matrix is touched)
    int2 mine = lane < m ? __ldcg(sorted + lo + lane) : make_int2(-1, 0);
    mine = make_int2((int)min((unsigned)mine.x, (unsigned)a.vocab - 1), (int)min((unsigned)mine.y, (unsigned)a.n - 1));
    const int prev = lo > 0 ? __ldcg(&sorted[lo - 1].x) : -1;
    const int next = lo + m < count ? __ldcg(&sorted[lo + m].x) : -1;
    if (!a.accumulate && g < 32) {  // once, with the first span: a row's first token marks it
        const int before = __shfl_up_sync(kFull, mine.x, 1);
        if (lane < m && mine.x != (lane ? before : prev)) atomicOr(w.marks + (mine.x >> 5), 1u << (mine.x & 31));
    }
    auto gradient = [&](int j) {
        return static_cast<const S*>(a.grad.data) + (int64_t)__shfl_sync(kFull, mine.y, j & 31) * a.grad.stride + c0;
    };
    auto fetch = [&](int j) {
        const S* from = gradient(j);
        if (j < m) span_fetch<kAligned>(slots + j % kFlight * kOne, from, 0, left, lane);
        async_commit();
    };
    Cols acc = all(0.0f);
    int cur = -1;
    bool open = false;  // cur began in an earlier chunk
    for (int j = 0; j < kFlight - 1; ++j) fetch(j);
#pragma unroll 1
    for (int j = 0; j < m; ++j) {
        fetch(j + kFlight - 1);
        async_wait<kFlight - 1>();
        __syncwarp();
        Raw<S> in;
        span_read<kAligned>(in, slots + j % kFlight * kOne, gradient(j), 0, lane);
        const int row = __shfl_sync(kFull, mine.x, j);
        if (row != cur) {
            if (cur >= 0) {
                if (!open)
                    store_row<D, kAligned>(a, cur, g, acc, lane);
                else if (n)
                    store_part(w.part + chunk * w.stride + c, acc);
            }
            open = cur < 0 && row == prev;
            cur = row;
            acc = widened(in);
        } else {
            acc = acc + widened(in);
        }
        __syncwarp();  // before the slot is filled again
    }
    if (open) {
        if (n) store_part(w.part + chunk * w.stride + c, acc);
    } else if (cur == next) {
        if (n) store_part(w.part + (w.nchunks + chunk) * w.stride + c, acc);
        if (g < 32) list_crossing(w, sorted, count, cur, (int)chunk, lane);  // once, with the first span
    } else {
        store_row<D, kAligned>(a, cur, g, acc, lane);
    }
}

// The sum of a crossing row's parts p0 ... p1 - 1: the first chunk's tail, then
// what the others leave at their heads. Where a row has few granules, `wide`
// lanes (a power of two) hold it and the warp adds 32 / wide parts at a time;
// all lanes take part, and every wide of them get the sum.
__device__ __forceinline__ Cols sum_parts(const GradWork& w, const int4& x, int p0, int p1, int64_t c, bool on, int wide, int lane) {
    Cols acc = all(0.0f);
    if (on)
#pragma unroll 8
        for (int p = p0 + lane / wide; p < p1; p += 32 / wide)
            acc = acc + load_part(w.part + (x.y + p + (p == 0 ? w.nchunks : 0)) * w.stride + c);
    for (int d = wide; d < 32; d *= 2)
#pragma unroll
        for (int e = 0; e < kGran; ++e) acc.set(e, acc.get(e) + __shfl_xor_sync(kFull, acc.get(e), d));
    return acc;
}

__device__ __forceinline__ bool sound(const EmbeddingGradArgs& a, const GradWork& w, const int4& x) {
    return (unsigned)x.x < (unsigned)a.vocab && (unsigned)x.y < (unsigned)w.nchunks && (unsigned)x.z < (unsigned)(w.nchunks - x.y);
}

// The first spans * y blocks, block (span, y): the rows that cross chunks, for
// a span of columns. Its warps take the listed rows of up to kShort parts in
// turn, one each, and then the others together, a share of the parts each. The
// other blocks write zeros.
constexpr int kShort = 8;
template <typename D, bool kAligned>
__global__ void __launch_bounds__(32 * kEmbWarps) embedding_join_kernel(EmbeddingGradArgs a, GradWork w, int spans, int ys, int per, int wide) {
    __shared__ float4 sums[kEmbWarps][2][32];
    wait_for_previous();
    if ((int)blockIdx.x >= spans * ys) {
        write_zeros<D>(a, w.marks, blockIdx.x - spans * ys, per);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, y = blockIdx.x / spans;
    const int64_t g = (int64_t)(blockIdx.x - y * spans) * 32 + lane, c = (g - lane + lane % wide) * kGran;
    const bool on = c < a.cols;
    const int crossings = min(__ldcg(w.crossings), w.nchunks);
    for (int i = y * kEmbWarps + warp; i < crossings; i += ys * kEmbWarps) {
        const int4 x = __ldcg(reinterpret_cast<const int4*>(w.cross + i));
        if (x.z >= kShort || !sound(a, w, x)) continue;
        store_row<D, kAligned>(a, x.x, g, sum_parts(w, x, 0, x.z + 1, c, on, wide, lane), lane);
    }
    for (int i = y; i < crossings; i += ys) {
        const int4 x = __ldcg(reinterpret_cast<const int4*>(w.cross + i));
        const int parts = x.z + 1;
        if (parts <= kShort || !sound(a, w, x)) continue;
        Cols acc = sum_parts(w, x, parts * warp / kEmbWarps, parts * (warp + 1) / kEmbWarps, c, on, wide, lane);
        sums[warp][0][lane] = make_float4(acc.p[0].x, acc.p[0].y, acc.p[1].x, acc.p[1].y);
        sums[warp][1][lane] = make_float4(acc.p[2].x, acc.p[2].y, acc.p[3].x, acc.p[3].y);
        __syncthreads();
        if (warp == 0) {
            for (int q = 1; q < kEmbWarps; ++q) {
                const float4 u = sums[q][0][lane], v = sums[q][1][lane];
                acc = acc + Cols{{make_float2(u.x, u.y), make_float2(u.z, u.w), make_float2(v.x, v.y), make_float2(v.z, v.w)}};
            }
            store_row<D, kAligned>(a, x.x, g, acc, lane);
        }
        __syncthreads();
    }
}

// -------------------------------------------- gradient: up to kFewTokens tokens

// Adds to acc the gradients of the listed tokens for the 256 columns from c0
// on (left of them), kFlight in flight.
template <typename S, bool kAligned>
__device__ __forceinline__ Cols sum_tokens(const EmbeddingGradArgs& a, const short* list, int m, int64_t c0, int left, uint4* slots,
                                           int lane) {
    constexpr int kOne = kSlot<kAligned, S>;
    auto gradient = [&](int j) { return static_cast<const S*>(a.grad.data) + list[j] * a.grad.stride + c0; };
    auto fetch = [&](int j) {
        if (j < m) span_fetch<kAligned>(slots + j % kFlight * kOne, gradient(j), 0, left, lane);
        async_commit();
    };
    Cols acc = all(0.0f);
    for (int j = 0; j < kFlight - 1; ++j) fetch(j);
#pragma unroll 1
    for (int j = 0; j < m; ++j) {
        fetch(j + kFlight - 1);
        async_wait<kFlight - 1>();
        __syncwarp();
        Raw<S> in;
        span_read<kAligned>(in, slots + j % kFlight * kOne, gradient(j), 0, lane);
        acc = acc + widened(in);
        __syncwarp();  // before the slot is filled again
    }
    return acc;
}

// One kernel and no sort: every block holds all tokens' rows, and a warp looks
// for those of its own `per` rows among them, for a group of kGroup spans of
// columns (blockIdx.y). It writes zeros, or sums up to kAlone tokens by itself;
// rows of more tokens are left for the whole block, its warps taking a span
// and a share of the tokens each. (Groups of 4 spans: 300 tokens, most in three
// rows of 1027, 17 us instead of 12; of 1 span, 32000 x 4096 takes 64 us
// instead of 42.)
constexpr int kAlone = 8, kGroup = 2;
template <typename S, typename D, bool kAligned>
__global__ void __launch_bounds__(32 * kEmbWarps)
    embedding_few_kernel(EmbeddingGradArgs a, int per) {
    extern __shared__ uint4 flight[];
    __shared__ int keys[kFewTokens];
    __shared__ short list[kEmbWarps][kAlone], shared_list[kFewTokens];
    __shared__ int64_t many[kEmbWarps * 32];
    __shared__ int manies, found;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = (int)a.n, quads = (n + 31) / 32;
    constexpr int kMine = kFlight * kSlot<kAligned, S>;
    uint4* const slots = flight + warp * kMine;
    const int64_t first = (int64_t)blockIdx.y * (kGroup * kSpan);
    const int width = (int)(a.cols - first < kGroup * kSpan ? a.cols - first : kGroup * kSpan), spans = (width + kSpan - 1) / kSpan;
    for (int i = threadIdx.x; i < quads * 32; i += 32 * kEmbWarps)
        keys[i] = i < n ? row_of(read_id(a.ids, a.wide_ids, i), a.first, a.vocab) : -1;
    if (threadIdx.x == 0) manies = 0;
    __syncthreads();
    // the sums of a span of the group, and their store
    auto sum = [&](const short* tokens, int m, int s) {
        const int left = width - s * kSpan < kSpan ? width - s * kSpan : kSpan;
        return sum_tokens<S, kAligned>(a, tokens, m, first + s * kSpan, left, slots, lane);
    };
    auto store = [&](int64_t row, int s, const Cols& acc) {
        store_row<D, kAligned>(a, (int)row, (first / kSpan + s) * 32 + lane, acc, lane);
    };

    const int64_t r0 = ((int64_t)blockIdx.x * kEmbWarps + warp) * per;
    if (r0 < a.vocab) {
        // which of the warp's rows are named
        uint32_t named = 0;
        for (int q = 0; q < quads; ++q) {
            const uint32_t at = (uint32_t)keys[q * 32 + lane] - (uint32_t)r0;
            if (at < (uint32_t)per) named |= 1u << at;
        }
        named = __reduce_or_sync(kFull, named);
        const int rows = (int)(a.vocab - r0 < per ? a.vocab - r0 : per);
        if (!a.accumulate) zero_rows<D>(a, r0, rows, named, first, width, lane);
        for (int i = 0; i < rows; ++i) {
            const int64_t row = r0 + i;
            if (!(named >> i & 1)) continue;
            int m = 0;  // its tokens, in ascending order
            for (int q = 0; q < quads; ++q) {
                const unsigned hit = __ballot_sync(kFull, keys[q * 32 + lane] == (int)row);
                const int at = m + __popc(hit & ((1u << lane) - 1));
                if ((hit >> lane & 1) && at < kAlone) list[warp][at] = (short)(q * 32 + lane);
                m += __popc(hit);
            }
            __syncwarp();
            if (m > kAlone) {
                if (lane == 0) many[atomicAdd(&manies, 1)] = row;
                continue;
            }
            for (int s = 0; s < spans; ++s) store(row, s, sum(list[warp], m, s));
            __syncwarp();
        }
    }
    __syncthreads();
    const int count = manies, shares = kEmbWarps / spans;
    for (int k = 0; k < count; ++k) {
        const int64_t row = many[k];
        if (warp == 0) {
            int m = 0;
            for (int q = 0; q < quads; ++q) {
                const unsigned hit = __ballot_sync(kFull, keys[q * 32 + lane] == (int)row);
                if (hit >> lane & 1) shared_list[m + __popc(hit & ((1u << lane) - 1))] = (short)(q * 32 + lane);
                m += __popc(hit);
            }
            if (lane == 0) found = m;
        }
        __syncthreads();
        const int m = found;
        const int share = warp / spans, s = warp - share * spans;
        Cols acc = all(0.0f);
        if (share < shares) {
            const int j0 = m * share / shares, j1 = m * (share + 1) / shares;
            acc = sum(shared_list + j0, j1 - j0, s);
            store_part(reinterpret_cast<float*>(slots + 2 * lane), acc);  // what was in flight has been read
        }
        __syncthreads();
        if (share == 0) {
            for (int q = 1; q < shares; ++q) {
                const float4* other = reinterpret_cast<const float4*>(slots + q * spans * kMine + 2 * lane);
                const float4 u = other[0], v = other[1];
                acc = acc + Cols{{make_float2(u.x, u.y), make_float2(u.z, u.w), make_float2(v.x, v.y), make_float2(v.z, v.w)}};
            }
            store(row, s, acc);
        }
        __syncthreads();
    }
}

template <typename S, typename D, bool kAligned>
cudaError_t embedding_grad_few(const EmbeddingGradArgs& a, cudaStream_t s) {
    const int64_t groups = (a.cols + kGroup * kSpan - 1) / (kGroup * kSpan), width = groups > 1 ? kGroup * kSpan : a.cols;
    // a warp takes rows that make up 8 KB of zeros, but one token on average
    // (438 tokens into 411 rows of 5: 42 us by 32 rows, 5 by one)
    int per = 1;
    while (per < 32 && 2 * per * width * (int64_t)sizeof(D) <= 8192 && 2 * per * a.n <= a.vocab) per *= 2;
    const int64_t blocks = (a.vocab + per * kEmbWarps - 1) / (per * kEmbWarps);
    constexpr int smem = kEmbWarps * kFlight * kSlot<kAligned, S> * 16;
    static std::atomic<uint64_t> done{0};
    auto kernel = embedding_few_kernel<S, D, kAligned>;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem, done);
    if (e != cudaSuccess) return e;
    kernel<<<dim3((unsigned)blocks, (unsigned)groups), 32 * kEmbWarps, smem, s>>>(a, per);
    count_launch();
    return cudaGetLastError();
}

template <typename S, typename D, bool kAligned>
cudaError_t embedding_grad_as(const EmbeddingGradArgs& a, cudaStream_t s) {
    // One kernel against three, calls in a row: 64 tokens into 32000 x 4096 bf16
    // 41 and 53 us, 300 into 4099 x 1027 fp32, nine in ten of them in three
    // rows, 14 and 23, spread 10 and 23. With many tokens a row it falls behind,
    // a block having a row's tokens to itself: 512 into 7 rows of 8192 45 and 20.
    if (a.n <= kFewTokens && a.n <= 8 * a.vocab && a.cols <= (int64_t)65535 * kGroup * kSpan)
        return embedding_grad_few<S, D, kAligned>(a, s);
    const GradWork w = grad_work(a.work, a.n, a.vocab, a.cols, nullptr);
    int need = 1;
    while (((int64_t)1 << need) <= a.vocab) ++need;  // bits of the values 0 .. vocab
    const int passes = (need + kMaxBits - 1) / kMaxBits, bits = (need + passes - 1) / passes;
    const int spans = (int)((a.cols + kSpan - 1) / kSpan);
    const int64_t sums = (w.nchunks * (int64_t)spans + kEmbWarps - 1) / kEmbWarps;
    // a warp of zeros takes one row, or more that make up 8 KB
    int per = 1;
    while (per < 32 && 2 * per * a.cols * (int64_t)sizeof(D) <= 8192) per *= 2;
    const int64_t zeros = a.accumulate ? 0 : (a.vocab + per * kEmbWarps - 1) / (per * kEmbWarps);
    const int ys = w.nchunks <= 1 ? 0 : (w.nchunks - 1 < 64 ? w.nchunks - 1 : 64);
    int wide = 32;  // lanes of a row's granules in the joins
    while (wide > 1 && (wide / 2) * kGran >= a.cols) wide /= 2;
    if (sums > 0x7fffffff || zeros + (int64_t)spans * ys > 0x7fffffff) return cudaErrorInvalidValue;
    cudaError_t e = cudaSuccess;
    {
        const size_t smem = SortSmem::bytes(1 << bits);
        static std::atomic<uint64_t> done{0};
        e = allow_smem(reinterpret_cast<const void*>(embedding_sort_kernel), (int)SortSmem::bytes(1 << kMaxBits), done);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(a.n <= 4096 ? 1 : kSortCluster);
        cfg.blockDim = dim3(kSortThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = cfg.gridDim.x;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        if ((e = cudaLaunchKernelEx(&cfg, embedding_sort_kernel, a, w, passes, bits)) != cudaSuccess) return e;
        count_launch();
    }
    const int2* const sorted = w.sorted[(passes - 1) & 1];
    {
        constexpr int smem = kEmbWarps * kFlight * kSlot<kAligned, S> * 16;
        static std::atomic<uint64_t> done{0};
        auto kernel = embedding_sum_kernel<S, D, kAligned>;
        if ((e = allow_smem(reinterpret_cast<const void*>(kernel), smem, done)) != cudaSuccess) return e;
        e = launch_next(kernel, dim3((unsigned)sums), 32 * kEmbWarps, smem, s, a, w, sorted, spans);
        if (e != cudaSuccess) return e;
        count_launch();
    }
    if (zeros + spans * ys == 0) return cudaSuccess;
    e = launch_next(embedding_join_kernel<D, kAligned>, dim3((unsigned)(zeros + spans * ys)), 32 * kEmbWarps, 0, s, a, w, spans, ys, per, wide);
    if (e == cudaSuccess) count_launch();
    return e;
}

template <typename S, typename D>
cudaError_t embedding_grad(const EmbeddingGradArgs& a, cudaStream_t s) {
    const bool aligned = a.cols % kGran == 0 && on_grid(a.grad, sizeof(S)) && on_grid(a.table, sizeof(D));
    return aligned ? embedding_grad_as<S, D, true>(a, s) : embedding_grad_as<S, D, false>(a, s);
}

template <typename S, typename D>
cudaError_t embedding(const EmbeddingArgs& a, cudaStream_t s) {
    const int64_t spans = (a.cols + kSpan - 1) / kSpan, steps = (spans + kEmbSpans<S, D> - 1) / kEmbSpans<S, D>, items = steps * a.n;
    const int per = (int)((spans + steps - 1) / steps);
    const int64_t blocks = (items + kEmbWarps - 1) / kEmbWarps;
    const unsigned grid = (unsigned)(blocks < 0x7fffffff ? blocks : 0x7fffffff);
    const bool aligned = a.cols % kGran == 0 && on_grid(a.table, sizeof(S)) && on_grid(a.out, sizeof(D));
    if (narrow_rows(a.n, a.cols, aligned)) {
        const uint32_t grans = (uint32_t)((a.cols + kGran - 1) / kGran), all = (uint32_t)a.n * grans;
        const uint32_t each = kNarrow * 32 * kEmbWarps, blocks32 = (all + each - 1) / each;
        if (aligned)
            embedding_narrow_kernel<S, D, true><<<blocks32, 32 * kEmbWarps, 0, s>>>(a, grans, all);
        else
            embedding_narrow_kernel<S, D, false><<<blocks32, 32 * kEmbWarps, 0, s>>>(a, grans, all);
    } else if (aligned)
        embedding_kernel<S, D, true><<<grid, 32 * kEmbWarps, 0, s>>>(a, steps, per, items);
    else
        embedding_kernel<S, D, false><<<grid, 32 * kEmbWarps, 0, s>>>(a, steps, per, items);
    count_launch();
    return cudaGetLastError();
}

}  // namespace

size_t embedding_grad_bytes(int64_t n, int64_t vocab, int64_t cols) {
    size_t bytes = 0;
    grad_work(nullptr, n, vocab, cols, &bytes);
    return bytes;
}

// What any number of tokens up to n may need. While a chunk's tokens stay the
// same, more tokens need more; where a chunk grows there are fewer parts, so
// the last numbers of tokens before that count too.
size_t embedding_grad_most_bytes(int64_t n, int64_t vocab, int64_t cols) {
    const ChunkRule r = chunk_rule(cols);
    size_t most = embedding_grad_bytes(n, vocab, cols);
    for (const int64_t last : {r.most8, r.most16})
        if (last < n) most = std::max(most, embedding_grad_bytes(last, vocab, cols));
    return most;
}

cudaError_t launch_embedding(int table_dt, int out_dt, const EmbeddingArgs& a, cudaStream_t s) {
    if (a.n == 0 || a.cols == 0) return cudaSuccess;
    if (table_dt == FSDP_F32) return out_dt == FSDP_F32 ? embedding<float, float>(a, s) : embedding<float, uint16_t>(a, s);
    return out_dt == FSDP_F32 ? embedding<uint16_t, float>(a, s) : embedding<uint16_t, uint16_t>(a, s);
}

cudaError_t launch_embedding_grad(int grad_dt, int table_dt, const EmbeddingGradArgs& a, cudaStream_t s) {
    if (a.vocab == 0 || a.cols == 0) return cudaSuccess;
    if (a.accumulate && a.n == 0) return cudaSuccess;
    if (grad_dt == FSDP_F32) return table_dt == FSDP_F32 ? embedding_grad<float, float>(a, s) : embedding_grad<float, uint16_t>(a, s);
    return table_dt == FSDP_F32 ? embedding_grad<uint16_t, float>(a, s) : embedding_grad<uint16_t, uint16_t>(a, s);
}

}  // namespace fsdp
