// Orthogonalisation of an update by Newton-Schulz products.
//
// The iterate X is kept in two binary16 planes, X = 2^-sx (hi + 2^-11 lo), of
// which the products take hi. A product with binary16 factors is off by 2^-12
// of its factors' sizes, and the iteration lifts small singular values by up
// to a^steps (485 times), and what is off in their directions with them. So
// the term that lifts them, shift * X, is added in binary32 from both planes,
// and the product only brings (b A + c A A + (a - shift) I) X, where A is small
// in those directions and damps what is off. (Five steps against 64 bits, in
// the 2-norm, a few strong directions over 3% or 0.1% of noise: 0.002; with
// one plane 0.02 and 0.04; in bfloat16 0.17 and 0.34. Noise alone 0.002, 0.002
// and 0.011. Rounding the result to bfloat16 alone is 0.0017.) In the last two
// steps the singular values are near one, and so is the whole polynomial: with
// shift = a the product would bring a - 1 times X that has to go again, so shift
// is (1 + a) / 2 there, which halves that.
#include <algorithm>
#include <cmath>
#include <utility>

#include "fsdp_gemm.cuh"

namespace fsdp {
namespace {

constexpr int kSquareBlocks = 304, kSquareThreads = 256;

__device__ __forceinline__ uint32_t half_bits(float v) { return (uint32_t)__half_as_ushort(__float2half_rn(v)); }
__device__ __forceinline__ float half_value(uint32_t b) { return __half2float(__ushort_as_half((unsigned short)b)); }
__device__ __forceinline__ void round_half(const Cols& v, Raw<uint16_t>& r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = half_bits(v.p[i].x) | half_bits(v.p[i].y) << 16;
}
__device__ __forceinline__ Cols widened_half(const Raw<uint16_t>& r) {
    Cols v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.p[i] = make_float2(half_value(r.w[i] & 0xffffu), half_value(r.w[i] >> 16));
    return v;
}
__device__ __forceinline__ uint16_t* at(const Mat& m, int64_t row, int64_t col) {
    return static_cast<uint16_t*>(m.data) + row * m.stride + col;
}
__device__ __forceinline__ void put_half(const Mat& m, int64_t row, int64_t col, int n, const Cols& v) {
    Raw<uint16_t> r;
    round_half(v, r);
    store_granule(at(m, row, col), r, n);
}
constexpr float kLow = 2048.0f;  // the second plane's scale
// Both planes of values of the first plane's scale.
__device__ __forceinline__ void put_planes(const Mat& hi, const Mat& lo, int64_t row, int64_t col, int n, const Cols& v) {
    Raw<uint16_t> r;
    round_half(v, r);
    store_granule(at(hi, row, col), r, n);
    const Cols rest = (v + widened_half(r) * all(-1.0f)) * all(kLow);
    put_half(lo, row, col, n, rest);
}

// ------------------------------------------------------- the first iterate

// A block's sums of squares, of values by their size, so that no square
// overflows or vanishes: those of at least 2^50 by 2^-90, those below 2^-40 by
// 2^90 (Blue, "A portable Fortran program to find the Euclidean norm of a
// vector", 1978). The squares lie between 2^-118 and 2^100, so binary32 holds a
// thread's next 64 granules' sums of any of the three; beyond that they are
// added up in 64 bits, which no number of values overflows or wears out.
template <typename T>
__global__ void __launch_bounds__(kSquareThreads) square_kernel(Mat x, int64_t rows, int64_t cols, double* parts) {
    wait_for_previous();
    const int64_t per = (cols + kGran - 1) / kGran, all_granules = rows * per;
    double total[3] = {0.0, 0.0, 0.0};
    int64_t g = (int64_t)blockIdx.x * kSquareThreads + threadIdx.x;
    while (g < all_granules) {
        float sum[3] = {0.0f, 0.0f, 0.0f};
        for (int n = 0; n < 64 && g < all_granules; ++n, g += (int64_t)kSquareBlocks * kSquareThreads) {
            const int64_t row = g / per, i = g - row * per;
            Raw<T> r;
            load_granule(r, static_cast<const T*>(x.data) + row * x.stride, i * kGran, granule_cols(i, cols));
            const Cols v = widened(r);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = v.get(e), m = fabsf(f);
                const int which = m >= 0x1p50f ? 2 : (m < 0x1p-40f ? 0 : 1);
                const float q = which == 2 ? f * 0x1p-90f : (which == 0 ? f * 0x1p90f : f);
                sum[0] = which == 0 ? __fmaf_rn(q, q, sum[0]) : sum[0];
                sum[2] = which == 2 ? __fmaf_rn(q, q, sum[2]) : sum[2];
                sum[1] = which == 1 ? __fmaf_rn(q, q, sum[1]) : sum[1];  // NaN too
            }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) total[k] += (double)sum[k];
    }
    __shared__ double box[3][kSquareThreads / 32];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) total[k] += __shfl_xor_sync(kFull, total[k], d);
        if (threadIdx.x % 32 == 0) box[k][threadIdx.x / 32] = total[k];
    }
    __syncthreads();
    if (threadIdx.x < 3) {
        double of_block = 0.0;
        for (int w = 0; w < kSquareThreads / 32; ++w) of_block += box[threadIdx.x][w];
        parts[threadIdx.x * kSquareBlocks + blockIdx.x] = of_block;
    }
}

// What x is multiplied by on its way into X, as a product of two factors neither
// of which leaves binary32's range, and the power of two by which X is then above
// x / (|x| + eps).
struct Factor {
    float first, second;
    int lift;
    __device__ __forceinline__ float of(float v) const { return v * first * second; }
    __device__ __forceinline__ Cols of(const Cols& v) const { return v * all(first) * all(second); }
};

// 2^sx 2^e / (|x| + eps) from the parts. Where `full`, e brings X to a norm
// between 1/4 and 1 if it is below; else e is 0. All threads of a block of at
// least 96 take part.
__device__ __forceinline__ Factor norm_factor(const double* parts, double eps, int sx, bool full) {
    __shared__ double sums[3];
    __shared__ Factor factor;
    if (threadIdx.x < 96) {
        double s = 0.0;
        for (int i = threadIdx.x % 32; i < kSquareBlocks; i += 32) s += parts[threadIdx.x / 32 * kSquareBlocks + i];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
        if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = s;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        const double norm = sqrt(sums[0] * 0x1p-180 + sums[1] + sums[2] * 0x1p180);
        const int lift = full && norm > 0.0 && isfinite(norm) ? max(0, ilogb(norm + eps) - ilogb(norm) - 1) : 0;
        // a norm is 0 or at least 2^-149: a quotient above 2^165 has only zeros to scale (without an eps it is 0 / 0)
        double f = ldexp(1.0 / (norm + eps), sx + lift);
        if (norm + eps > 0.0) f = fmin(f, 0x1p200);
        int e = 0;
        const double m = frexp(f, &e);
        factor = isfinite(f) ? Factor{ldexpf(1.0f, e / 2), (float)ldexp(m, e - e / 2), lift} : Factor{(float)f, 1.0f, lift};
    }
    __syncthreads();
    return factor;
}

// X = x / (|x| + eps) as two planes scaled by 2^sx, and by what `lift` receives.
// (Without that, where eps is far above |x|, all of X would lie below what the
// planes resolve: half of it was gone at eps = 10^7 |x|.)
template <typename T>
__global__ void __launch_bounds__(256) planes_kernel(Mat x, int64_t rows, int64_t cols, const double* parts, double eps, int sx, Mat hi, Mat lo,
                                                     int* lift) {
    wait_for_previous();
    const Factor f = norm_factor(parts, eps, sx, true);
    if (blockIdx.x == 0 && threadIdx.x == 0) *lift = f.lift;
    const int64_t per = (cols + kGran - 1) / kGran, all_granules = rows * per;
    for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < all_granules; g += (int64_t)gridDim.x * 256) {
        const int64_t row = g / per, i = g - row * per;
        const int n = granule_cols(i, cols);
        Raw<T> r;
        load_granule(r, static_cast<const T*>(x.data) + row * x.stride, i * kGran, n);
        put_planes(hi, lo, row, i * kGran, n, f.of(widened(r)));
    }
}

// The power of two e by which a step's X is above the iteration's: what
// planes_kernel began with, less what the steps may have grown by since. With
// g_t for the most that step t multiplies a singular value by, in powers of two
// rounded up, e becomes max(0, e - g_t), so no singular value leaves the range;
// in closed form over the steps, max(first - less, least). (Looked up once a
// thread: once a granule 4096 x 11008 took 2.63 ms instead of 2.35.)
struct Lift {
    const int* first;
    int less, least;
    __device__ __forceinline__ int now() const { return max(*first - less, least); }
};
// ------------------------------------------------------ one short side
//
// With at most 64 rows (or columns) X stays in binary32, in blocks of 64 of its
// columns (rows, where tall), and every step forms A from it anew: a block of
// threads multiplies its blocks of columns by a I + b A + c A A and adds up what
// they are to the next A. (So few values average no rounding: in binary16 a 1 x
// 1 matrix is 0.007 off. A <- M M A, with M the polynomial, would need no X
// until the end, but where x has nothing A's eigenvalues are what rounding
// leaves, of either sign, and that recursion multiplies them by a a a step: 64 x
// 200 of eight strong directions over 0.1% of noise were off by half after
// eight steps, and NaN after twelve. X X^T has no negative ones but for one
// step's rounding.)
//
// None of these kernels lets the next one's blocks in early: those would take
// their places on the SMs that are free first, several to one (64 x 4096, five
// steps: 85 us, and 151 with that; 64 x 28672 144 and 171; 64 x 200 77 and 145).
constexpr int kSide = 64, kChunk = 64, kSidePitch = kSide + 4, kGramBlocks = 608, kNarrowThreads = 256;
constexpr int kSideValues = kSide * kSidePitch;
constexpr int kNarrowSmem = 3 * kSideValues * 4;

__device__ __forceinline__ float value_of(const float* p) { return *p; }
__device__ __forceinline__ float value_of(const uint16_t* p) { return bf16_to_f32(*p); }

// A thread's 4 x 4 values of sum over k of a[k][i] b[k][j].
__device__ __forceinline__ void small_product(float (&s)[4][4], const float* a, const float* b, int k_end, int i0, int j0) {
#pragma unroll 4
    for (int k = 0; k < k_end; ++k) {
        const float4 u = *reinterpret_cast<const float4*>(a + k * kSidePitch + i0), v = *reinterpret_cast<const float4*>(b + k * kSidePitch + j0);
        const float x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[r][c] = __fmaf_rn(x[r], y[c], s[r][c]);
    }
}

// A thread's 4 x 4 values of a block's share of A. After 32 blocks of columns
// the sums start again, and what they were is added to the share in memory: no
// chain of additions is longer than 2048 and as many as there are such stretches.
// (In one chain a row of a hundred million equal values had an A that was 0.1%
// off. Sums that keep what an addition cut off take 32 registers more: 33 x
// 1000003 1525 us instead of 1420.)
struct GramShare {
    float s[4][4];
    int blocks;
    bool put;
    __device__ __forceinline__ GramShare() : s{}, blocks(0), put(false) {}
    __device__ __forceinline__ void add(const float* columns, int p, int i0, int j0, float* shares) {
        if (i0 < p && j0 < p) small_product(s, columns, columns, kChunk, i0, j0);
        if (++blocks == 32) keep(i0, j0, shares);
    }
    __device__ __forceinline__ void keep(int i0, int j0, float* shares) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float4* at = reinterpret_cast<float4*>(shares + ((int64_t)blockIdx.x * kSide + i0 + r) * kSide + j0);
            const float4 old = put ? *at : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            *at = make_float4(old.x + s[r][0], old.y + s[r][1], old.z + s[r][2], old.w + s[r][3]);
#pragma unroll
            for (int c = 0; c < 4; ++c) s[r][c] = 0.0f;
        }
        put = true;
        blocks = 0;
    }
};

// X_0 in blocks of columns, [block][p][kChunk], and the shares of its A.
template <typename T>
__global__ void __launch_bounds__(kNarrowThreads) narrow_first_kernel(Mat x, int tall, int p, int64_t q, const double* parts, double eps, float* held,
                                                                      float* shares) {
    __shared__ __align__(16) float columns[kChunk * kSidePitch];
    wait_for_previous();
    const Factor f = norm_factor(parts, eps, 0, false);
    const T* data = static_cast<const T*>(x.data);
    const int i0 = threadIdx.x / 16 * 4, j0 = threadIdx.x % 16 * 4;
    GramShare share;
    for (int64_t block = blockIdx.x; block * kChunk < q; block += gridDim.x) {
        const int64_t first = block * kChunk;
        for (int c = threadIdx.x; c < kSide * kChunk; c += kNarrowThreads) {
            const int i = tall ? c % kSide : c / kChunk, j = tall ? c / kSide : c % kChunk;
            float v = 0.0f;
            if (i < p && first + j < q) v = f.of(value_of(tall ? data + (first + j) * x.stride + i : data + i * x.stride + first + j));
            columns[j * kSidePitch + i] = v;
        }
        __syncthreads();
        for (int c = threadIdx.x; c < p * kChunk; c += kNarrowThreads) held[block * p * kChunk + c] = columns[c % kChunk * kSidePitch + c / kChunk];
        share.add(columns, p, i0, j0, shares);
        __syncthreads();
    }
    share.keep(i0, j0, shares);
}

// A from its shares: 16 values a block of threads, 16 threads a value.
constexpr int kSumValues = 16, kSumBlocks = kSide * kSide / kSumValues;
__global__ void __launch_bounds__(kNarrowThreads) narrow_sum_kernel(const float* shares, int n_shares, float* gram) {
    __shared__ float box[kNarrowThreads];
    wait_for_previous();
    const int e = blockIdx.x * kSumValues + threadIdx.x % kSumValues;
    float sum = 0.0f;
#pragma unroll 8
    for (int k = threadIdx.x / kSumValues; k < n_shares; k += kNarrowThreads / kSumValues) sum += shares[(int64_t)k * kSide * kSide + e];
    box[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x < kSumValues) {
        float total = 0.0f;
#pragma unroll
        for (int k = 0; k < kNarrowThreads; k += kSumValues) total += box[threadIdx.x + k];
        gram[e] = total;
    }
}

// X <- a X + (b A + c A A) X and the shares of the next A; in the last step
// scale * X to the caller's matrix. Four blocks to an SM, 64 registers a thread:
// 33 x 1000003 in 1420 us, 2033 with three.
__global__ void __launch_bounds__(kNarrowThreads, 4) narrow_step_kernel(float* held, int tall, int p, int64_t q, const float* gram, float a, float b, float c,
                                                                     float scale, float* shares, Mat out) {
    extern __shared__ __align__(16) float room[];
    float *M = room, *now = room + kSideValues, *next = room + 2 * kSideValues;
    wait_for_previous();
    const int i0 = threadIdx.x / 16 * 4, j0 = threadIdx.x % 16 * 4, k_end = (p + 3) / 4 * 4;
    for (int e = threadIdx.x; e < kSide * kSide; e += kNarrowThreads) now[e / kSide * kSidePitch + e % kSide] = gram[e];
    __syncthreads();
    float m[4][4] = {};
    if (i0 < p && j0 < p) small_product(m, now, now, k_end, i0, j0);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            M[(i0 + r) * kSidePitch + j0 + e] = __fmaf_rn(c, m[r][e], __fmaf_rn(b, now[(i0 + r) * kSidePitch + j0 + e], i0 + r == j0 + e ? a : 0.0f));
    GramShare share;
    for (int64_t block = blockIdx.x; block * kChunk < q; block += gridDim.x) {
        const int64_t first = block * kChunk;
        float* at_block = held + block * p * kChunk;
        __syncthreads();
        for (int e = threadIdx.x; e < kSide * kChunk / 4; e += kNarrowThreads) {
            const int i = e / (kChunk / 4), j = e % (kChunk / 4) * 4;
            *reinterpret_cast<float4*>(now + i * kSidePitch + j) =
                i < p ? *reinterpret_cast<const float4*>(at_block + i * kChunk + j) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        __syncthreads();
        float s[4][4] = {};
        if (i0 < p) small_product(s, M, now, k_end, i0, j0);
        if (!out.data) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (i0 + r < p) *reinterpret_cast<float4*>(at_block + (i0 + r) * kChunk + j0) = make_float4(s[r][0], s[r][1], s[r][2], s[r][3]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<float4*>(next + (j0 + e) * kSidePitch + i0) = make_float4(s[0][e], s[1][e], s[2][e], s[3][e]);
            __syncthreads();
            share.add(next, p, i0, j0, shares);
            continue;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + r;
                const int64_t j = first + j0 + e;
                if (i < p && j < q) *(tall ? at(out, j, i) : at(out, i, j)) = (uint16_t)f32_to_bf16(s[r][e] * scale);
            }
    }
    if (!out.data) share.keep(i0, j0, shares);
}

// -------------------------------------------------------------- epilogues

// A = X X^T.
struct Gram {
    static constexpr bool kMirror = true;
    struct Before {};
    struct Once {};
    Mat out;
    float scale;
    __device__ __forceinline__ Once once() const { return {}; }
    __device__ __forceinline__ void bring(int, int64_t, int64_t, int, Before&) const {}
    __device__ __forceinline__ void put(int64_t row, int64_t col, int n, const Raw<uint16_t>& r) const { store_granule(at(out, row, col), r, n); }
    __device__ __forceinline__ void operator()(int, int, int64_t row, int64_t col, int n, const Cols& v, const Cols&, const Before&,
                                               Once, Raw<uint16_t>& r) const {
        round_half(v * all(scale), r);
        put(row, col, n, r);
    }
};

// c A A + b A + d I, of an A that is 2^(2 e) of what it stands for.
struct Poly {
    static constexpr bool kMirror = true;
    struct Before {
        Raw<uint16_t> a;
    };
    struct Once {
        float square, linear;
    };
    Mat a, out;
    float square, linear, diagonal;
    Lift lift;
    __device__ __forceinline__ Once once() const {
        const int e = lift.now();
        return {ldexpf(square, -4 * e), ldexpf(linear, -2 * e)};
    }
    __device__ __forceinline__ void bring(int, int64_t row, int64_t col, int n, Before& b) const { load_granule(b.a, at(a, row, col), 0, n); }
    __device__ __forceinline__ void put(int64_t row, int64_t col, int n, const Raw<uint16_t>& r) const { store_granule(at(out, row, col), r, n); }
    __device__ __forceinline__ void operator()(int, int, int64_t row, int64_t col, int n, const Cols& v, const Cols&, const Before& b, Once by,
                                               Raw<uint16_t>& r) const {
        Cols s = fma(v, all(by.square), widened_half(b.a) * all(by.linear));
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e == row) s.set(e, s.get(e) + diagonal);
        round_half(s, r);
        put(row, col, n, r);
    }
};

// X <- shift X + D, into the planes, or at the end into the caller's matrix.
struct Next {
    static constexpr bool kMirror = false;
    struct Before {
        Raw<uint16_t> hi, lo;
    };
    struct Once {
        float scale, shift;
    };
    Mat hi, lo, next, out;  // out.data: the caller's
    float scale, shift;
    Lift lift, after;  // X's, and that of the next
    __device__ __forceinline__ Once once() const {
        const int e = (out.data ? 0 : after.now()) - lift.now();
        return {ldexpf(scale, e), ldexpf(shift, e)};
    }
    __device__ __forceinline__ void bring(int, int64_t row, int64_t col, int n, Before& b) const {
        load_granule(b.hi, at(hi, row, col), 0, n);
        load_granule(b.lo, at(lo, row, col), 0, n);
    }
    __device__ __forceinline__ void operator()(int, int, int64_t row, int64_t col, int n, const Cols& v, const Cols&, const Before& b, Once by,
                                               Raw<uint16_t>& r) const {
        Cols x = fma(widened_half(b.lo), all(1.0f / kLow), widened_half(b.hi));
        x = fma(v, all(by.scale), x * all(by.shift));
        if (!out.data) {
            put_planes(next, lo, row, col, n, x);
        } else {
            round_to(x, r);
            store_granule(at(out, row, col), r, n);
        }
    }
};

constexpr size_t kPartsRoom = ((3 * kSquareBlocks + 1) * 8 + 255) / 256 * 256;  // and the first lift

// Blocks of columns, shares of A, and their room with A and X.
int64_t narrow_blocks(int64_t q) { return (q + kChunk - 1) / kChunk; }
int64_t narrow_shares(int64_t q) { return std::min<int64_t>(narrow_blocks(q), kGramBlocks); }
size_t narrow_room(int64_t p, int64_t q) { return (size_t)((narrow_shares(q) + 1) * kSide * kSide + narrow_blocks(q) * kChunk * p) * 4; }

template <typename T>
cudaError_t narrow(const OrthoArgs& a, cudaStream_t s) {
    const int tall = a.rows > a.cols;
    const int p = (int)(tall ? a.cols : a.rows);
    const int64_t q = tall ? a.rows : a.cols;
    const int n_shares = (int)narrow_shares(q);
    const double* parts = reinterpret_cast<const double*>(a.work);
    float* shares = reinterpret_cast<float*>(a.work + kPartsRoom);
    float* gram = shares + (size_t)n_shares * kSide * kSide;
    float* held = gram + kSide * kSide;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(narrow_step_kernel), kNarrowSmem, done);
    if (e == cudaSuccess) e = launch_next(narrow_first_kernel<T>, dim3(n_shares), kNarrowThreads, 0, s, a.x, tall, p, q, parts, a.eps, held, shares);
    count_launch();
    for (int t = 0; t < a.steps && e == cudaSuccess; ++t) {
        const Mat out = t + 1 == a.steps ? a.out : Mat{nullptr, 0};
        e = launch_next(narrow_sum_kernel, dim3(kSumBlocks), kNarrowThreads, 0, s, (const float*)shares, n_shares, gram);
        count_launch();
        if (e == cudaSuccess)
            e = launch_next(narrow_step_kernel, dim3(n_shares), kNarrowThreads, kNarrowSmem, s, held, tall, p, q, (const float*)gram, a.a, a.b, a.c, a.scale,
                            shares, out);
        count_launch();
    }
    return e;
}

int log2_near(double v) { return (int)std::nearbyint(std::log2(v)); }
int log2_above(double v) { return (int)std::ceil(std::log2(v)); }

// The products of a step; which factor's rows are neighbours in memory goes by
// the longer side.
Product gram_product(int64_t p, int64_t q, int tall, const Mat& x) {
    return {p, p, 1, {q, 0}, {x, {}}, {x, {}}, tall, tall, 1, 0, 1};
}
Product square_product(int64_t p, const Mat& a) { return {p, p, 1, {p, 0}, {a, {}}, {a, {}}, 0, 0, 1, 0, 1}; }
Product next_product(int64_t rows, int64_t cols, const Mat& poly, const Mat& x) {
    if (rows > cols) return {rows, cols, 1, {cols, 0}, {x, {}}, {poly, {}}, 0, 0, 1, 0, 0};
    return {rows, cols, 1, {rows, 0}, {poly, {}}, {x, {}}, 0, 1, 1, 0, 0};
}
size_t sums_bytes(int64_t rows, int64_t cols) {
    const int64_t p = std::min(rows, cols), q = std::max(rows, cols);
    const size_t most = std::max({parts_bytes(gram_product(p, q, 0, {})), parts_bytes(square_product(p, {})), parts_bytes(next_product(rows, cols, {}, {}))});
    return (most + 255) / 256 * 256;
}

}  // namespace

size_t ortho_bytes(int64_t rows, int64_t cols) {
    if (rows == 0 || cols == 0) return 0;
    const int64_t p = rows < cols ? rows : cols;
    if (p <= kSide) return kPartsRoom + narrow_room(p, std::max(rows, cols));
    return kPartsRoom + 3 * aligned_room(rows, cols) + 2 * aligned_room(p, p) + sums_bytes(rows, cols);
}

namespace {
// What a step does to singular values from [0, s]: the most of |a s + b s^3 + c
// s^5|, and of that over s.
struct Reach {
    double value, growth;
};
Reach reach_of(double s, double a, double b, double c) {
    const double u = s * s, root = 9.0 * b * b - 20.0 * a * c;
    // of u = s^2: the range's end, and where the derivatives a + 3 b u + 5 c u^2 and b + 2 c u are 0
    double at[4] = {u, 0.0, 0.0, 0.0};
    if (root >= 0.0) {
        const double half = -0.5 * (3.0 * b + std::copysign(std::sqrt(root), b));
        if (c != 0.0) at[1] = half / (5.0 * c);
        if (half != 0.0) at[2] = a / half;
    }
    if (c != 0.0) at[3] = -b / (2.0 * c);
    Reach r = {0.0, std::fabs(a)};
    for (const double v : at) {
        if (!(v > 0.0 && v <= u)) continue;
        const double growth = std::fabs(a + b * v + c * v * v);
        r.value = std::max(r.value, std::sqrt(v) * growth);
        r.growth = std::max(r.growth, growth);
    }
    return r;
}
}  // namespace

double ortho_reach(int steps, double a, double b, double c) {
    double most = 1.0, s = 1.0;
    for (int t = 1; t < steps && most <= 2 * kMostReach; ++t) {
        s = reach_of(s, a, b, c).value;
        most = std::max(most, s);
    }
    return most;
}

cudaError_t launch_ortho(int dt, const OrthoArgs& a, cudaStream_t s) {
    if (a.rows == 0 || a.cols == 0) return cudaSuccess;
    const bool tall = a.rows > a.cols;
    const int64_t p = tall ? a.cols : a.rows, q = tall ? a.rows : a.cols;
    const size_t plane = aligned_room(a.rows, a.cols);
    const int64_t ld = whole_granules(a.cols), lp = whole_granules(p);
    double* parts = reinterpret_cast<double*>(a.work);
    char* w = a.work + kPartsRoom;
    Mat hi = {w, ld}, next = {w + plane, ld};
    const Mat lo = {w + 2 * plane, ld}, gram = {w + 3 * plane, lp}, poly = {w + 3 * plane + aligned_room(p, p), lp};
    float* sums = reinterpret_cast<float*>(w + 3 * plane + 2 * aligned_room(p, p));
    // Scales by powers of two that keep values in binary16's normal range: X's
    // elements are about 1/sqrt(p q) at first and 1/sqrt(q) at the end, never
    // above the largest singular value, `reach`; A's diagonal is about 1/p at
    // first, and nothing in it above reach^2; the polynomial's at most |a| +
    // |b| reach^2 + |c| reach^4.
    const double reach = std::max(ortho_reach(a.steps, a.a, a.b, a.c), std::sqrt(1.5)), square = reach * reach;
    const int sx = std::min(log2_near(std::sqrt((double)q)), 15 - log2_above(reach));
    const int sa = std::min({13, log2_near((double)p), 15 - log2_above(square)});
    const double most = std::fabs(a.a) + square * std::fabs(a.b) + square * square * std::fabs(a.c);
    const int sb = std::min(sa, 15 - log2_above(std::max(most, 1.0)));
    int* first_lift = reinterpret_cast<int*>(parts + 3 * kSquareBlocks);
    if (dt == FSDP_F32)
        square_kernel<float><<<kSquareBlocks, kSquareThreads, 0, s>>>(a.x, a.rows, a.cols, parts);
    else
        square_kernel<uint16_t><<<kSquareBlocks, kSquareThreads, 0, s>>>(a.x, a.rows, a.cols, parts);
    count_launch();
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (p <= kSide) return dt == FSDP_F32 ? narrow<float>(a, s) : narrow<uint16_t>(a, s);
    const int64_t granules = a.rows * ((a.cols + kGran - 1) / kGran);
    const int grid = (int)std::min<int64_t>((granules + 255) / 256, 8 * sm_count());
    e = dt == FSDP_F32 ? launch_next(planes_kernel<float>, dim3(grid), 256, 0, s, a.x, a.rows, a.cols, (const double*)parts, a.eps, sx, hi, lo, first_lift)
                       : launch_next(planes_kernel<uint16_t>, dim3(grid), 256, 0, s, a.x, a.rows, a.cols, (const double*)parts, a.eps, sx, hi, lo, first_lift);
    count_launch();
    double from = 1.0;
    Lift lift = {first_lift, 0, 0};
    for (int i = 0; i < a.steps && e == cudaSuccess; ++i) {
        const float shift = i + 2 < a.steps ? a.a : 0.5f * (1.0f + a.a);
        e = launch_product(gram_product(p, q, tall, hi), Gram{gram, std::ldexp(1.0f, sa - 2 * sx)}, sums, s, false);
        const Poly mix = {gram, poly, std::ldexp(a.c, sb - 2 * sa), std::ldexp(a.b, sb - sa), std::ldexp(a.a - shift, sb), lift};
        if (e == cudaSuccess) e = launch_product(square_product(p, gram), mix, sums, s, false);
        const bool last = i + 1 == a.steps;
        const float out = last ? std::ldexp(a.scale, -sx) : 1.0f;
        const Reach step = reach_of(from, a.a, a.b, a.c);
        const int grown = std::max(-16, log2_above(std::max(step.growth, 0x1p-20)));
        const Lift after = {first_lift, lift.less + grown, std::max(0, lift.least - grown)};
        if (e == cudaSuccess)
            e = launch_product(next_product(a.rows, a.cols, poly, hi),
                               Next{hi, lo, next, last ? a.out : Mat{nullptr, 0}, std::ldexp(out, -sb), shift * out, lift, after}, sums, s, false);
        lift = after;
        from = step.value;
        std::swap(hi, next);
    }
    return e;
}

cudaError_t ortho_gave_up(int* value, cudaStream_t s) { return take_gave_up(value, s); }

}  // namespace fsdp
