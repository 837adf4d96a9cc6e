// Device helpers of the training operators: granules of 8 columns at any
// alignment, the counter-based dropout mask, sums over a warp. Included by
// the operators' translation units only.
#pragma once

#include "fsdp_device.cuh"
#include "fsdp_ops.h"

namespace fsdp {
namespace {

// A lane holds granules of 8 consecutive columns, a warp a span of 256.
constexpr int kSpan = 32 * kGran;

// Bytes [sh, sh + 16) of the 32-byte string lo:hi, sh below 16 and a multiple
// of T's size: two rounds of selections by sh's bits, and for 16-bit elements
// a shift. (Beside the data path's funnel, which branches on sh: 16384 rows of
// 5001 bf16, the norm with dropout and residual takes 268 us by this and 278 by
// that, its gradient 358 and 374; the dropout of 32768 275 and 223, lookups 115
// and 113.)
template <typename T>
__device__ __forceinline__ uint4 shifted(uint4 lo, uint4 hi, unsigned sh) {
    const bool two = sh & 8u, one = sh & 4u;
    const uint32_t a0 = two ? lo.z : lo.x, a1 = two ? lo.w : lo.y, a2 = two ? hi.x : lo.z, a3 = two ? hi.y : lo.w;
    const uint32_t a4 = two ? hi.z : hi.x, a5 = two ? hi.w : hi.y;
    uint4 v = make_uint4(one ? a1 : a0, one ? a2 : a1, one ? a3 : a2, one ? a4 : a3);
    if (sizeof(T) == 2) {
        const uint32_t last = one ? a5 : a4;
        const unsigned r = (sh & 2u) * 8u;
        v = make_uint4(__funnelshift_r(v.x, v.y, r), __funnelshift_r(v.y, v.z, r), __funnelshift_r(v.z, v.w, r),
                       __funnelshift_r(v.w, last, r));
    }
    return v;
}

// The n (1..8) columns from c on of a row, at any alignment; the others are
// zero. A shifted granule is put together from the 16-byte blocks that hold
// it, each of which has at least one byte of the row.
template <typename T>
__device__ __forceinline__ void load_granule(Raw<T>& r, const T* row, int64_t c, int n) {
    constexpr int kV = Raw<T>::kVec;
    if (n == kGran) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
        const unsigned sh = (unsigned)(at & 15u);
        const uint4* q = reinterpret_cast<const uint4*>(at - sh);
        if (sh == 0) {
#pragma unroll
            for (int v = 0; v < kV; ++v) put(r.w + 4 * v, ld_stream(q + v));
        } else {
            uint4 b[kV + 1];
#pragma unroll
            for (int v = 0; v <= kV; ++v) b[v] = ld_reuse(q + v);
#pragma unroll
            for (int v = 0; v < kV; ++v) put(r.w + 4 * v, shifted<T>(b[v], b[v + 1], sh));
        }
        return;
    }
    zero_raw(r);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < kGran; ++e)
            if (e < n) r.w[e] = reinterpret_cast<const uint32_t*>(row)[c + e];
    } else {
#pragma unroll
        for (int e = 0; e < kGran; ++e)
            if (e < n) r.w[e >> 1] |= (uint32_t)row[c + e] << ((e & 1) * 16);
    }
}

template <typename T>
__device__ __forceinline__ void store_elem(T* p, const Raw<T>& r, int e) {
    if constexpr (sizeof(T) == 4)
        *reinterpret_cast<uint32_t*>(p) = r.w[e];
    else
        *p = (T)(r.w[e >> 1] >> ((e & 1) * 16));
}

// Stores a warp's span of granules at any alignment: lane l holds the n
// (0..8; less than 8 only past a row's end) columns at p, lane l + 1 those
// behind them. All 32 lanes take part. Where p is off the 16-byte grid by sh
// bytes, a lane stores the aligned blocks that end inside its granule, the
// first of them begun by the lane below: whole 16-byte stores but for the
// span's two ends, where element stores by 8 columns a lane would cost eight
// times the store instructions.
template <typename T>
__device__ __forceinline__ void store_span(T* p, const Raw<T>& r, int n, int lane) {
    constexpr int kV = Raw<T>::kVec;
    const unsigned sh = (unsigned)(reinterpret_cast<uintptr_t>(p) & 15u);  // the same in all lanes
    if (sh == 0) {
        if (n == kGran)
            store_raw(p, r);
        else
#pragma unroll
            for (int e = 0; e < kGran; ++e)
                if (e < n) store_elem(p + e, r, e);
        return;
    }
    const uint32_t* l = r.w + 4 * (kV - 1);
    uint4 below;
    below.x = __shfl_up_sync(kFull, l[0], 1);
    below.y = __shfl_up_sync(kFull, l[1], 1);
    below.z = __shfl_up_sync(kFull, l[2], 1);
    below.w = __shfl_up_sync(kFull, l[3], 1);
    const int head = (int)sh / (int)sizeof(T);  // elements of the first block below p
    if (n == kGran && lane > 0) {
        uint4* q = reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(p) - sh);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const uint4 lo = v == 0 ? below : make_uint4(r.w[4 * v - 4], r.w[4 * v - 3], r.w[4 * v - 2], r.w[4 * v - 1]);
            const uint4 hi = make_uint4(r.w[4 * v], r.w[4 * v + 1], r.w[4 * v + 2], r.w[4 * v + 3]);
            st_stream(q + v, shifted<T>(lo, hi, 16u - sh));
        }
    }
    if (__all_sync(kFull, n == kGran)) {
        // the first lane's elements before the second's block, and the last
        // lane's behind its own: eight in all, one for each of the first lanes
        const int e = lane & 7, from = e < kGran - head ? 0 : 31;
        uint32_t v = 0;
#pragma unroll
        for (int i = 0; i < Raw<T>::kWords; ++i) {
            const uint32_t x = __shfl_sync(kFull, r.w[i], from);
            v = i == e * (int)sizeof(T) / 4 ? x : v;
        }
        if (lane < 8) {
            T* q = p - lane * kGran + (from ? 31 * kGran : 0) + e;
            if constexpr (sizeof(T) == 4)
                *reinterpret_cast<uint32_t*>(q) = v;
            else
                *q = (T)(v >> ((e & 1) * 16));
        }
        return;
    }
    // a row's last span. What no whole block of this or the next lane covers:
    // the first lane's first kGran - head elements, a short granule, and the
    // last head elements of a granule whose upper neighbour stores no block
    const int nextn = __shfl_down_sync(kFull, n, 1);
    const bool whole = n == kGran && lane > 0;
    const bool covered = lane < 31 && nextn == kGran;
    const int first = whole ? kGran - head : 0;
    const int last = covered ? kGran - head : n;
#pragma unroll
    for (int e = 0; e < kGran; ++e)
        if (e >= first && e < last) store_elem(p + e, r, e);
}

// A granule stored by one thread, at any alignment.
template <typename T>
__device__ __forceinline__ void store_granule(T* p, const Raw<T>& r, int n) {
    if (n == kGran && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        store_raw(p, r);
    } else {
#pragma unroll
        for (int e = 0; e < kGran; ++e)
            if (e < n) store_elem(p + e, r, e);
    }
}

// Narrow rows: kernels that give a warp a span of a row would leave most of
// its lanes or of its loads unused, so a thread takes granules of any rows,
// kNarrow of them. On one GB300, dropout of 32768 rows of bf16 with a residual,
// by threads and by spans: 20 columns 7 and 25 us, 200 10 and 27, 1000 35 and
// 31. Off the 16-byte grid a thread stores element by element, and spans are
// ahead sooner (lookup of 32768 tokens, 201 columns: 21 and 14 us).
constexpr int kNarrow = 4, kNarrowCols = 512, kNarrowShifted = 96;
inline bool narrow_rows(int64_t rows, int64_t cols, bool aligned) {
    return cols <= (aligned ? kNarrowCols : kNarrowShifted) && rows * ((cols + kGran - 1) / kGran) < ((int64_t)1 << 31);
}

// The granules of a warp's span, as load_granule and store_span do them, where
// kAligned says that every row starts on the 16-byte grid and holds whole
// granules (n is 8, or 0 past the row's end).
template <bool kAligned, typename T>
__device__ __forceinline__ void load_cols(Raw<T>& r, const T* row, int64_t c, int n) {
    if constexpr (!kAligned)
        load_granule(r, row, c, n);
    else if (n)
        load_aligned(r, row + c);
}
template <bool kAligned, typename T>
__device__ __forceinline__ void store_cols(T* p, const Raw<T>& r, int n, int lane) {
    if constexpr (!kAligned)
        store_span(p, r, n, lane);
    else if (n)
        store_raw(p, r);
}

// The 8 columns of a granule in binary32, as pairs: one instruction works on
// two values, and these kernels are bound by instructions before memory.
struct Cols {
    float2 p[4];
    __device__ __forceinline__ float get(int e) const { return e & 1 ? p[e >> 1].y : p[e >> 1].x; }
    __device__ __forceinline__ void set(int e, float v) {
        if (e & 1)
            p[e >> 1].y = v;
        else
            p[e >> 1].x = v;
    }
};
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ Cols all(float v) { return {{both(v), both(v), both(v), both(v)}}; }
__device__ __forceinline__ Cols operator+(const Cols& a, const Cols& b) {
    Cols r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = __fadd2_rn(a.p[i], b.p[i]);
    return r;
}
__device__ __forceinline__ Cols operator*(const Cols& a, const Cols& b) {
    Cols r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = __fmul2_rn(a.p[i], b.p[i]);
    return r;
}
__device__ __forceinline__ Cols fma(const Cols& a, const Cols& b, const Cols& c) {
    Cols r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = __ffma2_rn(a.p[i], b.p[i], c.p[i]);
    return r;
}
// Sums over a granule, two columns at a time.
__device__ __forceinline__ void sum_into(float2& s, const Cols& a) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __fadd2_rn(s, a.p[i]);
}
__device__ __forceinline__ void dot_into(float2& s, const Cols& a, const Cols& b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __ffma2_rn(a.p[i], b.p[i], s);
}

__device__ __forceinline__ Cols widened(const Raw<uint16_t>& r) {
    Cols x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x.p[i] = make_float2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xffff0000u));
    return x;
}
__device__ __forceinline__ Cols widened(const Raw<float>& r) {
    Cols x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x.p[i] = make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
    return x;
}
// Rounded to a granule, NaN to some NaN: the data path's rule for a NaN's bits
// takes eight comparisons a granule, and no sum here keeps them.
__device__ __forceinline__ void round_to(const Cols& x, Raw<uint16_t>& r) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.w[i]) : "f"(x.p[i].y), "f"(x.p[i].x));
}
__device__ __forceinline__ void round_to(const Cols& x, Raw<float>& r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.w[2 * i] = __float_as_uint(x.p[i].x);
        r.w[2 * i + 1] = __float_as_uint(x.p[i].y);
    }
}
// Columns past a row's end become 0.
__device__ __forceinline__ void cut(Cols& x, int n) {
    if (n == kGran) return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e >= n) x.set(e, 0.0f);
}

// -------------------------------------------------- rows on their way in

// A warp's span of one row in shared memory, filled by asynchronous 16-byte
// copies: the granules' blocks and, for a row off the 16-byte grid, one more.
// The blocks are copied in the order of memory (a lane's own 32 bytes of fp32
// would make every copy half a sector), so a warp meets between its copies'
// arrival and its reads, and again before the next copies.
template <bool kAligned, typename T>
constexpr int kSlot = 32 * Raw<T>::kVec + (kAligned ? 0 : 1);

// kCached: through the L1 cache, for what an SM reads again.
template <bool kCached>
__device__ __forceinline__ void async_copy(uint4* dst, uintptr_t src) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (kCached)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Starts the copies of the 16-byte blocks that hold a row's columns c0 ...
// c0 + 255; no block that lies wholly past the row's end is touched.
template <bool kAligned, bool kCached = false, typename T>
__device__ __forceinline__ void span_fetch(uint4* slot, const T* row, int c0, int cols, int lane) {
    constexpr int kV = Raw<T>::kVec;
    const uintptr_t from = reinterpret_cast<uintptr_t>(row + c0);
    const int sh = kAligned ? 0 : (int)(from & 15u);
    const int bytes = cols > c0 ? (cols - c0) * (int)sizeof(T) + sh : 0;  // all of the row's: blocks past the span are not asked for
#pragma unroll
    for (int v = 0; v < kV + (kAligned ? 0 : 1); ++v) {
        const int b = v * 32 + lane;
        if ((v < kV || lane == 0) && b * 16 < bytes) async_copy<kCached>(slot + b, from - sh + b * 16);
    }
}

// The lane's granule of a span that has arrived; what it holds past the row's
// end is not defined.
template <bool kAligned, typename T>
__device__ __forceinline__ void span_read(Raw<T>& r, const uint4* slot, const T* row, int c0, int lane) {
    constexpr int kV = Raw<T>::kVec;
    const unsigned sh = kAligned ? 0u : (unsigned)(reinterpret_cast<uintptr_t>(row + c0) & 15u);
    uint4 b[kV + 1];
#pragma unroll
    for (int v = 0; v < kV; ++v) b[v] = slot[lane * kV + v];
    if (kAligned || sh == 0) {
#pragma unroll
        for (int v = 0; v < kV; ++v) put(r.w + 4 * v, b[v]);
        return;
    }
    b[kV] = slot[lane * kV + kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) put(r.w + 4 * v, shifted<T>(b[v], b[v + 1], sh));
}

// ------------------------------------------------------------- dropout mask

// Adds to y the dropout of x, the 8 columns 8 * block ... of a row. The
// generator is Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011). One block of it serves 8 columns, 16
// bits each: with 32 bits each, two blocks, its multiplications bound the
// kernel (1 GiB of bf16 on one GB300: 5004 GB/s against 6563, and 6928 for the
// copy alone).
__device__ __forceinline__ void add_dropped(Cols& y, const Cols& x, const Mask& m, int64_t row, uint32_t block) {
    uint32_t c0 = block, c1 = (uint32_t)row, c2 = (uint32_t)((uint64_t)row >> 32), c3 = m.draw;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ m.key[2 * i];
        c2 = (uint32_t)(a >> 32) ^ c3 ^ m.key[2 * i + 1];
        c1 = (uint32_t)b;
        c3 = (uint32_t)a;
    }
    const uint32_t w[4] = {c0, c1, c2, c3};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // a word's lower bits do not decide on its upper half
        if (w[i] << 16 < m.limit) y.p[i].x = __fmaf_rn(x.p[i].x, m.scale, y.p[i].x);
        if (w[i] < m.limit) y.p[i].y = __fmaf_rn(x.p[i].y, m.scale, y.p[i].y);
    }
}

// -------------------------------------------------------------------- sums

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}

// A row of a matrix whose row stride is below 2^32 bytes: one multiply-add.
template <typename T>
__device__ __forceinline__ T* row_at(void* data, uint32_t row, uint32_t stride_bytes) {
    return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(data) + (uint64_t)row * stride_bytes);
}

// Columns of granule g of a row, 0 past its end.
template <typename I>
__device__ __forceinline__ int granule_cols(I g, I cols) {
    const I left = cols - g * kGran;
    return left >= kGran ? kGran : (left > 0 ? (int)left : 0);
}

// ----------------------------------------------------- launches in a chain

// A kernel that follows another of the same call may be launched before that
// one has ended (programmatic dependent launch), so that its start costs no
// time of its own; it waits here before it touches what the other wrote.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel's blocks start as soon as all of this one's have.
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... A>
cudaError_t launch_next(void (*kernel)(A...), dim3 grid, int block, int smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
}  // namespace fsdp
