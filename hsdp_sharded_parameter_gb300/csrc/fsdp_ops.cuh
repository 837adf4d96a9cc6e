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

// The types as the kernels hold them.
template <int DT>
struct ElemOf {
    using type = float;
};
template <>
struct ElemOf<FSDP_BF16> {
    using type = uint16_t;
};

// The n (1..8) columns from c on of a row, at any alignment; the others are
// zero. A shifted granule is put together from the 16-byte blocks that hold
// it, each of which has at least one byte of the row.
template <typename T>
__device__ __forceinline__ void load_granule(Raw<T>& r, const T* row, int64_t c, int n) {
    if (n == kGran) {
        load_raw_at<T>(r, reinterpret_cast<uintptr_t>(row + c));
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
    const int nextn = __shfl_down_sync(kFull, n, 1);
    const int head = (int)sh / (int)sizeof(T);  // elements of the first block below p
    if (n == kGran && lane > 0) {
        uint4* q = reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(p) - sh);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const uint4 lo = v == 0 ? below : make_uint4(r.w[4 * v - 4], r.w[4 * v - 3], r.w[4 * v - 2], r.w[4 * v - 1]);
            const uint4 hi = make_uint4(r.w[4 * v], r.w[4 * v + 1], r.w[4 * v + 2], r.w[4 * v + 3]);
            st_stream(q + v, funnel(lo, hi, 16u - sh));
        }
    }
    // what no whole block of this or the next lane covers: the span's first
    // kGran - head elements, a short granule, and the last head elements of a
    // granule whose upper neighbour stores no whole block
    const bool whole = n == kGran && lane > 0;
    const bool covered = lane < 31 && nextn == kGran;
    const int first = whole ? kGran - head : 0;
    const int last = covered ? kGran - head : n;
#pragma unroll
    for (int e = 0; e < kGran; ++e)
        if (e >= first && e < last) store_elem(p + e, r, e);
}

// ------------------------------------------------------------- dropout mask

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011).
__device__ __forceinline__ uint4 philox(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = (uint64_t)0xD2511F53u * c.x, b = (uint64_t)0xCD9E8D57u * c.z;
        c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ k0, (uint32_t)b, (uint32_t)(a >> 32) ^ c.w ^ k1, (uint32_t)a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}

// Drops and scales the 8 columns 8 * block ... of a row. One generator block
// serves them, 16 bits each: with 32 bits each, two blocks, the generator's
// multiplications bound the kernel (1 GiB of bf16 on one GB300: 5004 GB/s
// against 6563, and 6928 for the copy alone).
__device__ __forceinline__ void drop(float (&x)[8], const Mask& m, int64_t row, uint32_t block) {
    const uint4 r = philox(make_uint4(block, (uint32_t)row, (uint32_t)((uint64_t)row >> 32), m.draw), m.key0, m.key1);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = (w[i] & 0xffffu) < m.limit ? x[2 * i] * m.scale : 0.0f;
        x[2 * i + 1] = (w[i] >> 16) < m.limit ? x[2 * i + 1] * m.scale : 0.0f;
    }
}

// -------------------------------------------------------------------- sums

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}

// Columns of granule g of a row, 0 past its end.
__device__ __forceinline__ int granule_cols(int64_t g, int64_t cols) {
    const int64_t left = cols - g * kGran;
    return left >= kGran ? kGran : (left > 0 ? (int)left : 0);
}

}  // namespace
}  // namespace fsdp
