// elem.h -- element access and the counter-based generator, shared by the
// operators around the layer (norm.hip, logprob.hip, head_i8.hip).
#pragma once
#include "common.h"
#include "kernels.h"

namespace haste {

template <bool BF>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    return BF ? bf16_to_f32(((const unsigned short *)p)[i]) : ((const float *)p)[i];
}
template <bool BF>
__device__ __forceinline__ void store1(void *p, int64_t i, float v) {
    if (BF) ((unsigned short *)p)[i] = f32_to_bf16(v);
    else ((float *)p)[i] = v;
}

// Eight elements as they lie in memory, to be unpacked when they are used: a
// row's vectors can be on their way while the row before it is worked on.
template <bool BF>
struct Raw8 {
    u32x4 w[BF ? 1 : 2];
};

// Wave reductions on DPP operands: within rows of 16 lanes, then the four rows'
// results through scalar registers; a fixed order, every lane gets the result.
__device__ __forceinline__ unsigned lane_u32(unsigned v, int lane) {
    return (unsigned)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ __forceinline__ float lane_f32(float v, int lane) { return __uint_as_float(lane_u32(__float_as_uint(v), lane)); }
__device__ __forceinline__ float wave_sum_dpp(float v) {
    v += dpp_f32<0xB1>(v);
    v += dpp_f32<0x4E>(v);
    v += dpp_f32<0x141>(v);
    v += dpp_f32<0x140>(v);
    return (lane_f32(v, 0) + lane_f32(v, 16)) + (lane_f32(v, 32) + lane_f32(v, 48));
}
__device__ __forceinline__ unsigned wave_max_dpp(unsigned v) {
    v = max(v, dpp_u32<0xB1>(v));
    v = max(v, dpp_u32<0x4E>(v));
    v = max(v, dpp_u32<0x141>(v));
    v = max(v, dpp_u32<0x140>(v));
    return max(max(lane_u32(v, 0), lane_u32(v, 16)), max(lane_u32(v, 32), lane_u32(v, 48)));
}
// Vectors at any element of the type: rows of odd widths and strides start
// anywhere, and the hardware's wide accesses take any alignment of the type.
typedef __attribute__((ext_vector_type(4), aligned(2))) unsigned u32x4h;
typedef __attribute__((ext_vector_type(4), aligned(4))) unsigned u32x4w;
typedef __attribute__((ext_vector_type(4), aligned(4))) float f32x4u;

// eight elements from element i
template <bool BF>
__device__ __forceinline__ void load8(const void *p, int64_t i, float *v) {
    if (BF) {
        const u32x4 t = *(const u32x4h *)((const unsigned short *)p + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(j & 1 ? t[j >> 1] & 0xffff0000u : t[j >> 1] << 16);
    } else {
        const f32x4 a = *(const f32x4u *)((const float *)p + i), b = *(const f32x4u *)((const float *)p + i + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    }
}
template <bool BF>
__device__ __forceinline__ void store8(void *p, int64_t i, const float *v) {
    if (BF) {
        *(u32x4h *)((unsigned short *)p + i) = (u32x4){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                       pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    } else {
        *(f32x4u *)((float *)p + i) = (f32x4){v[0], v[1], v[2], v[3]};
        *(f32x4u *)((float *)p + i + 4) = (f32x4){v[4], v[5], v[6], v[7]};
    }
}
// the first n (0 .. 8) of eight; the others read as `other` / are not written
template <bool BF>
__device__ __forceinline__ void load8n(const void *p, int64_t i, int n, float other, float *v) {
    if (n >= 8) {
        load8<BF>(p, i, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? load1<BF>(p, i + j) : other;
}
template <bool BF>
__device__ __forceinline__ void store8n(void *p, int64_t i, int n, const float *v) {
    if (n >= 8) {
        store8<BF>(p, i, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < n) store1<BF>(p, i + j, v[j]);
}

template <bool BF>
__device__ __forceinline__ Raw8<BF> raw8n(const void *p, int64_t i, int n) {
    Raw8<BF> r;
    if (n >= 8) {
        if (BF) {
            r.w[0] = *(const u32x4h *)((const unsigned short *)p + i);
        } else {
            r.w[0] = *(const u32x4w *)((const unsigned *)p + i);
            r.w[BF ? 0 : 1] = *(const u32x4w *)((const unsigned *)p + i + 4);
        }
        return r;
    }
#pragma unroll
    for (int k = 0; k < (BF ? 1 : 2); ++k) r.w[k] = (u32x4){0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 7; ++j) {
        if (j >= n) continue;
        if (BF) r.w[0][j >> 1] |= (unsigned)((const unsigned short *)p)[i + j] << (16 * (j & 1));
        else r.w[BF ? 0 : j >> 2][j & 3] = ((const unsigned *)p)[i + j];
    }
    return r;
}
template <bool BF>
__device__ __forceinline__ void unpack8(const Raw8<BF> &r, float *v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (BF) v[j] = __uint_as_float(j & 1 ? r.w[0][j >> 1] & 0xffff0000u : r.w[0][j >> 1] << 16);
        else v[j] = __uint_as_float(r.w[BF ? 0 : j >> 2][j & 3]);
    }
}

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as
// easy as 1, 2, 3", 2011): ten rounds of two 32 x 32 -> 64-bit products, the
// key advanced by two odd constants after each round.
__device__ __forceinline__ u32x4 philox10(unsigned c0, unsigned c1, unsigned c2, unsigned c3, unsigned k0,
                                          unsigned k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
        c0 = (unsigned)(p1 >> 32) ^ c1 ^ k0;
        c1 = (unsigned)p1;
        c2 = (unsigned)(p0 >> 32) ^ c3 ^ k1;
        c3 = (unsigned)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return (u32x4){c0, c1, c2, c3};
}

// Dropout of the eight elements 8v .. 8v+7 of row r, in place: element j's 16
// bits are the low (j even) or high half of word j / 2, compared in the word's
// upper half.
__device__ __forceinline__ void drop8(const DropArgs &d, unsigned v, unsigned r, float *a) {
    if (d.thr > 0xffffu) {      // p = 1 (uniform)
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = 0.f;
        return;
    }
    const u32x4 w = philox10(v, r, d.o0, d.o1, d.k0, d.k1);
    const unsigned t = d.thr << 16;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const unsigned h = j & 1 ? w[j >> 1] : w[j >> 1] << 16;
        const float y = a[j] * d.scale;
        a[j] = h >= t ? y : 0.f;
    }
}

}  // namespace haste
