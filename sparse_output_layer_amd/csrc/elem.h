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
typedef __attribute__((ext_vector_type(2), aligned(2))) unsigned u32x2h;
typedef __attribute__((ext_vector_type(2), aligned(4))) float f32x2u;
typedef __attribute__((aligned(2))) unsigned u32h;

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
// The eight elements from column c (a multiple of 8) of a row of D, i the
// element's index; past the row's end zeros, or with LAST the row's last element
// in a vector that holds it.  tail (the same for the wave): the vector may be one
// that the row ends inside.  Such a one is read as the row's last eight elements,
// one access whatever is left, and unpack8n, which is when they have to be there,
// shifts them down.
template <bool BF, bool LAST = false>
__device__ __forceinline__ Raw8<BF> raw8n(const void *p, int64_t i, int c, int D, bool tail) {
    Raw8<BF> r;
#pragma unroll
    for (int k = 0; k < (BF ? 1 : 2); ++k) r.w[k] = (u32x4){0u, 0u, 0u, 0u};
    if (tail && D < 8) {                             // a row of fewer than eight
        if (c > 0) return r;
        constexpr int N = BF ? 4 : 8;
        if (LAST && D > 0) {
            const unsigned e = BF ? ((const unsigned short *)p)[i + D - 1] * 0x10001u : ((const unsigned *)p)[i + D - 1];
#pragma unroll
            for (int j = 0; j < N; ++j) r.w[j / 4][j % 4] = e;
        }
#pragma unroll 1
        for (int e = D - 1; e >= 0; --e) {
#pragma unroll
            for (int j = N - 1; j >= 0; --j) {
                const unsigned below = j ? r.w[(j ? j - 1 : 0) / 4][(j ? j - 1 : 0) % 4] : 0u;
                r.w[j / 4][j % 4] = BF ? r.w[j / 4][j % 4] << 16 | below >> 16 : below;
            }
            r.w[0][0] |= BF ? ((const unsigned short *)p)[i + e] : ((const unsigned *)p)[i + e];
        }
        return r;
    }
    if (c < D) {
        const int64_t at = i - (tail ? max(0, c - (D - 8)) : 0);
        if (BF) {
            r.w[0] = *(const u32x4h *)((const unsigned short *)p + at);
        } else {
            r.w[0] = *(const u32x4w *)((const unsigned *)p + at);
            r.w[BF ? 0 : 1] = *(const u32x4w *)((const unsigned *)p + at + 4);
        }
    }
    return r;
}
// raw8n's elements as floats
template <bool BF, bool LAST = false>
__device__ __forceinline__ void unpack8n(const Raw8<BF> &r, int c, int D, bool tail, float *v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (BF) v[j] = __uint_as_float(j & 1 ? r.w[0][j >> 1] & 0xffff0000u : r.w[0][j >> 1] << 16);
        else v[j] = __uint_as_float(r.w[BF ? 0 : j >> 2][j & 3]);
    }
    if (tail && D > 8) {
        const int s = max(0, c - (D - 8));             // 8 and more: zeros as they are
#pragma unroll
        for (int e = 4; e > 0; e >>= 1)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = !(s & e) ? v[j] : j + e < 8 ? v[j + e] : LAST ? v[7] : 0.f;
    }
}
// both at once, `other` past the end
template <bool BF>
__device__ __forceinline__ void load8n(const void *p, int64_t i, int c, int D, float other, float *v) {
    const bool tail = (D & 7) != 0;
    unpack8n<BF>(raw8n<BF>(p, i, c, D, tail), c, D, tail, v);
    if (c > D - 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < D - c ? v[j] : other;
    }
}
// the first n of eight, in pieces of four, two and one
template <bool BF>
__device__ __forceinline__ void store8n(void *p, int64_t i, int n, const float *v) {
    if (n >= 8) {
        store8<BF>(p, i, v);
        return;
    }
    if (n <= 0) return;
    float t[4] = {v[0], v[1], v[2], v[3]};
    if (n & 4) {
        if (BF) *(u32x2h *)((unsigned short *)p + i) = (u32x2){pack_bf16x2(t[0], t[1]), pack_bf16x2(t[2], t[3])};
        else *(f32x4u *)((float *)p + i) = (f32x4u){t[0], t[1], t[2], t[3]};
        i += 4;
#pragma unroll
        for (int j = 0; j < 3; ++j) t[j] = v[4 + j];
    }
    if (n & 2) {
        if (BF) *(u32h *)((unsigned short *)p + i) = pack_bf16x2(t[0], t[1]);
        else *(f32x2u *)((float *)p + i) = (f32x2u){t[0], t[1]};
        i += 2;
        t[0] = t[2];
    }
    if (n & 1) store1<BF>(p, i, t[0]);
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
