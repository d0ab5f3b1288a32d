// rows.h -- rows of features held in the registers of the threads that share
// them: row sums, row ends and weights, for the norms (norm.hip, addnorm.hip,
// addnorm_bwd.hip) and the embedding (embed.hip).
#pragma once
#include "elem.h"

namespace haste {

// ---- rows spread over TPR threads: 8, 16, 32 or 64 lanes of a wave, or several waves

// Sum over a row's TPR threads in a fixed order; every thread of the row gets
// it.  s: LDS room for two sums' partials a wave, used alternately (`turn`), so
// that one barrier a sum is enough.
template <int TPR, int NTH>
__device__ __forceinline__ float row_sum(float v, float (*s)[NTH / 64], int &turn) {
    if (TPR <= 16) {
        v += dpp_f32<0xB1>(v);
        v += dpp_f32<0x4E>(v);
        v += dpp_f32<0x141>(v);
        return TPR == 8 ? v : v + dpp_f32<0x140>(v);
    }
    if (TPR == 32) {
        v += dpp_f32<0xB1>(v);
        v += dpp_f32<0x4E>(v);
        v += dpp_f32<0x141>(v);
        v += dpp_f32<0x140>(v);
        const float lo = lane_f32(v, 0) + lane_f32(v, 16), hi = lane_f32(v, 32) + lane_f32(v, 48);
        return (threadIdx.x & 32) ? hi : lo;
    }
    v = wave_sum_dpp(v);
    if (TPR == 64) return v;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) s[turn][threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.f;
    const int first = (int)threadIdx.x / TPR * (TPR / 64);
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) t += s[turn][first + i];
    return t;
}
template <int TPR, int NTH>
__device__ __forceinline__ void row_sum2(float &a, float &b, float (*s)[NTH / 64], float (*q)[NTH / 64], int &turn) {
    if (TPR <= 64) {
        a = row_sum<TPR, NTH>(a, s, turn);
        b = row_sum<TPR, NTH>(b, q, turn);
        return;
    }
    a = wave_sum_dpp(a);
    b = wave_sum_dpp(b);
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
        s[turn][threadIdx.x >> 6] = a;
        q[turn][threadIdx.x >> 6] = b;
    }
    __syncthreads();
    a = b = 0.f;
    const int first = (int)threadIdx.x / TPR * (TPR / 64);
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) {
        a += s[turn][first + i];
        b += q[turn][first + i];
    }
}

// A kernel's rows end inside a vector (TAIL) or never do, which is decided at the
// launch: aligned rows pay nothing for the others (dropout of 65536 x 1024 bf16: 48.8
// us, 52.5 with the tests in).  Of a thread's vectors only this one can hold a
// row's end.
template <bool TAIL, int TPR>
__device__ __forceinline__ int tail_of(int D) {
    return TAIL && (D & 7) ? D / 8 / TPR : -1;
}
template <bool TAIL, bool BF>
__device__ __forceinline__ void put8(void *p, int64_t i, int n, const float *v) {
    if (TAIL) store8n<BF>(p, i, n, v);
    else if (n > 0) store8<BF>(p, i, v);
}

// eight weights from column c (1 or 0 where there are none)
__device__ __forceinline__ void load_w8(const void *w, bool bf, int c, int D, float none, float *v) {
    if (w && c < D) {
        if (bf) load8n<true>(w, c, c, D, none, v);
        else load8n<false>(w, c, c, D, none, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = none;
    }
}

// the same value, not known to be: loads at it stay inside the loop they stand in
__device__ __forceinline__ int opaque_index(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// F<o, r, y are bf16, the rows end inside a vector>(a, st), of the types and width in a
#define HASTE_PICK_TYPES(F, a, st)                                                              \
    const int pick_ = a.obf * 8 + a.rbf * 4 + a.ybf * 2 + ((a.D & 7) != 0);                     \
    switch (pick_) {                                                                            \
    case 0: return F<false, false, false, false>(a, st);                                        \
    case 1: return F<false, false, false, true>(a, st);                                         \
    case 2: return F<false, false, true, false>(a, st);                                         \
    case 3: return F<false, false, true, true>(a, st);                                          \
    case 4: return F<false, true, false, false>(a, st);                                         \
    case 5: return F<false, true, false, true>(a, st);                                          \
    case 6: return F<false, true, true, false>(a, st);                                          \
    case 7: return F<false, true, true, true>(a, st);                                           \
    case 8: return F<true, false, false, false>(a, st);                                         \
    case 9: return F<true, false, false, true>(a, st);                                          \
    case 10: return F<true, false, true, false>(a, st);                                         \
    case 11: return F<true, false, true, true>(a, st);                                          \
    case 12: return F<true, true, false, false>(a, st);                                         \
    case 13: return F<true, true, false, true>(a, st);                                          \
    case 14: return F<true, true, true, false>(a, st);                                          \
    default: return F<true, true, true, true>(a, st);                                           \
    }

}  // namespace haste
