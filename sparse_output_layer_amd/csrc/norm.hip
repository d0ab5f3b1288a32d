// norm.hip -- layer norm (forward, backward, weight gradient) and dropout
// from a counter-based generator.
//
// All of it is bound by memory: every element is read once and written once,
// in vectors of eight (one generator call's worth), a row's elements staying
// in the registers of the threads that share it from the mean to the result.
// Times are a kernel's on one MI355X, where a copy of 1 GiB moves 5.2 TB/s
// (read and written); less than 256 MB of inputs partly come from the last
// cache, which lets a kernel pass that rate.
#include "elem.h"

namespace haste {

namespace {

constexpr int NT = 256;

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

}  // namespace

// ---------------------------------------------------------------- dropout
// y = x / (1 - p) where the element's 16 random bits reach p 65536, else 0.
// Element (r, c) takes half-word c % 8 of the generator's block (c / 8, r), so
// forward and backward form the same mask and none is stored.  A thread a
// vector of eight elements and one generator call; rows and columns advance
// without a division.  65536 x 1024 bf16: 42.5 us, 6.3 TB/s; 512 x 768 fp32:
// 2.9 us, the launch.  The generator's 20 wide products a vector are hidden
// behind the memory.
template <bool XB, bool YB, bool TAIL>
__global__ __launch_bounds__(NT) void k_dropout(int B, int D, const void *x, DropArgs d, void *y) {
    const unsigned nv = ((unsigned)D + 7) / 8;
    const uint64_t stride = (uint64_t)gridDim.x * NT;
    const unsigned dr = (unsigned)(stride / nv), dv = (unsigned)(stride % nv);
    const uint64_t t = (uint64_t)blockIdx.x * NT + threadIdx.x;
    uint64_t r = t / nv;
    unsigned v = (unsigned)(t % nv);
    while (r < (uint64_t)B) {
        const int c = 8 * (int)v, n = D - c;
        const int64_t i = (int64_t)r * D + c;
        float a[8];
        unpack8n<XB>(raw8n<XB>(x, i, c, D, TAIL), c, D, TAIL, a);
        if (d.thr) drop8(d, v, (unsigned)r, a);
        put8<TAIL, YB>(y, i, n, a);
        r += dr;
        v += dv;
        if (v >= nv) {
            v -= nv;
            ++r;
        }
    }
}

hipError_t launch_dropout(int B, int D, bool xbf, bool ybf, const void *x, const DropArgs &dr, void *y,
                          hipStream_t st) {
    const int64_t want = ((int64_t)B * (((int64_t)D + 7) / 8) + NT - 1) / NT;
    const dim3 grid((unsigned)(want < 65536 ? want : 65536));
#define GO(X, Y) \
    if (D & 7) hipLaunchKernelGGL((k_dropout<X, Y, true>), grid, dim3(NT), 0, st, B, D, x, dr, y); \
    else hipLaunchKernelGGL((k_dropout<X, Y, false>), grid, dim3(NT), 0, st, B, D, x, dr, y)
    if (xbf && ybf) {
        GO(true, true);
    } else if (xbf) {
        GO(true, false);
    } else if (ybf) {
        GO(false, true);
    } else {
        GO(false, false);
    }
#undef GO
    return hipGetLastError();
}

// ------------------------------------------------------ layer norm forward
// mean and variance of the row in registers, the variance from the deviations
// (no cancellation of squares), then y = drop((x - mean) rstd gamma + beta): one
// reading, one writing.  NV vectors a thread, TPR threads a row: D <= 8 NV TPR.
// What hides the memory's latency is the bytes in flight: the next row's vectors
// are loaded while this one is worked on, and a lane has two or three vectors of
// a row (fewer: too little in flight; four: too few waves a SIMD).
// Measured on both sides of the widths where the form changes, 2^26 bf16
// elements (their copy takes 52 us):
//   64 (2^25 elements): 8 lanes 32, 16 lanes 43
//   128 (2^25): 2 vectors on 8 lanes 30.5, 1 on 16 lanes 32
//   100 (2^25): 2 on 8 lanes 38, 1 on 16 42; of 65536 rows 11.7 and 10.1
//   256: 2 on 16 lanes 51, 1 on 32 61
//   512: 2 on 32 lanes 51, 1 on 64 59
//   768: 3 on 32 52.7, 2 on 64 53.5
//   1024: 2 on 64 50, 3 on 64 52       1536: 3 on 64 51, 4 on 64 54
//   2048: 2 on 128 52, 4 on 64 54      4096: 2 on 256 52, 4 on 256 63
//   8192: 2 on 512 55, read three times (below) 81
// 65536 x 768 bf16 with dropout: 40.5 us, 5.0 TB/s; one row of 1024: 3.1 us, the
// launch.
template <bool XB, bool YB, bool TAIL, int NV, int TPR>
__global__ __launch_bounds__(TPR > NT ? TPR : NT) void k_norm_fwd(NormArgs a) {
    constexpr int NTH = TPR > NT ? TPR : NT, RW = NTH / TPR;
    __shared__ float s[2][NTH / 64];
    int turn = 0;
    const int li = threadIdx.x % TPR, tail = tail_of<TAIL, TPR>(a.D);
    float ga[NV][8], be[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        load_w8(a.gamma, a.wbf, 8 * (li + k * TPR), a.D, 1.f, ga[k]);
        load_w8(a.beta, a.wbf, 8 * (li + k * TPR), a.D, 0.f, be[k]);
    }
    // the next row's vectors are loaded while this one is worked on
    auto fetch = [&](int64_t r, Raw8<XB> (&t)[NV]) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = 8 * (li + k * TPR);
            t[k] = raw8n<XB>(a.x, r * a.ldx + c, c, r < a.B ? a.D : 0, TAIL && k == tail);
        }
    };
    const int64_t step = (int64_t)gridDim.x * RW;
    Raw8<XB> next[NV];
    fetch((int64_t)blockIdx.x * RW + threadIdx.x / TPR, next);
    for (int64_t rb = (int64_t)blockIdx.x * RW; rb < a.B; rb += step) {
        const int64_t r = rb + threadIdx.x / TPR;
        const bool live = r < a.B;                      // all lanes stay for the row sums
        float x[NV][8], sum = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) unpack8n<XB>(next[k], 8 * (li + k * TPR), a.D, TAIL && k == tail, x[k]);
        fetch(r + step, next);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            sum += ((x[k][0] + x[k][1]) + (x[k][2] + x[k][3])) + ((x[k][4] + x[k][5]) + (x[k][6] + x[k][7]));
        const float mean = row_sum<TPR, NTH>(sum, s, turn) / (float)a.D;
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int n = a.D - 8 * (li + k * TPR);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[k][j] = j < n ? x[k][j] - mean : 0.f;
                sum = __builtin_fmaf(x[k][j], x[k][j], sum);
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<TPR, NTH>(sum, s, turn) / (float)a.D + a.eps);
        if (live) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int v = li + k * TPR, c = 8 * v;
                if (c >= a.D) continue;
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = __builtin_fmaf(x[k][j] * rstd, ga[k][j], be[k][j]);
                if (a.drop.thr) drop8(a.drop, (unsigned)v, (unsigned)r, y);
                put8<TAIL, YB>(a.y, r * a.D + c, a.D - c, y);
            }
            if (a.mean && li == 0) {
                a.mean[r] = mean;
                a.rstd[r] = rstd;
            }
        }
    }
}

// Any D: a workgroup a row, read three times (from L2 after the first: 8192 x
// 8192 bf16 81 us, floor 52).
template <bool XB, bool YB>
__global__ __launch_bounds__(NT) void k_norm_fwd_wide(NormArgs a) {
    __shared__ float s[2][NT / 64];
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.B; r += gridDim.x) {
        const int64_t o = r * a.ldx;
        float x[8], w[8], sum = 0.f;
        for (int64_t c = 8 * (int64_t)threadIdx.x; c < a.D; c += 8 * NT) {
            load8n<XB>(a.x, o + c, (int)c, a.D, 0.f, x);
            sum += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
        }
        const float mean = row_sum<NT, NT>(sum, s, turn) / (float)a.D;
        sum = 0.f;
        for (int64_t c = 8 * (int64_t)threadIdx.x; c < a.D; c += 8 * NT) {
            load8n<XB>(a.x, o + c, (int)c, a.D, mean, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(x[j] - mean, x[j] - mean, sum);
        }
        const float rstd = 1.0f / sqrtf(row_sum<NT, NT>(sum, s, turn) / (float)a.D + a.eps);
        for (int64_t c = 8 * (int64_t)threadIdx.x; c < a.D; c += 8 * NT) {
            const int n = a.D - (int)c;
            load8n<XB>(a.x, o + c, (int)c, a.D, mean, x);
            load_w8(a.gamma, a.wbf, (int)c, a.D, 1.f, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = (x[j] - mean) * rstd * w[j];
            load_w8(a.beta, a.wbf, (int)c, a.D, 0.f, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] += w[j];
            if (a.drop.thr) drop8(a.drop, (unsigned)(c >> 3), (unsigned)r, x);
            store8n<YB>(a.y, r * a.D + c, n, x);
        }
        if (a.mean && threadIdx.x == 0) {
            a.mean[r] = mean;
            a.rstd[r] = rstd;
        }
    }
}

template <bool XB, bool YB, bool TAIL>
static hipError_t norm_fwd(const NormArgs &a, hipStream_t st) {
    auto grid = [&](int rows_per_wg, int64_t most) {
        const int64_t want = ((int64_t)a.B + rows_per_wg - 1) / rows_per_wg;
        return dim3((unsigned)(want < most ? want : most));
    };
#define GO(NV, TPR) \
    hipLaunchKernelGGL((k_norm_fwd<XB, YB, TAIL, NV, TPR>), grid(TPR > NT ? 1 : NT / TPR, 2048), dim3(TPR > NT ? TPR : NT), 0, st, a)
    constexpr int kNarrow = TAIL ? 64 : 128;      // rows with ends inside vectors gain from eight lanes to 64 only
    if (a.D <= 64) GO(1, 8);
    else if (a.D <= kNarrow) GO(TAIL ? 1 : 2, 8);
    else if (a.D <= 128) GO(1, 16);
    else if (a.D <= 256) GO(2, 16);
    else if (a.D <= 512) GO(2, 32);
    else if (a.D <= 768) GO(3, 32);
    else if (a.D <= 1024) GO(2, 64);
    else if (a.D <= 1536) GO(3, 64);
    else if (a.D <= 2048) GO(2, 128);
    else if (a.D <= 4096) GO(2, 256);
    else if (a.D <= 8192) GO(2, 512);
    else hipLaunchKernelGGL((k_norm_fwd_wide<XB, YB>), grid(1, 4096), dim3(NT), 0, st, a);
#undef GO
    return hipGetLastError();
}

hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t st) {
    const bool t = a.D & 7;
    if (a.xbf && a.ybf) return t ? norm_fwd<true, true, true>(a, st) : norm_fwd<true, true, false>(a, st);
    if (a.xbf) return t ? norm_fwd<true, false, true>(a, st) : norm_fwd<true, false, false>(a, st);
    if (a.ybf) return t ? norm_fwd<false, true, true>(a, st) : norm_fwd<false, true, false>(a, st);
    return t ? norm_fwd<false, false, true>(a, st) : norm_fwd<false, false, false>(a, st);
}

// ----------------------------------------------------- layer norm backward
// Row by row: dx, and the thread's columns of a * h and a summed over the
// workgroup's rows in registers.  At the end the workgroup's row groups lay
// theirs side by side in LDS, a thread adds a column's up in their order, and
// one partial sum a workgroup is left for k_norm_wsum.
//
//   a = drop(dy), g = a gamma, h = (x - mean) rstd
//   dx = rstd (g - mean(g) - h mean(g h)),  dgamma = sum_rows a h,  dbeta = sum_rows a
//
// Bytes: x, dy and dx once, and the partials (2 D fp32 each) written and read.
// At most 512 of them, so that two workgroups a CU run: little for many rows (4 MB
// beside 481 for 40001 x 1001 fp32: 99 us and 5 for the partials, 4.8 TB/s), much
// for few wide ones (17 MB beside 34 for 1024 x 4096 bf16, dy fp32: a call of 17 us,
// its own bytes 6.5; 20 beside 201 for 6710 x 5001 bf16: 80 us, 39, where also 398
// of a row's 1024 threads have nothing to do).  512 x 768, its columns in the same
// launch (norm_columns): 6.1.
// Threads a row, both sides of each change, 2^25 elements bf16 / fp32 dy (copy
// 51.7 us): 64, bf16 dy (copy 39.5): 8 lanes 47, 16 lanes 66; 128: 16 lanes 1
// or 2 vectors 55; 256: 16 lanes 56, 64 lanes 79; 512: 64 lanes 1 or 2 vectors
// 55; 1024: 64 lanes 56, 256 threads 88; 2048: 256 threads 57, 512 81; 4096:
// 512 threads 60, 2 vectors 86; 8192: 1024 threads 67, read twice (below) 111.
constexpr int NB = 512;       // threads

// Few rows: the weight gradient of 32 columns over all rows by one workgroup of
// its own, from x, dy and the rows' statistics, so that no second launch adds
// partials up.  A thread a vector and every (NTH / 4)-th row; at the end the
// threads' sums are laid out in LDS (16 NTH floats) and added in a fixed order.
// us a call, this way and with a second launch, fp32 dy: 512 x 768 bf16 8.7 and
// 11.8, 16 rows 9.3 and 12; 512 x 4096 fp32 8.9 and 14.2; 1024 x 100 14.1 and
// 11.2, 2048 x 768 17 and 11.5.
template <bool XB, bool YB, bool TAIL, int NTH>
__device__ __forceinline__ void norm_columns(const NormArgs &a, int block, float *room) {
    constexpr int G = NTH / 4, U = 4;
    const int tid = threadIdx.x, v = 4 * block + (tid & 3), c = 8 * v;
    const bool tail = TAIL && a.D / 32 == block;      // only these columns hold the rows' end
    float dg[8], db[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[j] = db[j] = 0.f;
    for (int64_t r0 = tid >> 2; r0 < a.B; r0 += U * G) {
        Raw8<XB> hr[U];
        Raw8<YB> gr[U];
        float mean[U], rstd[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t r = r0 + i * G;
            const bool live = r < a.B;
            mean[i] = live ? a.mean[r] : 0.f;
            rstd[i] = live ? a.rstd[r] : 0.f;
            hr[i] = raw8n<XB>(a.x, r * a.ldx + c, c, live ? a.D : 0, tail);
            gr[i] = raw8n<YB>(a.dy, r * a.D + c, c, live ? a.D : 0, tail);
        }
#pragma unroll 1
        for (int i = 0; i < U; ++i) {
            const int64_t r = r0 + i * G;
            if (r >= a.B) break;
            float h[8], g[8];
            unpack8n<XB>(i == 0 ? hr[0] : i == 1 ? hr[1] : i == 2 ? hr[2] : hr[3], c, a.D, tail, h);
            unpack8n<YB>(i == 0 ? gr[0] : i == 1 ? gr[1] : i == 2 ? gr[2] : gr[3], c, a.D, tail, g);
            const float m = i == 0 ? mean[0] : i == 1 ? mean[1] : i == 2 ? mean[2] : mean[3];
            const float s = i == 0 ? rstd[0] : i == 1 ? rstd[1] : i == 2 ? rstd[2] : rstd[3];
            if (a.drop.thr && c < a.D) drop8(a.drop, (unsigned)v, (unsigned)r, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dg[j] = __builtin_fmaf(g[j], (h[j] - m) * s, dg[j]);
                db[j] += g[j];
            }
        }
    }
    // sum e of thread t at e NTH + (t + 4 e) mod NTH: 64 sums' threads read 64 banks
    auto at = [](int e, int t) { return e * NTH + ((t + 4 * e) & (NTH - 1)); };
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        room[at(j, tid)] = dg[j];
        room[at(8 + j, tid)] = db[j];
    }
    __syncthreads();
    // a wave a share of the row groups, a lane one of the 64 sums: dgamma, then dbeta
    constexpr int W = NTH / 64, PER = G / W;
    const int o = tid & 63, w = tid >> 6, e = (o >> 5) * 8 + (o & 7);
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) t += room[at(e, 4 * (w * PER + i) + (o >> 3 & 3))];
    __syncthreads();
    room[tid] = t;
    __syncthreads();
    if (tid < 64) {
        t = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) t += room[64 * i + tid];
        const int col = 32 * block + (tid & 31);
        float *out = tid < 32 ? a.dgamma : a.dbeta;
        if (out && col < a.D) out[col] = a.accumulate ? out[col] + t : t;
    }
}

// FEW: the first a.columns workgroups sum the weight gradient (norm_columns).
template <bool XB, bool YB, bool TAIL, bool FEW, int NV, int TPR>
__global__ __launch_bounds__(TPR > NB ? TPR : NB, TPR >= 512 ? 2 : 4) void k_norm_bwd(NormArgs a) {
    constexpr int NTH = TPR > NB ? TPR : NB, RW = NTH / TPR;
    __shared__ float s[2][NTH / 64], q[2][NTH / 64];
    __shared__ __attribute__((aligned(16))) float acc[2][RW][8 * NV * TPR];
    if (FEW && (int)blockIdx.x < a.columns) {
        norm_columns<XB, YB, TAIL, NTH>(a, blockIdx.x, acc[0][0]);
        return;
    }
    const unsigned block = blockIdx.x - (FEW ? a.columns : 0), blocks = gridDim.x - (FEW ? a.columns : 0);
    int turn = 0;
    const int li = threadIdx.x % TPR, tail = tail_of<TAIL, TPR>(a.D);
    const bool wgrad = !FEW && (a.dgamma || a.dbeta);
    float ga[NV][8], dg[NV][8], db[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        load_w8(a.gamma, a.wbf, 8 * (li + k * TPR), a.D, 1.f, ga[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dg[k][j] = db[k][j] = 0.f;
    }
    for (int64_t rb = (int64_t)block * RW; rb < a.B; rb += (int64_t)blocks * RW) {
        const int64_t r = rb + threadIdx.x / TPR;
        const bool live = r < a.B;
        const float mean = live ? a.mean[r] : 0.f, rstd = live ? a.rstd[r] : 0.f;
        Raw8<XB> hr[NV];
        Raw8<YB> gr[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {      // past the row's end g = 0 adds nothing, with an h that is
            const int c = 8 * (li + k * TPR);      // finite: the last element's, or 0 (0 - mean may overflow)
            hr[k] = raw8n<XB, true>(a.x, r * a.ldx + c, c, live ? a.D : 0, TAIL && k == tail);
            gr[k] = raw8n<YB>(a.dy, r * a.D + c, c, live ? a.D : 0, TAIL && k == tail);
        }
        float h[NV][8], g[NV][8], sg = 0.f, sgh = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = li + k * TPR;
            const float m = 8 * v < a.D ? mean : 0.f;
            unpack8n<XB, true>(hr[k], 8 * v, a.D, TAIL && k == tail, h[k]);
            unpack8n<YB>(gr[k], 8 * v, a.D, TAIL && k == tail, g[k]);
            if (a.drop.thr && 8 * v < a.D) drop8(a.drop, (unsigned)v, (unsigned)r, g[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[k][j] = (h[k][j] - m) * rstd;
                dg[k][j] = __builtin_fmaf(g[k][j], h[k][j], dg[k][j]);
                db[k][j] += g[k][j];
                g[k][j] *= ga[k][j];
                sg += g[k][j];
                sgh = __builtin_fmaf(g[k][j], h[k][j], sgh);
            }
        }
        row_sum2<TPR, NTH>(sg, sgh, s, q, turn);
        sg /= (float)a.D;
        sgh /= (float)a.D;
        if (live) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = 8 * (li + k * TPR);
                if (c >= a.D) continue;
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = rstd * (g[k][j] - sg - h[k][j] * sgh);
                put8<TAIL, XB>(a.dx, r * a.lddx + c, a.D - c, o);
            }
        }
    }
    if (!wgrad) return;
    const int w = threadIdx.x / TPR;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            *(f32x4 *)(acc[0][w] + 8 * (li + k * TPR) + e) = (f32x4){dg[k][e], dg[k][e + 1], dg[k][e + 2], dg[k][e + 3]};
            *(f32x4 *)(acc[1][w] + 8 * (li + k * TPR) + e) = (f32x4){db[k][e], db[k][e + 1], db[k][e + 2], db[k][e + 3]};
        }
    __syncthreads();
    float *part = a.part + (int64_t)block * 2 * a.D;
    for (int c = threadIdx.x; c < a.D; c += NTH) {
        float x = acc[0][0][c], y = acc[1][0][c];
#pragma unroll
        for (int i = 1; i < RW; ++i) {
            x += acc[0][i][c];
            y += acc[1][i][c];
        }
        part[c] = x;
        part[a.D + c] = y;
    }
}

// Any D, the row sums and dx: a workgroup a row, read twice.
template <bool XB, bool YB>
__global__ __launch_bounds__(NT) void k_norm_bwd_wide(NormArgs a) {
    __shared__ float s[2][NT / 64], q[2][NT / 64];
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.B; r += gridDim.x) {
        const float mean = a.mean[r], rstd = a.rstd[r];
        float sg = 0.f, sgh = 0.f, h[8], g[8], w[8];
        for (int pass = 0; pass < 2; ++pass) {
            for (int64_t c = 8 * (int64_t)threadIdx.x; c < a.D; c += 8 * NT) {
                const int n = a.D - (int)c;
                load8n<XB>(a.x, r * a.ldx + c, (int)c, a.D, mean, h);
                load8n<YB>(a.dy, r * a.D + c, (int)c, a.D, 0.f, g);
                load_w8(a.gamma, a.wbf, (int)c, a.D, 1.f, w);
                if (a.drop.thr) drop8(a.drop, (unsigned)(c >> 3), (unsigned)r, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    h[j] = (h[j] - mean) * rstd;
                    g[j] *= w[j];
                    if (pass == 0) {
                        sg += g[j];
                        sgh = __builtin_fmaf(g[j], h[j], sgh);
                    } else {
                        g[j] = rstd * (g[j] - sg - h[j] * sgh);
                    }
                }
                if (pass == 1) store8n<XB>(a.dx, r * a.lddx + c, n, g);
            }
            if (pass == 0) {
                row_sum2<NT, NT>(sg, sgh, s, q, turn);
                sg /= (float)a.D;
                sgh /= (float)a.D;
            }
        }
    }
}

// Any D, the weight gradient's partial sums: a thread eight columns, the rows
// y, y + parts, ...
template <bool XB, bool YB>
__global__ __launch_bounds__(64) void k_norm_wgrad(NormArgs a) {
    const int64_t c = 8 * ((int64_t)blockIdx.x * 64 + threadIdx.x);
    if (c >= a.D) return;
    const int n = a.D - (int)c;
    float dg[8], db[8], h[8], g[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[j] = db[j] = 0.f;
    for (int64_t r = blockIdx.y; r < a.B; r += gridDim.y) {
        const float mean = a.mean[r], rstd = a.rstd[r];
        load8n<XB>(a.x, r * a.ldx + c, (int)c, a.D, mean, h);
        load8n<YB>(a.dy, r * a.D + c, (int)c, a.D, 0.f, g);
        if (a.drop.thr) drop8(a.drop, (unsigned)(c >> 3), (unsigned)r, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dg[j] = __builtin_fmaf(g[j], (h[j] - mean) * rstd, dg[j]);
            db[j] += g[j];
        }
    }
    float *part = a.part + (int64_t)blockIdx.y * 2 * a.D;
    store8n<false>(part, c, n, dg);
    store8n<false>(part, a.D + c, n, db);
}

// The partial sums of a column (of 2 D: dgamma, then dbeta) added up: 16 waves
// of 64 columns, a sixteenth of the partials each, joined in LDS.  A fixed
// order: equal inputs give equal bits.
__global__ __launch_bounds__(1024) void k_norm_wsum(NormArgs a, int parts) {
    __shared__ float s[16][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t cols = 2 * (int64_t)a.D;
    for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < cols; c0 += (int64_t)gridDim.x * 64) {
        const int64_t c = c0 + lane;
        float t = 0.f;
        if (c < cols) {
            constexpr int U = 8;
            for (int p0 = w; p0 < parts; p0 += 16 * U) {
                float v[U];
#pragma unroll
                for (int i = 0; i < U; ++i) v[i] = p0 + 16 * i < parts ? a.part[(int64_t)(p0 + 16 * i) * cols + c] : 0.f;
#pragma unroll
                for (int i = 0; i < U; ++i) t += v[i];
            }
        }
        s[w][lane] = t;
        __syncthreads();
        if (w == 0 && c < cols) {
            t = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) t += s[i][lane];
            float *o = c < a.D ? a.dgamma : a.dbeta;
            if (o) {
                o += c < a.D ? c : c - a.D;
                *o = a.accumulate ? *o + t : t;
            }
        }
        __syncthreads();
    }
}

namespace {
constexpr int kPartMost = 512;
constexpr int kFewRows = 512;
// rows of a workgroup of k_norm_bwd; 0: the wide kernels
int norm_bwd_rows(int D) {
    return D <= 64 ? NB / 8 : D <= 256 ? NB / 16 : D <= 1024 ? NB / 64 : D <= 2048 ? NB / 256 : D <= 8192 ? 1 : 0;
}
}  // namespace

int norm_parts(int B, int D) {
    const int rows = norm_bwd_rows(D);
    const int64_t want = rows ? ((int64_t)B + rows - 1) / rows : ((int64_t)B + 15) / 16;
    return (int)(want < kPartMost ? want : kPartMost);
}

template <bool XB, bool YB, bool TAIL>
static hipError_t norm_bwd(const NormArgs &args, hipStream_t st) {
    NormArgs a = args;
    const int parts = norm_parts(a.B, a.D);
    const bool w = a.dgamma || a.dbeta;
    a.columns = w && a.B <= kFewRows && a.D <= 8192 ? (a.D + 31) / 32 : 0;
#define GO(NV, TPR) \
    if (a.columns) hipLaunchKernelGGL((k_norm_bwd<XB, YB, TAIL, true, NV, TPR>), dim3(parts + a.columns), dim3(TPR > NB ? TPR : NB), 0, st, a); \
    else hipLaunchKernelGGL((k_norm_bwd<XB, YB, TAIL, false, NV, TPR>), dim3(parts), dim3(TPR > NB ? TPR : NB), 0, st, a)
    if (a.D <= 64) {
        GO(1, 8);
    } else if (a.D <= 128) {
        GO(1, 16);
    } else if (a.D <= 256) {
        GO(2, 16);
    } else if (a.D <= 512) {
        GO(1, 64);
    } else if (a.D <= 1024) {
        GO(2, 64);
    } else if (a.D <= 2048) {
        GO(1, 256);
    } else if (a.D <= 4096) {
        GO(1, 512);
    } else if (a.D <= 8192) {
        GO(1, 1024);
    } else {
        hipLaunchKernelGGL((k_norm_bwd_wide<XB, YB>), dim3((unsigned)(a.B < 4096 ? a.B : 4096)), dim3(NT), 0, st, a);
        if (w) hipLaunchKernelGGL((k_norm_wgrad<XB, YB>), dim3((unsigned)(((int64_t)a.D + 511) / 512), parts), dim3(64), 0, st, a);
    }
#undef GO
    const int64_t cols = (2 * (int64_t)a.D + 63) / 64;
    if (w && !a.columns) hipLaunchKernelGGL(k_norm_wsum, dim3((unsigned)(cols < 65536 ? cols : 65536)), dim3(1024), 0, st, a, parts);
    return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t st) {
    const bool t = a.D & 7;
    if (a.xbf && a.ybf) return t ? norm_bwd<true, true, true>(a, st) : norm_bwd<true, true, false>(a, st);
    if (a.xbf) return t ? norm_bwd<true, false, true>(a, st) : norm_bwd<true, false, false>(a, st);
    if (a.ybf) return t ? norm_bwd<false, true, true>(a, st) : norm_bwd<false, true, false>(a, st);
    return t ? norm_bwd<false, false, true>(a, st) : norm_bwd<false, false, false>(a, st);
}

}  // namespace haste
