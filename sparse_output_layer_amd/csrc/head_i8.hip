// head_i8.hip -- rows in 8-bit integers with one scale each, and the head's
// logits from them:
//   q = x / s to nearest even, s = max|x| (1/127)
//   Z[b][h] = (sum_d Xq[b][d] Wq[h][d]) xs[b] ws[h], the sum exact in 32 bits
// (at most 127 * 127 * 131072 < 2^31), one rounding of the sum to fp32, two of
// the products and one to the result's type.
#include "elem.h"

#include <type_traits>

namespace haste {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(16))) int i32x16;

namespace {
constexpr int NT = 256;
// |v|'s bits: ordered as the numbers are, infinity and then NaN above them
__device__ __forceinline__ unsigned abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
}  // namespace

// ---------------------------------------------------------------- the rows
// s = max|x| * (1/127), q = x / s to nearest even; zeros in a row whose scale
// is 0 or no number (so that the logits of the latter are NaN).  The product
// with the rounded reciprocal is what a tensor divided by a constant gives on
// the device, so that rows quantised there and here agree in every bit: max
// and x of a few bits often make x / s a tie but for the last bit of s.
constexpr float kScale = 1.0f / 127.0f;
struct Quant {
    float s, r;      // scale and its reciprocal
    int way;         // 0: zeros, 1: by the reciprocal, 2: by division
};
__device__ __forceinline__ Quant quant_by(unsigned max_bits) {
    Quant q;
    q.s = __uint_as_float(max_bits) * kScale;
    q.r = 1.0f / q.s;
    q.way = !(q.s > 0.f && q.s < __builtin_inff()) ? 0 : q.s > 0x1p-60f && q.s < 0x1p60f ? 1 : 2;
    return q;
}
// Eight elements.  The quotient, correctly rounded, is q0 = x r, q0 + (x - q0 s) r
// with r the rounded reciprocal (Markstein, "Computation of elementary functions
// on the IBM RISC System/6000 processor", 1990; the residual is exact wherever
// |q0| is near 1/2 or more, and scales are kept away from both ends of the
// range).  1.5 * 2^23 added leaves the integer, rounded to nearest even, in the
// sum's low bits.  8192 x 1024 bf16: 15.3 us with a division each, 13.6 this way.
__device__ __forceinline__ u32x2 quant8(const float *v, const Quant &q) {
    u32x2 r = {0u, 0u};
    if (q.way == 1) {
        unsigned w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float q0 = v[j] * q.r;
            w[j] = __float_as_uint(__builtin_fmaf(__builtin_fmaf(-q0, q.s, v[j]), q.r, q0) + 0x1.8p23f);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            r[h] = __builtin_amdgcn_perm(w[4 * h + 1], w[4 * h], 0x0c0c0400u) |
                   __builtin_amdgcn_perm(w[4 * h + 3], w[4 * h + 2], 0x04000c0cu);
    } else if (q.way == 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            r[j >> 2] |= ((unsigned)(int)fminf(fmaxf(rintf(v[j] / q.s), -127.f), 127.f) & 255u) << (8 * (j & 3));
    }
    return r;
}

// A wave a row, the row in registers: one reading.  NV vectors of eight
// elements a lane, D <= 512 NV.  2^25 bf16 elements in rows of 2048: 23 us, read
// twice by a workgroup a row (below) 27.
template <bool BF, int NV>
__global__ __launch_bounds__(NT) void k_quantize_wave(int rows, int D, int64_t ldx, const void *x, int8_t *q,
                                                      float *scale) {
    const int lane = threadIdx.x & 63, D64 = (D + 63) / 64 * 64;
    for (int64_t r = (int64_t)blockIdx.x * (NT / 64) + (threadIdx.x >> 6); r < rows; r += (int64_t)gridDim.x * (NT / 64)) {
        float v[NV][8];
        unsigned m = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = 8 * (64 * k + lane);
            load8n<BF>(x, r * ldx + c, c, D, 0.f, v[k]);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[k][j]));
        const Quant by = quant_by(wave_max_dpp(m));
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = 8 * (64 * k + lane);
            if (c < D64) *(u32x2 *)(q + r * D64 + c) = quant8(v[k], by);
        }
        if (lane == 0) scale[r] = by.s;
    }
}

// A workgroup a row, read twice (wider rows).
template <bool BF>
__global__ __launch_bounds__(NT) void k_quantize_wide(int rows, int D, int64_t ldx, const void *x, int8_t *q,
                                                      float *scale) {
    __shared__ unsigned part[NT / 64];
    const int D64 = (D + 63) / 64 * 64;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        unsigned m = 0;
        float v[8];
        for (int c = 8 * threadIdx.x; c < D; c += 8 * NT) {
            load8n<BF>(x, r * ldx + c, c, D, 0.f, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
        }
        m = wave_max_dpp(m);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
        __syncthreads();
        m = part[0];
        for (int i = 1; i < NT / 64; ++i) m = max(m, part[i]);
        const Quant by = quant_by(m);
        for (int c = 8 * threadIdx.x; c < D64; c += 8 * NT) {
            load8n<BF>(x, r * ldx + c, c, D, 0.f, v);
            *(u32x2 *)(q + r * D64 + c) = quant8(v, by);
        }
        if (threadIdx.x == 0) scale[r] = by.s;
    }
}

template <bool BF>
static hipError_t launch_quantize(int rows, int D, int64_t ldx, const void *x, int8_t *q, float *scale,
                                  hipStream_t st) {
    const int wg = (int)(((int64_t)rows + 3) / 4);
    const dim3 few((unsigned)(wg < 4096 ? wg : 4096)), wide((unsigned)(rows < 4096 ? rows : 4096));
#define GO(NV) hipLaunchKernelGGL((k_quantize_wave<BF, NV>), few, dim3(NT), 0, st, rows, D, ldx, x, q, scale)
    if (D <= 512) GO(1);
    else if (D <= 1024) GO(2);
    else if (D <= 2048) GO(4);
    else hipLaunchKernelGGL(k_quantize_wide<BF>, wide, dim3(NT), 0, st, rows, D, ldx, x, q, scale);
#undef GO
    return hipGetLastError();
}

hipError_t launch_quantize_rows(int rows, int D, bool bf, int64_t ldx, const void *x, int8_t *q, float *scale,
                                hipStream_t st) {
    return bf ? launch_quantize<true>(rows, D, ldx, x, q, scale, st) : launch_quantize<false>(rows, D, ldx, x, q, scale, st);
}

// ------------------------------------------------------------ the product
// Labels are the MFMA's rows and batch rows its columns, so that a lane ends
// with runs of four consecutive labels of one batch row.

struct I8Args {
    const int8_t *X, *W;       // M and N rows of K64 bytes
    const float *xs, *ws;
    void *Z;                   // M x N
    int M, N, K64;
    bool stream;               // results past every cache: stored without keeping their lines
};

namespace {

// Four results at element o: rows of an odd length leave any alignment that
// the type has.
template <bool ZB>
__device__ __forceinline__ void put4(void *Z, int64_t o, const float *v) {
    if (ZB) {
        typedef __attribute__((ext_vector_type(2), aligned(2))) unsigned u2;
        *(u2 *)((unsigned short *)Z + o) = (u2){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    } else {
        *(f32x4u *)((float *)Z + o) = (f32x4u){v[0], v[1], v[2], v[3]};
    }
}

// Up to four consecutive labels n.. of batch row m, scaled and stored.
template <bool ZB>
__device__ __forceinline__ void store_z4(const I8Args &a, int m, int n, const int *acc) {
    if (m >= a.M || n >= a.N) return;
    const float x = a.xs[m];
    float v[4];
    const int left = a.N - n;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)acc[e] * x * a.ws[e < left ? n + e : n];
    const int64_t o = (int64_t)m * a.N + n;
    if (left >= 4) {
        put4<ZB>(a.Z, o, v);
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < left) store1<ZB>(a.Z, o + e, v[e]);
    }
}

// s_waitcnt with only the vector-memory count constrained
template <int N>
__device__ __forceinline__ void wait_copies() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// The wave's own LDS writes before this are seen by its lanes' reads after it
__device__ __forceinline__ void wave_lds_fence() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Order of the N products of a half step and what goes between them (one wave
// a SIMD has nothing else to hide it behind): after each an LDS read, and with
// COPIES a global-to-LDS copy and its address arithmetic.  Nothing is
// scheduled across the end.
template <int N, int COPIES>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);      // MFMA
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);      // LDS read
        if (COPIES) {
            __builtin_amdgcn_sched_group_barrier(0x006, 6, 0);  // VALU, SALU
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // VMEM read
        }
    }
    __builtin_amdgcn_sched_barrier(0);
}

// the same value, not known to be: what is formed from it stays where it is written
__device__ __forceinline__ int opaque(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// 32x32 output, K = 32 int8 per instruction.  A / B: lane l holds row / col
// (l % 32) and K slots 16*(l/32) .. +15.  Output as mfma32x32.
__device__ __forceinline__ i32x16 mfma32x32_i8(i32x4 a, i32x4 b, i32x16 c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}
// 16 bytes a lane from global memory to 1 KB of LDS at S (wave-uniform)
__device__ __forceinline__ void copy_kb(const int8_t *src, int8_t *S) {
    __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void *)S, 16, 0, 0);
}

// 4 bytes a lane to 256 bytes of LDS, for both operands' scales
__device__ __forceinline__ void copy_scales(const float *w, const float *x, float *sw, float *sx) {
    __builtin_amdgcn_global_load_lds(w, (__attribute__((address_space(3))) void *)sw, 4, 0, 0);
    __builtin_amdgcn_global_load_lds(x, (__attribute__((address_space(3))) void *)sx, 4, 0, 0);
}

constexpr int KB = 64;     // bytes of a row per step

// s_waitcnt with only the LDS count constrained, to zero: written as the
// builtin, so that the compiler knows of it and does not wait for the reads
// that follow when it first uses these
__device__ __forceinline__ void wait_reads() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4)); }

// 16-byte segment s of a tile's row r sits at slot s ^ ((r >> 2) & 3) of its
// 64 bytes: 16 consecutive rows read at one s cover 16 different slots of the
// LDS's 256 bytes.
__device__ __forceinline__ int seg_slot(int r, int s) { return s ^ ((r >> 2) & 3); }

}  // namespace

namespace {
__device__ __forceinline__ i32x4 few_step(i32x4 w, i32x4 x, i32x4 acc) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, acc, 0, 0, 0);
}
}  // namespace

// Up to 16 batch rows (the product's columns): the weights' bytes count.  A wave
// takes 16 labels and streams their rows straight into MFMA operands, 16 loads of
// 64 bytes a row in flight (of 4096 features 29.8 us, with 8 of them 33.2); the
// batch rows come from L2 (a lane past the batch reads the last one).  1 x 1024 ->
// 32768: 7.5 us with its launch, 34 MB, 4.5 TB/s.  Against the 64 x 64 tiles
// below, us: 1 row 7.5 and 8.9, 8 rows 8.4 and 8.9 (256 -> 100000: 8.8 and 11.2);
// 16 rows 9.6 and 9.0, of 256 -> 100000 10.2 and 11.7, of 512 -> 32768 6.2 and
// 6.8, of 2048 -> 16384 9.9 and 8.9.
template <bool ZB>
__global__ __launch_bounds__(256) void k_i8_few(I8Args a) {
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int64_t step = (int64_t)gridDim.x * 64;
    for (int64_t n = (int64_t)blockIdx.x * 64 + 16 * (threadIdx.x >> 6); n < a.N; n += step) {
        const int n0 = (int)n;
        const int8_t *pw = a.W + (int64_t)min(n0 + r, a.N - 1) * a.K64 + 16 * q;
        const int8_t *px = a.X + (int64_t)min(r, a.M - 1) * a.K64 + 16 * q;
        i32x4 acc = (i32x4){0, 0, 0, 0};
        int k = 0;
        auto steps = [&](auto u) {
            constexpr int U = decltype(u)::value;
            for (; k + U * KB <= a.K64; k += U * KB) {
                i32x4 fw[U], fx[U];
#pragma unroll
                for (int i = 0; i < U; ++i) fw[i] = *(const i32x4 *)(pw + k + i * KB);
#pragma unroll
                for (int i = 0; i < U; ++i) fx[i] = *(const i32x4 *)(px + k + i * KB);
#pragma unroll
                for (int i = 0; i < U; ++i) acc = few_step(fw[i], fx[i], acc);
            }
        };
        steps(std::integral_constant<int, 16>{});
        steps(std::integral_constant<int, 4>{});
        for (; k < a.K64; k += KB)
            acc = few_step(*(const i32x4 *)(pw + k), *(const i32x4 *)(px + k), acc);
        const int v[4] = {acc[0], acc[1], acc[2], acc[3]};
        store_z4<ZB>(a, r, n0 + 4 * q, v);
    }
}

// what a step past the end multiplies with
__device__ __attribute__((aligned(16))) int8_t kZeros[16];

// Tiles of 64 WL labels x 64 WB batch rows, four waves (2 x 2) of WL x WB
// MFMA tiles of 32 x 32, K in steps of 64 bytes through a ring of four LDS
// stages filled by direct global-to-LDS copies.  A workgroup walks over
// several tiles: the copies of the next tile's first steps are under way
// while this one's results are scaled and stored.
//
// What bounds it is power: 8192^3 runs at 2.1 POP/s (515 us) with the clock
// down to 1.83 GHz, all-zero operands take 417 us; so the form with the fewest
// LDS bytes an operation, 256 x 192 in registers, wins, though its results'
// stores (88 us of 8192 x 1024 -> 32768's 360, 537 MB) are hardly hidden: a tile
// is scaled and stored while nothing multiplies.  128 x
// 192 with two workgroups a CU hides more, but pays for it in LDS traffic:
// 8192 x 1024 -> 32768 376 us (zeros 280), 8192^3 623.
template <int WL, int WB, int PER_CU, bool ZB>
__global__ __launch_bounds__(256, PER_CU) void k_i8_tile(I8Args a) {
    constexpr int TL = 64 * WL, TB = 64 * WB, STAGE = (TL + TB) * KB, NS = 4;
    constexpr int LPS = WL + WB;      // copies per wave and step
    // results pass through LDS, RP batch rows of 16-byte slots at a time: as
    // many as the room beside the stages and scales holds
    constexpr int SLOTS = (ZB ? 4 : 8) * WL, PER = ZB ? 8 : 4;     // a row's slots, labels a slot
    constexpr int ROOM = (163840 / PER_CU - NS * STAGE - 2048) / 4 / (16 * SLOTS);
    constexpr int RP = ROOM >= 32 ? 32 : ROOM >= 16 ? 16 : ROOM >= 8 ? 8 : 4;
    static_assert(ROOM >= 4, "the workgroups' share of the LDS");
    __shared__ __attribute__((aligned(1024))) int8_t st0[STAGE];
    __shared__ __attribute__((aligned(1024))) int8_t st1[STAGE];
    __shared__ __attribute__((aligned(1024))) int8_t st2[STAGE];
    __shared__ __attribute__((aligned(1024))) int8_t st3[STAGE];
    __shared__ __attribute__((aligned(1024))) int8_t out[4 * RP * 16 * SLOTS];
    __shared__ __attribute__((aligned(16))) float sw[256], sx[256];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5;
    const int wl = (w >> 1) * 32 * WL, wb = (w & 1) * 32 * WB;
    // Workgroups go round-robin over the 8 XCDs: each XCD gets a run of
    // consecutive tiles, eight batch tiles wide, so that tiles running
    // together share rows of both operands in its L2.
    const int nl = (a.N + TL - 1) / TL, nb = (a.M + TB - 1) / TB, T = nl * nb;
    const int per = (T + 7) / 8, stride = (int)gridDim.x >> 3;
    const int tend = min(T, ((int)(blockIdx.x & 7) + 1) * per);
    int t = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if (t >= tend) return;
    const int nk = a.K64 / KB;

    struct Tile {
        const int8_t *pw, *px;   // its first rows
        int n0, m0;
        unsigned off[LPS];       // copy c of a wave: 16 rows of the stage (labels, then batch
                                 // rows), rows past the end reading the last one
    };
    auto place = [&](int i) {
        Tile x;
        const int band = i / (8 * nl), wide = min(8, nb - 8 * band), u = i - band * 8 * nl;
        x.n0 = (u / wide) * TL;
        x.m0 = (8 * band + u % wide) * TB;
        x.pw = a.W + (int64_t)x.n0 * a.K64;
        x.px = a.X + (int64_t)x.m0 * a.K64;
#pragma unroll
        for (int c = 0; c < LPS; ++c) {
            const int blk = w * LPS + c, row = 16 * blk + (lane >> 2);
            const int g = 16 * blk < TL ? min(row, a.N - 1 - x.n0) : min(row - TL, a.M - 1 - x.m0);
            x.off[c] = (unsigned)g * (unsigned)a.K64 + 16u * seg_slot(row, lane & 3);
        }
        return x;
    };
    // step kt of a tile into stage S; the labels of a step past the end are zeros
    auto issue = [&](const Tile &x, int kt, int8_t *S) {
        const bool past = kt >= nk;
        const unsigned k0 = past ? 0u : (unsigned)kt * KB;
#pragma unroll
        for (int c = 0; c < LPS; ++c) {
            const int blk = w * LPS + c;
            const bool zero = past && 16 * blk < TL;
            const int8_t *base = zero ? kZeros : 16 * blk < TL ? x.pw : x.px;
            copy_kb(base + (zero ? 0u : x.off[c] + k0), S + blk * 1024);
        }
    };
    i32x16 acc[WL][WB];
    i32x4 pa[WL], pb[WB], qa[WL], qb[WB];
    auto read = [&](const int8_t *S, int ks, i32x4 *av, i32x4 *bv) {
#pragma unroll
        for (int i = 0; i < WL; ++i) {
            const int row = wl + 32 * i + r;
            av[i] = *(const i32x4 *)(S + row * KB + 16 * seg_slot(row, 2 * ks + h));
        }
#pragma unroll
        for (int j = 0; j < WB; ++j) {
            const int row = TL + wb + 32 * j + r;
            bv[j] = *(const i32x4 *)(S + row * KB + 16 * seg_slot(row, 2 * ks + h));
        }
    };
    auto multiply = [&](const i32x4 *av, const i32x4 *bv) {
#pragma unroll
        for (int i = 0; i < WL; ++i)
#pragma unroll
            for (int j = 0; j < WB; ++j) acc[i][j] = mfma32x32_i8(av[i], bv[j], acc[i][j]);
    };
    // A step on stage S: the operands of its first half are in registers, the
    // second half's are read while the first multiplies.  Then this wave's
    // copies of the next step have landed (those of the two after it stay in
    // flight), and the barrier makes that everyone's and says that every wave
    // has read all of stage S, which the copies of four steps on (or of the
    // next tile's first steps) fill.
    auto first_half = [&](const int8_t *S) {
        wait_reads();
        read(S, 1, qa, qb);
        multiply(pa, pb);
        interleave<WL * WB, 0>();
        wait_reads();
        wait_copies<(NS - 2) * LPS>();
        lds_barrier();
    };
    auto second_half = [&](const Tile &x, int kt, int8_t *S, const int8_t *next) {
        issue(x, kt, S);
        read(next, 0, pa, pb);
        multiply(qa, qb);
        interleave<WL * WB, 1>();
    };
    Tile src = place(t);         // the tile that is being copied
    issue(src, 0, st0);
    issue(src, 1, st1);
    issue(src, 2, st2);
    issue(src, 3, st3);
    wait_copies<(NS - 1) * LPS>();
    lds_barrier();
    read(st0, 0, pa, pb);
    for (;;) {
        const int tn = t + stride, n0 = src.n0, m0 = src.m0;
        const float *pfw = a.ws + min(n0 + (int)threadIdx.x, a.N - 1), *pfx = a.xs + min(m0 + (int)threadIdx.x, a.M - 1);
#pragma unroll
        for (int i = 0; i < WL; ++i)
#pragma unroll
            for (int j = 0; j < WB; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
        for (int kt = 0; kt < nk; kt += NS) {
            const bool last = kt + NS >= nk;
            const int kn = last ? 0 : kt + NS;
            if (last) src = place(tn < tend ? tn : t);      // after the last tile: copies that nothing multiplies
            first_half(st0);
            // the tile's scales (every time, so that every path's copies are the same)
            copy_scales(pfw, pfx, sw + 64 * w, sx + 64 * w);
            second_half(src, kn, st0, st1);
            first_half(st1);
            second_half(src, kn + 1, st1, st2);
            first_half(st2);
            second_half(src, kn + 2, st2, st3);
            first_half(st3);
            second_half(src, kn + 3, st3, st0);
        }

        // The lane's runs of four labels leave as 16 bytes a lane of whole
        // row pieces (64 WL bytes bf16).  Slot s of row q sits at
        // s ^ (q & (slots - 1)).
        int8_t *S = out + w * (RP * 16 * SLOTS);
        const bool whole = m0 + TB <= a.M && n0 + TL <= a.N;
        const int le = opaque(lane), re = le & 31, he = le >> 5;   // addresses formed here, not kept through the steps
        f32x4 sc[WL][4];
#pragma unroll
        for (int i = 0; i < WL; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) sc[i][g] = *(const f32x4 *)(sw + wl + 32 * i + 8 * g + 4 * he);
        float xr[WB];
        u32x4 pk[WL][4];
#pragma unroll
        for (int j = 0; j < WB; ++j) xr[j] = sx[wb + 32 * j + re];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int jp = 0; jp < WB * (32 / RP); ++jp) {
            const int j = jp / (32 / RP), p0 = jp % (32 / RP) * RP;     // rows p0 .. p0 + RP - 1 of MFMA tile j
            if (p0 == 0) {
#pragma unroll
                for (int i = 0; i < WL; ++i)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        float v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][j][4 * g + e] * xr[j] * sc[i][g][e];
                        if (ZB) pk[i][g] = (u32x4){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), 0u, 0u};
                        else pk[i][g] = __builtin_bit_cast(u32x4, (f32x4){v[0], v[1], v[2], v[3]});
                    }
            }
            if (re >= p0 && re < p0 + RP) {
#pragma unroll
                for (int i = 0; i < WL; ++i)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int slot = ZB ? 4 * i + g : 8 * i + 2 * g + he;
                        int8_t *p = S + (re - p0) * (16 * SLOTS) + 16 * (slot ^ (re & (SLOTS - 1)));
                        if (ZB) *(u32x2 *)(p + 8 * he) = (u32x2){pk[i][g][0], pk[i][g][1]};
                        else *(u32x4 *)p = pk[i][g];
                    }
            }
            wave_lds_fence();
            constexpr int RPI = 64 / SLOTS;        // rows a store instruction
            static_assert(RP % RPI == 0, "whole store instructions");
            int8_t *z = (int8_t *)a.Z + ((int64_t)(m0 + wb + 32 * j + p0 + le / SLOTS) * a.N + n0 + wl) * (ZB ? 2 : 4) +
                        16 * (le % SLOTS);
            if (whole) {
                const int64_t step = (int64_t)a.N * (RPI * (ZB ? 2 : 4));
                u32x4 v[RP / RPI];
#pragma unroll
                for (int i = 0; i < RP / RPI; ++i) {
                    const int q = i * RPI + le / SLOTS;
                    v[i] = *(const u32x4 *)(S + q * (16 * SLOTS) + 16 * ((le % SLOTS) ^ ((p0 + q) & (SLOTS - 1))));
                }
                if (a.stream) {
#pragma unroll
                    for (int i = 0; i < RP / RPI; ++i) {
                        if (ZB) __builtin_nontemporal_store(v[i], (u32x4h *)(z + i * step));
                        else __builtin_nontemporal_store(v[i], (u32x4w *)(z + i * step));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < RP / RPI; ++i) {
                        if (ZB) *(u32x4h *)(z + i * step) = v[i];
                        else *(u32x4w *)(z + i * step) = v[i];
                    }
                }
            } else {
#pragma unroll 1
                for (int t0 = 0; t0 < RP; t0 += RPI) {
                    const int q = t0 + le / SLOTS;
                    const u32x4 v = *(const u32x4 *)(S + q * (16 * SLOTS) + 16 * ((le % SLOTS) ^ ((p0 + q) & (SLOTS - 1))));
                    const int left = m0 + wb + 32 * j + p0 + q < a.M ? a.N - (n0 + wl + PER * (le % SLOTS)) : 0;
                    if (left >= PER) {
                        if (ZB) *(u32x4h *)z = v;
                        else *(u32x4w *)z = v;
                    } else {
#pragma unroll
                        for (int e = 0; e < PER - 1; ++e)
                            if (e < left) {
                                if (ZB) ((unsigned short *)z)[e] = (unsigned short)(v[e >> 1] >> (16 * (e & 1)));
                                else ((unsigned *)z)[e] = v[e];
                            }
                    }
                    z += (int64_t)a.N * (RPI * (ZB ? 2 : 4));
                }
            }
            wave_lds_fence();
        }
        if (tn >= tend) break;
        t = tn;
    }
    wait_copies<0>();
}

template <bool ZB>
static hipError_t launch_i8(const I8Args &a, hipStream_t st) {
    if (a.M <= 16) {
        const int64_t wg = ((int64_t)a.N + 63) / 64;
        hipLaunchKernelGGL((k_i8_few<ZB>), dim3((unsigned)(wg < 65536 ? wg : 65536)), dim3(256), 0, st, a);
        return hipGetLastError();
    }
    // Large tiles or small ones by their cost: a round over the CUs measured 5.3
    // + 11 us per 1024 features for 256 x 192 (one workgroup a CU) and 2.8 + 9.6
    // us for 128 x 128 (two; 11.3 a 1024 where the results are past the caches).
    // us, large and small, bf16 logits: 8192 x 1024 -> 32768 356 and 445, x 768
    // 301 and 381, x 256 172 and 189; 4096 x 1024 -> 8192 48.4 and 49.4, x 512
    // 32.4 and 30.0; 512 x 1024 -> 32768 32 and 26; 384 rows 19.7 and 21.0; 2048 x
    // 768 -> 8192 28 and 23.  64 x 64 where the small ones leave a quarter of the
    // CUs without work or half of each tile is past the batch (256 x 768 -> 8192
    // 6.9 against 7.6, 512 rows 11.0 and 8.6; 32 x 1024 -> 32768 9.8 and 11.2).
    auto tiles = [&](int64_t tl, int64_t tb) { return ((a.N + tl - 1) / tl) * ((a.M + tb - 1) / tb); };
    auto grid = [&](int64_t T, int wg_per_cu) {
        const int64_t up = (T + 7) / 8 * 8, most = 256 * wg_per_cu;
        return dim3((unsigned)(up < most ? up : most));
    };
    const int64_t big = tiles(256, 192), mid = tiles(128, 128), few = tiles(64, 64);
    if (big > (1 << 30) || few > INT32_MAX - 8) return hipErrorInvalidValue;
    const double k = (a.K64 + 255) / 256 * 0.25;      // of 1024 features, in whole turns of the ring
    const double tb = (double)((big + 255) / 256) * (5.3 + 11.0 * k),
                 tm = (double)((mid + 511) / 512) * (2.8 + (a.stream ? 11.3 : 9.6) * k);
    if (big >= 256 && tb < tm) hipLaunchKernelGGL((k_i8_tile<4, 3, 1, ZB>), grid(big, 1), dim3(256), 0, st, a);
    else if (a.M > 64 && mid >= 192) hipLaunchKernelGGL((k_i8_tile<2, 2, 2, ZB>), grid(mid, 2), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_i8_tile<1, 1, 4, ZB>), grid(few, 4), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_gemm_i8(int M, int N, int K, const int8_t *A, const float *as, const int8_t *Bm, const float *bs,
                          void *Z, bool zbf, hipStream_t st) {
    I8Args a{A, Bm, as, bs, Z, M, N, (K + 63) / 64 * 64, false};
    a.stream = (int64_t)M * N * (zbf ? 2 : 4) > ((int64_t)256 << 20);
    return zbf ? launch_i8<true>(a, st) : launch_i8<false>(a, st);
}

}  // namespace haste
