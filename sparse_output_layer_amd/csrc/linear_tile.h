// linear_tile.h -- the tiled product of the feature projections
// (linear_bf16.hip, linear_f32.hip):
//
//   C[m][n] = sum_k P[m][k] Q[n][k],   y = act(C + bias) + residual
//
// each operand stored along k (rows m or n) or along m / n (rows k), so that
// the forward product, the input's gradient and the weights' gradient read
// their operands where they lie.  Rows start at 16-byte boundaries and are
// readable to the end of their last 16-byte piece (along k, what is past the
// end there is zeros); M, N and K may be anything.
#pragma once
#include "elem.h"

#include <type_traits>
#include <utility>

namespace haste {

namespace lin {

// what a step past the end multiplies with
__device__ __attribute__((aligned(16))) const unsigned kZeros[4] = {0u, 0u, 0u, 0u};

// s_waitcnt with only the vector-memory count constrained
template <int N>
__device__ __forceinline__ void wait_copies() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// ... with only the LDS count constrained, to zero: the builtin, so that the
// compiler knows of it and does not wait again for reads that follow
__device__ __forceinline__ void wait_reads() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4)); }
// The wave's own LDS writes before this are seen by its lanes' reads after it
__device__ __forceinline__ void wave_lds_fence() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// the same value, not known to be: what is formed from it stays where it is written
__device__ __forceinline__ int opaque(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// Order of N products, R LDS reads and C copies (with their address
// arithmetic) of a half step, spread evenly; nothing is scheduled across the end.
template <int N, int R, int C, int I>
__device__ __forceinline__ void interleave_one() {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);          // MFMA
    constexpr int r = (I + 1) * R / N - I * R / N, c = (I + 1) * C / N - I * C / N;
    if constexpr (r > 0) __builtin_amdgcn_sched_group_barrier(0x100, r, 0);     // LDS read
    if constexpr (c > 0) {
        __builtin_amdgcn_sched_group_barrier(0x006, 10 * c, 0);  // VALU, SALU
        __builtin_amdgcn_sched_group_barrier(0x020, c, 0);       // VMEM read
    }
}
template <int N, int R, int C, int... I>
__device__ __forceinline__ void interleave_all(std::integer_sequence<int, I...>) {
    (interleave_one<N, R, C, I>(), ...);
    __builtin_amdgcn_sched_barrier(0);
}
template <int N, int R, int C>
__device__ __forceinline__ void interleave() {
    interleave_all<N, R, C>(std::make_integer_sequence<int, N>{});
}

// 16 bytes a lane from global memory to 1 KB of LDS at S (wave-uniform)
__device__ __forceinline__ void copy_kb(const char *src, char *S) {
    __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void *)S, 16, 0, 0);
}

constexpr int KB = 64;      // bytes of k per step, for a row of an operand

// Places in a stage.  Operand along k: row r's 16-byte piece s at slot
// s ^ ((r >> 2) & 3) of its 64 bytes: 16 consecutive rows read at one s cover
// the LDS's 256 bytes.  bf16 along m / n: of row k (T columns), the 64-byte
// chunks are permuted by two bits of k and their halves by one, so that the
// rows k .. k + 3 and k + 8 .. k + 11 that a transposing read takes at one
// column fall on different banks.
__device__ __forceinline__ int seg_slot(int r, int s) { return s ^ ((r >> 2) & 3); }
template <int T>
__device__ __forceinline__ int row_slot(int k, int s) {
    const int c = T == 64 ? (k >> 1) & 1 : k & 3;
    return s ^ (4 * c) ^ (2 * ((k >> 3) & 1));
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if (ACT == 0) return z;
    if (ACT == 1) return z > 0.f ? z : z != z ? z : 0.f;
    // z sigmoid(t): t = z, or 2 sqrt(2 / pi) (z + 0.044715 z^3), in powers of two
    constexpr float c = 2.0f * 0.7978845608028654f * kLog2e;
    const float t = ACT == 3 ? z * -kLog2e : z * __builtin_fmaf(z * z, -c * 0.044715f, -c);
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
}

// An operand of T rows / columns of a stage at S: 32 of them from `at`, half
// step ks.  BF: the eight k slots 16 ks + 8 h of column at + lane % 32; fp32:
// the four slots 8 ks + 4 h.
struct Frag {
    u32x4 w;
};
template <bool BF, bool ALONG_K, int T>
__device__ __forceinline__ Frag read_frag(const char *S, int at, int ks, int lane) {
    const int r = lane & 31, h = lane >> 5;
    Frag f;
    if (ALONG_K) {
        const int row = at + r;
        f.w = *(const u32x4 *)(S + row * KB + 16 * seg_slot(row, 2 * ks + h));
    } else if (BF) {
        const int k = 16 * ks + 8 * h + ((lane & 15) >> 2), col = at + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
        const char *p = S + k * (2 * T) + 16 * row_slot<T>(k, col >> 3) + 2 * (col & 7);
        const i16x4 a = lds_read_tr(p), b = lds_read_tr(p + 4 * (2 * T));     // (k + 4 has k's place bits)
        f.w = __builtin_bit_cast(u32x4, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
        const char *p = S + (8 * ks + 4 * h) * (4 * T) + 4 * (at + r);
#pragma unroll
        for (int j = 0; j < 4; ++j) f.w[j] = *(const unsigned *)(p + j * (4 * T));
    }
    return f;
}
template <bool BF>
__device__ __forceinline__ f32x16 multiply(const Frag &a, const Frag &b, f32x16 c) {
    if (BF) return mfma32x32(__builtin_bit_cast(bf16x8, a.w), __builtin_bit_cast(bf16x8, b.w), c);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.w[j]), __uint_as_float(b.w[j]), c, 0, 0, 0);
    return c;
}

// Four elements from element o, of the type
template <bool YB>
__device__ __forceinline__ void get4(const void *p, int64_t o, float *v) {
    if (YB) {
        const u32x2 t = *(const u32x2h *)((const unsigned short *)p + o);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(e & 1 ? t[e >> 1] & 0xffff0000u : t[e >> 1] << 16);
    } else {
        const f32x4 t = *(const f32x4u *)((const float *)p + o);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = t[e];
    }
}

}  // namespace lin

// Tiles of 64 WL columns n x 64 WB rows m, four waves (2 x 2) of WL x WB MFMA
// tiles of 32 x 32 (n its rows, so that a lane ends with runs of four
// consecutive n of one m), k in steps of 64 bytes through a ring of NS LDS
// stages filled by direct global-to-LDS copies.  A workgroup walks over several
// tiles: the copies of the next tile's first steps are under way while this
// one's results are worked on and stored.
template <bool BF, bool PK, bool QK, int WL, int WB, int NS, int PER_CU, bool YB, int ACT>
__global__ __launch_bounds__(256, PER_CU) void k_linear_tile(LinArgs a) {
    using namespace lin;
    constexpr int E = BF ? 2 : 4, KE = KB / E;                     // bytes of an element, elements of a step
    constexpr int TL = 64 * WL, TB = 64 * WB, STAGE = (TL + TB) * KB;
    constexpr int LPS = WL + WB;                                   // copies per wave and step
    constexpr int MF = WL * WB * (BF ? 1 : 4);                     // products and reads of a half step
    constexpr int RD = WL * (QK ? 1 : BF ? 2 : 4) + WB * (PK ? 1 : BF ? 2 : 4);
    constexpr int SLOTS = (YB ? 4 : 8) * WL, PER = YB ? 8 : 4;     // a row's 16-byte slots, elements a slot
    constexpr int ROOM = (163840 / PER_CU - NS * STAGE - 2048) / 4 / (16 * SLOTS);
    constexpr int RP = ROOM >= 32 ? 32 : ROOM >= 16 ? 16 : ROOM >= 8 ? 8 : 4;
    static_assert(ROOM >= 4, "the workgroups' share of the LDS");
    constexpr int RPI = 64 / SLOTS;                                // rows a store instruction
    static_assert(RP % RPI == 0, "whole store instructions");
    __shared__ __attribute__((aligned(1024))) char st0[STAGE];
    __shared__ __attribute__((aligned(1024))) char st1[STAGE];
    __shared__ __attribute__((aligned(1024))) char st2[STAGE];
    __shared__ __attribute__((aligned(1024))) char st3[NS > 3 ? STAGE : 16];
    __shared__ __attribute__((aligned(1024))) char out[4 * RP * 16 * SLOTS];
    __shared__ __attribute__((aligned(16))) float sb[2][256];      // the tile's bias, two tiles in turn
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wl = (w >> 1) * 32 * WL, wb = (w & 1) * 32 * WB;
    // Workgroups go round-robin over the 8 XCDs: each XCD gets a run of
    // consecutive tiles, eight row tiles wide, so that tiles running together
    // share rows of both operands in its L2.
    const int nl = (a.N + TL - 1) / TL, nb = (a.M + TB - 1) / TB, plane = nl * nb, T = plane * a.splits;
    const int per = (T + 7) / 8, stride = (int)gridDim.x >> 3;
    const int tend = min(T, ((int)(blockIdx.x & 7) + 1) * per);
    int t = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if (t >= tend) return;

    struct Tile {
        const char *q, *p;       // the operands at its first column, row and k
        int n0, m0, split;
        int k;                   // elements of k
        unsigned off[LPS];       // copy c of a wave: 1 KB of the stage (Q, then P); rows past the end
                                 // read the last one
    };
    // copy `blk` of an operand of T rows: the lane's k within the step
    auto k_of = [&](bool q, int blk) {
        const int along = (16 / E) * seg_slot((lane >> 2) & 15, lane & 3);
        return q ? (QK ? along : blk * (1024 / (TL * E)) + lane / (TL * E / 16))
                 : (PK ? along : blk * (1024 / (TB * E)) + lane / (TB * E / 16));
    };
    auto place = [&](int i) {
        Tile x;
        x.split = i / plane;
        i -= x.split * plane;
        const int band = i / (8 * nl), wide = min(8, nb - 8 * band), u = i - band * 8 * nl;
        x.n0 = (u / wide) * TL;
        x.m0 = (8 * band + u % wide) * TB;
        const int64_t k0 = (int64_t)x.split * a.k_split;
        x.k = (int)min((int64_t)a.k_split, a.K - k0);
        x.q = (const char *)a.Q + E * (QK ? x.n0 * a.ldq + k0 : k0 * a.ldq + x.n0);
        x.p = (const char *)a.P + E * (PK ? x.m0 * a.ldp + k0 : k0 * a.ldp + x.m0);
#pragma unroll
        for (int c = 0; c < LPS; ++c) {
            const int b = w * LPS + c;
            const bool q = 16 * b < TL;
            const int blk = q ? b : b - TL / 16, left = q ? a.N - x.n0 : a.M - x.m0;
            const unsigned ld = (unsigned)((q ? a.ldq : a.ldp) * E);
            if (q ? QK : PK) {
                const int row = 16 * blk + (lane >> 2);
                x.off[c] = (unsigned)min(row, left - 1) * ld + 16u * seg_slot(row, lane & 3);
            } else {
                const int k = k_of(q, blk), s = q ? lane % (TL * E / 16) : lane % (TB * E / 16);
                const int col = (16 / E) * (!BF ? s : q ? row_slot<TL>(k, s) : row_slot<TB>(k, s));
                x.off[c] = (unsigned)k * ld + (unsigned)(E * min(col, (left - 1) & ~(16 / E - 1)));
            }
        }
        return x;
    };
    // step kt of a tile into stage S; what is past the end is zeros
    auto issue = [&](const Tile &x, int kt, char *S) {
#pragma unroll
        for (int c = 0; c < LPS; ++c) {
            const int b = w * LPS + c;
            const bool q = 16 * b < TL;
            const bool in = kt * KE + k_of(q, q ? b : b - TL / 16) < x.k;
            const int64_t at = (int64_t)kt * (q ? (QK ? KB : KE * E * a.ldq) : (PK ? KB : KE * E * a.ldp));
            const char *src = (q ? x.q : x.p) + at + x.off[c];
            copy_kb(in ? src : (const char *)kZeros, S + b * 1024);
        }
    };
    f32x16 acc[WL][WB];
    Frag pa[WL], pb[WB], qa[WL], qb[WB];
    auto read = [&](const char *S, int ks, Frag *av, Frag *bv) {
#pragma unroll
        for (int i = 0; i < WL; ++i) av[i] = read_frag<BF, QK, TL>(S, wl + 32 * i, ks, lane);
#pragma unroll
        for (int j = 0; j < WB; ++j) bv[j] = read_frag<BF, PK, TB>(S + TL * KB, wb + 32 * j, ks, lane);
    };
    auto products = [&](const Frag *av, const Frag *bv) {
#pragma unroll
        for (int i = 0; i < WL; ++i)
#pragma unroll
            for (int j = 0; j < WB; ++j) acc[i][j] = lin::multiply<BF>(av[i], bv[j], acc[i][j]);
    };
    // A step on stage S: the operands of its first half are in registers, the
    // second half's are read while the first multiplies.  Then this wave's
    // copies of the next step have landed (those of the steps after it stay in
    // flight), and the barrier makes that everyone's and says that every wave
    // has read all of stage S, which the copies of NS steps on (or of the next
    // tile's first steps) fill.
    auto first_half = [&](const char *S) {
        wait_reads();
        read(S, 1, qa, qb);
        products(pa, pb);
        interleave<MF, RD, 0>();
        wait_reads();
        wait_copies<(NS - 2) * LPS>();
        lds_barrier();
    };
    auto second_half = [&](const Tile &x, int kt, char *S, const char *next) {
        issue(x, kt, S);
        read(next, 0, pa, pb);
        products(qa, qb);
        interleave<MF, RD, LPS>();
    };
    Tile src = place(t);         // the tile that is being copied
    issue(src, 0, st0);
    issue(src, 1, st1);
    issue(src, 2, st2);
    if (NS > 3) issue(src, 3, st3);
    wait_copies<(NS - 1) * LPS>();
    lds_barrier();
    read(st0, 0, pa, pb);
    int turn = 0;
    for (;;) {
        const int tn = t + stride, n0 = src.n0, m0 = src.m0, split = src.split;
        const int nk = (src.k + KE - 1) / KE;
        // The tile's bias: a wave that is ahead writes the one that the others,
        // still at the tile before, do not read
        turn ^= 1;
        if (a.bias) {
            const int n = min(n0 + (int)threadIdx.x, a.N - 1);
            auto *dst = (__attribute__((address_space(3))) void *)(sb[turn] + 64 * w);
            if (a.bias_bf) __builtin_amdgcn_global_load_lds((const unsigned short *)a.bias + n, dst, 2, 0, 0);
            else __builtin_amdgcn_global_load_lds((const float *)a.bias + n, dst, 4, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < WL; ++i)
#pragma unroll
            for (int j = 0; j < WB; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
        for (int kt = 0; kt < nk; kt += NS) {
            const bool last = kt + NS >= nk;
            const int kn = last ? 0 : kt + NS;
            if (last) src = place(tn < tend ? tn : t);      // after the last tile: copies that nothing multiplies
            first_half(st0);
            second_half(src, kn, st0, st1);
            first_half(st1);
            second_half(src, kn + 1, st1, st2);
            first_half(st2);
            second_half(src, kn + 2, st2, NS > 3 ? st3 : st0);
            if (NS > 3) {
                first_half(st3);
                second_half(src, kn + 3, st3, st0);
            }
        }

        // The lane's runs of four n: bias, activation and residual in
        // registers, then through LDS, so that 16 bytes a lane of whole row
        // pieces leave.  Slot s of row q sits at s ^ (q & (slots - 1)).
        char *S = out + w * (RP * 16 * SLOTS);
        const bool whole = m0 + TB <= a.M && n0 + TL <= a.N;
        const int le = opaque(lane), re = le & 31, he = le >> 5;   // addresses formed here, not kept through the steps
        char *C = (char *)a.C + (int64_t)split * a.M * a.ldc * (YB ? 2 : 4);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < WB; ++j) {
            const int m = m0 + wb + 32 * j + re;
            u32x4 pk[WL][4], zk[WL][4];
#pragma unroll
            for (int i = 0; i < WL; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int nn = wl + 32 * i + 8 * g + 4 * he, n = n0 + nn;
                    float v[4], r[4] = {};
                    f32x4 bias = {0.f, 0.f, 0.f, 0.f};
                    if (a.bias) {
                        bias = *(const f32x4 *)(sb[turn] + nn);
                        if (a.bias_bf) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) bias[e] = __uint_as_float(__float_as_uint(bias[e]) << 16);
                        }
                    }
                    if (a.res) {
                        if (whole || (m < a.M && n + 4 <= a.N)) {
                            get4<YB>(a.res, (int64_t)m * a.ldr + n, r);
                        } else if (m < a.M) {
#pragma unroll
                            for (int e = 0; e < 3; ++e)
                                if (n + e < a.N) r[e] = load1<YB>(a.res, (int64_t)m * a.ldr + n + e);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * g + e] + bias[e];
                    if (ACT) {
                        if (YB) zk[i][g] = (u32x4){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), 0u, 0u};
                        else zk[i][g] = __builtin_bit_cast(u32x4, (f32x4){v[0], v[1], v[2], v[3]});
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = activate<ACT>(v[e]) + r[e];
                    if (YB) pk[i][g] = (u32x4){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), 0u, 0u};
                    else pk[i][g] = __builtin_bit_cast(u32x4, (f32x4){v[0], v[1], v[2], v[3]});
                }
            auto leave = [&](const u32x4 (&k)[WL][4], char *to, int64_t ld) {
#pragma unroll
                for (int p0 = 0; p0 < 32; p0 += RP) {      // rows p0 .. p0 + RP - 1 of MFMA tile j
                    if (re >= p0 && re < p0 + RP) {
#pragma unroll
                        for (int i = 0; i < WL; ++i)
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                const int slot = YB ? 4 * i + g : 8 * i + 2 * g + he;
                                char *p = S + (re - p0) * (16 * SLOTS) + 16 * (slot ^ (re & (SLOTS - 1)));
                                if (YB) *(u32x2 *)(p + 8 * he) = (u32x2){k[i][g][0], k[i][g][1]};
                                else *(u32x4 *)p = k[i][g];
                            }
                    }
                    wave_lds_fence();
                    char *z = to + ((m0 + wb + 32 * j + p0 + le / SLOTS) * ld + n0 + wl) * (YB ? 2 : 4) + 16 * (le % SLOTS);
                    const int64_t step = ld * (RPI * (YB ? 2 : 4));
                    if (whole) {
                        u32x4 v[RP / RPI];
#pragma unroll
                        for (int i = 0; i < RP / RPI; ++i) {
                            const int q = i * RPI + le / SLOTS;
                            v[i] = *(const u32x4 *)(S + q * (16 * SLOTS) + 16 * ((le % SLOTS) ^ ((p0 + q) & (SLOTS - 1))));
                        }
#pragma unroll
                        for (int i = 0; i < RP / RPI; ++i) {
                            if (YB) *(u32x4h *)(z + i * step) = v[i];
                            else *(u32x4w *)(z + i * step) = v[i];
                        }
                    } else {
#pragma unroll 1
                        for (int t0 = 0; t0 < RP; t0 += RPI) {
                            const int q = t0 + le / SLOTS;
                            const u32x4 v = *(const u32x4 *)(S + q * (16 * SLOTS) + 16 * ((le % SLOTS) ^ ((p0 + q) & (SLOTS - 1))));
                            const int left = m0 + wb + 32 * j + p0 + q < a.M ? a.N - (n0 + wl + PER * (le % SLOTS)) : 0;
                            if (left >= PER) {
                                if (YB) *(u32x4h *)z = v;
                                else *(u32x4w *)z = v;
                            } else {
#pragma unroll
                                for (int e = 0; e < PER - 1; ++e)
                                    if (e < left) {
                                        if (YB) ((unsigned short *)z)[e] = (unsigned short)(v[e >> 1] >> (16 * (e & 1)));
                                        else ((unsigned *)z)[e] = v[e];
                                    }
                            }
                            z += step;
                        }
                    }
                    wave_lds_fence();
                }
            };
            if (ACT && a.Z) leave(zk, (char *)a.Z, a.N);
            leave(pk, C, a.ldc);
        }
        if (tn >= tend) break;
        t = tn;
    }
    wait_copies<0>();
}

}  // namespace haste
