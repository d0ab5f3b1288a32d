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

// s_waitcnt with only the vector-memory count constrained
template <int N>
__device__ __forceinline__ void wait_copies() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// ... with only the LDS count constrained, to zero: the builtin, so that the
// compiler knows of it and does not wait again for reads that follow
__device__ __forceinline__ void wait_reads() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4)); }
// the same value, not known to be: what is formed from it stays where it is written
__device__ __forceinline__ int opaque(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// f(0), f(1), ... f(N - 1), each with its number as a constant
template <class F, int... I>
__device__ __forceinline__ void each_of(F &&f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F &&f) { each_of(f, std::make_integer_sequence<int, N>{}); }

// Copies go through buffer descriptors that end with the operand's last
// element of the step (at most 2^31 bytes): what lies past it, rows and k past
// the end among it, reads as zeros without a comparison, and a copy is one
// instruction without 64-bit address arithmetic.  A lane whose offset is kPast
// reads zeros too.
constexpr unsigned kPast = 0x80000000u;
typedef u32x4 Buffer;
__device__ __forceinline__ Buffer buffer(const char *base, unsigned bytes) {      // both wave-uniform
    const uint64_t p = (uint64_t)base;
    Buffer b = {(unsigned)__builtin_amdgcn_readfirstlane((int)p), (unsigned)__builtin_amdgcn_readfirstlane((int)(p >> 32)) & 0xffffu,
                (unsigned)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
    asm volatile("s_nop 4" : "+s"(b));      // scalars that vector instructions wrote are not read by a load before
    return b;
}
// 16 bytes a lane to 1 KB of LDS at address S (wave-uniform).  Written out,
// because the compiler takes a transposing read for one of whatever a copy in
// flight writes and waits for all of them; it has no result register, and the
// kernel's own waits and barriers order what it writes.  (m0, the LDS address of
// such loads, is used by nothing else here.)
__device__ __forceinline__ void copy_kb(Buffer b, unsigned off, unsigned S) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(S), "v"(off), "s"(b));
}
// ... and an element a lane (a word of LDS each, bf16 in its low half)
__device__ __forceinline__ void copy_elements(Buffer b, unsigned off, unsigned S, bool bf) {
    if (bf) asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ushort %1, %2, 0 offen lds" ::"s"(S), "v"(off), "s"(b));
    else asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(S), "v"(off), "s"(b));
}
// a stage's address in LDS
__device__ __forceinline__ unsigned lds_at(const char *S) {
    return (unsigned)(uintptr_t)(__attribute__((address_space(3))) const char *)S;
}

// Bytes of k per row of a stage that holds rows along k: a cache line, so that
// a copy moves whole lines (64 bytes a step fetched every line twice: 8192^3 bf16
// zeros 950 us).
constexpr int LINE = 128;

// Places in a stage.  Operand along k: row r's 16-byte piece s at slot
// s ^ ((r >> 1) & 7) of its 128 bytes: 16 consecutive rows read at one s cover
// the LDS's 256 bytes.  bf16 along m / n: of row k (T columns), the 64-byte
// chunks are permuted by two bits of k and their halves by one, so that the
// rows k .. k + 3 and k + 8 .. k + 11 that a transposing read takes at one
// column fall on different banks.
__device__ __forceinline__ int seg_slot(int r, int s) { return s ^ ((r >> 1) & 7); }
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

// An operand of T rows / columns of a stage at S: 32 of them from `at`, part ks
// of the step.  BF: the eight k slots 16 ks + 8 h of column at + lane % 32; fp32:
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
        f.w = *(const u32x4 *)(S + row * LINE + 16 * seg_slot(row, 2 * ks + h));
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
// 16 bytes of results (PER elements) at z, of which `left` are in the row
template <bool YB>
__device__ __forceinline__ void put(char *z, u32x4 t, int left) {
    constexpr int PER = YB ? 8 : 4;
    if (left >= PER) {
        if (YB) *(u32x4h *)z = t;
        else *(u32x4w *)z = t;
        return;
    }
#pragma unroll 1
    for (int e = 0; e < left; ++e) {
        if (YB) {
            ((unsigned short *)z)[e] = (unsigned short)t[0];
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] = t[i] >> 16 | (i < 3 ? t[i < 3 ? i + 1 : 3] << 16 : 0u);
        } else {
            ((unsigned *)z)[e] = t[0];
#pragma unroll
            for (int i = 0; i < 3; ++i) t[i] = t[i + 1];
        }
    }
}
template <bool YB>
__device__ __forceinline__ u32x4 get(const char *z, int left) {
    constexpr int PER = YB ? 8 : 4;
    if (left >= PER) return YB ? *(const u32x4h *)z : *(const u32x4w *)z;
    u32x4 t = {0u, 0u, 0u, 0u};
#pragma unroll 1
    for (int e = left - 1; e >= 0; --e) {
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            if (YB) t[i] = t[i] << 16 | (i ? t[i ? i - 1 : 0] >> 16 : ((const unsigned short *)z)[e]);
            else t[i] = i ? t[i ? i - 1 : 0] : ((const unsigned *)z)[e];
        }
    }
    return t;
}

// The results of one MFMA tile (32 n x 32 m): lane l has m = l % 32 and the
// sixteen n 8 g + 4 (l / 32) + e (element 4 g + e).  They leave in 16-byte pieces
// of rows m: half-waves, rows of 16 lanes and half of those rows change places in
// registers until a store writes 128 bytes of each of 8 rows (NT = 2 bf16 tiles
// beside each other, or an fp32 one), or 64 bytes of each of 16 (one bf16 tile).
// Every exchange is its own inverse, so that the same ones in turn lead back.
template <bool YB, int NT>
struct Pieces {
    static constexpr int N = YB ? 2 * NT : 4;
    u32x4 w[N];
    // piece k of a lane: its row of the 32 and its first column
    __device__ __forceinline__ static int row(int k) { return N == 4 ? 16 * (k & 1) + 8 * (k >> 1) : 16 * k; }
    __device__ __forceinline__ static int lane_row(int l) { return N == 4 ? l & 7 : l & 15; }
    __device__ __forceinline__ static int lane_column(int l) {
        return (YB ? 8 : 4) * ((N == 4 ? 4 * ((l >> 3) & 1) : 0) + 2 * ((l >> 4) & 1) + (l >> 5));
    }
    __device__ __forceinline__ static void swap8(u32x4 &x, u32x4 &y) {      // lanes 8 .. 15 of x's rows with lanes 0 .. 7 of y's
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int p = (int)x[e], q = (int)y[e];                         // (0x128: row_ror:8)
            x[e] = (unsigned)__builtin_amdgcn_update_dpp(p, q, 0x128, 0xf, 0xc, false);
            y[e] = (unsigned)__builtin_amdgcn_update_dpp(q, p, 0x128, 0xf, 0x3, false);
        }
    }
    __device__ __forceinline__ static void swap16(u32x4 &x, u32x4 &y) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const auto r = __builtin_amdgcn_permlane16_swap(x[e], y[e], false, false);
            x[e] = r[0], y[e] = r[1];
        }
    }
    __device__ __forceinline__ static void swap32(u32x4 &x) {               // words 0, 1 of g with words 2, 3 of g + 1
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const auto r = __builtin_amdgcn_permlane32_swap(x[e], x[2 + e], false, false);
            x[e] = r[0], x[2 + e] = r[1];
        }
    }
    __device__ __forceinline__ void from(const f32x16 *v) {
        if constexpr (YB) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[k][e] = pack_bf16x2(v[k >> 1][8 * (k & 1) + 2 * e], v[k >> 1][8 * (k & 1) + 2 * e + 1]);
                swap32(w[k]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) w[k][e] = __float_as_uint(v[0][4 * k + e]);
        }
#pragma unroll
        for (int k = 0; k < N; k += 2) swap16(w[k], w[k + 1]);
        if constexpr (N == 4) swap8(w[0], w[2]), swap8(w[1], w[3]);
    }
    __device__ __forceinline__ void add_to(f32x16 *v) {
        if constexpr (N == 4) swap8(w[0], w[2]), swap8(w[1], w[3]);
#pragma unroll
        for (int k = 0; k < N; k += 2) swap16(w[k], w[k + 1]);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if constexpr (YB) {
                swap32(w[k]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[k >> 1][8 * (k & 1) + 2 * e] += __uint_as_float(w[k][e] << 16);
                    v[k >> 1][8 * (k & 1) + 2 * e + 1] += __uint_as_float(w[k][e] & 0xffff0000u);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[0][4 * k + e] += __uint_as_float(w[k][e]);
            }
        }
    }
};

}  // namespace lin

// Tiles of 64 WT columns n x 64 WT rows m, four waves (2 x 2) of WT x WT MFMA
// tiles of 32 x 32 (n its rows, so that a lane ends with runs of four
// consecutive n of one m), k in steps through a ring of LDS stages filled by
// direct global-to-LDS copies: two stages of 128 bytes of k a row, or, where
// both operands are stored across k and no copy is shorter than its rows, four
// of 64, which gives a copy three steps to land instead of one (weight gradient
// of 65536 x 768 -> 1024 164 us with two stages, 98 with four).  A workgroup
// walks over several tiles: the copies of the next tile's first steps are under
// way while this one's results are worked on and stored.
//
// Bound by the matrix cores, and by the stores, which nothing runs beside: with
// 256 x 256 tiles a CU's registers hold one workgroup.  bf16 65536 x 768 -> 2048
// 235 to 250 us (206 GFLOP; the products alone 185, the 268 MB of results alone
// 50), with gelu and z kept 292 to 305; 8192^3 880 us (1250 TFLOP/s; zeros 780).
// Two workgroups a CU (128 x 256) run stores beside products, but read more LDS
// for a product: 312 and 1080.  Results through LDS instead of exchanges of
// lanes: 265, and 340 with a residual (290).
template <bool BF, bool PK, bool QK, int WT, int PER_CU, bool YB, int ACT>
__global__ __launch_bounds__(256, PER_CU) void k_linear_tile(LinArgs a) {
    using namespace lin;
    constexpr bool FOUR = !PK && !QK;                              // stages
    constexpr int KB = FOUR ? 64 : LINE, NS = FOUR ? 4 : 2;        // bytes of k a step, stages
    constexpr int E = BF ? 2 : 4, KE = KB / E;                     // bytes of an element, elements of a step
    constexpr int T_ = 64 * WT, STAGE = 2 * T_ * KB;               // columns and rows of a tile, bytes of a stage
    constexpr int LPS = WT * KB / 32;                              // copies per wave and step
    constexpr int MF = WT * WT * (BF ? 1 : 4);                     // products of a part of a step
    constexpr int PER = YB ? 8 : 4, NT = YB && WT > 1 ? 2 : 1;     // elements of a 16-byte piece; MFMA tiles worked on at a time
    typedef Pieces<YB, NT> Unit;
    __shared__ __attribute__((aligned(1024))) char st0[STAGE];
    __shared__ __attribute__((aligned(1024))) char st1[STAGE];
    __shared__ __attribute__((aligned(1024))) char st2[FOUR ? STAGE : 16];
    __shared__ __attribute__((aligned(1024))) char st3[FOUR ? STAGE : 16];
    // fp32 results: the bias is added to the finished sums.  Sums that begin with
    // one that is large against them are rounded to its size at every step (bias
    // 100 times the sum, bf16 operands, 16384 k: 44 times as far from the exact
    // result).  A bf16 result is rounded to 2^-9 of itself, and its chain, a step
    // each 16 k, begins with the bias, which costs nothing: 65536 x 768 -> 2048 with
    // gelu 295 us, with the bias added at the end 304.
    constexpr bool BEGIN = YB;
    // The tile's bias, tiles in turn: it is copied during the tile before, whose
    // begin some waves reach while others still add theirs to the tile before that.
    constexpr int TURNS = BEGIN ? 2 : 3;
    __shared__ __attribute__((aligned(16))) float sb[TURNS][256];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wl = (w >> 1) * 32 * WT, wb = (w & 1) * 32 * WT;
    // Workgroups go round-robin over the 8 XCDs: each XCD gets a run of
    // consecutive tiles, eight row tiles wide, so that tiles running together
    // share rows of both operands in its L2.
    const int nl = (a.N - 1) / T_ + 1, nb = (a.M - 1) / T_ + 1, plane = nl * nb, T = plane * a.splits;
    const int per = (T + 7) / 8, stride = (int)gridDim.x >> 3;
    const int tend = min(T, ((int)(blockIdx.x & 7) + 1) * per);
    int t = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if (t >= tend) return;

    // Waves 0 and 1 copy Q's half of a stage, waves 2 and 3 P's; `mine` is the
    // wave's operand.  A copy is 1 KB of it: eight rows along k, or 1024 / (T E)
    // rows of T columns.
    const bool mine_q = w < 2, mine_k = mine_q ? QK : PK;
    const int64_t ld64 = mine_q ? a.ldq : a.ldp;
    const unsigned ld = (unsigned)ld64 * E, copy_ld = ld * (mine_k ? 8u : 1024u / (T_ * E));
    const int64_t step_bytes = mine_k ? KB : (int64_t)KE * ld;
    const int all = mine_q ? a.N : a.M;
    struct Tile {
        const char *src;         // mine at the tile's first column or row and k
        int n0, m0, split;
        int k, left;             // elements of k; rows or columns of mine, at most T_
    };
    auto place = [&](int i) {
        Tile x;
        x.split = i / plane;
        i -= x.split * plane;
        const int band = i / (8 * nl), wide = min(8, nb - 8 * band), u = i - band * 8 * nl;
        x.n0 = (u / wide) * T_;
        x.m0 = (8 * band + u % wide) * T_;
        const int64_t k0 = (int64_t)x.split * a.k_split, at = mine_q ? x.n0 : x.m0;
        x.k = (int)min((int64_t)a.k_split, a.K - k0);
        x.left = min(all - (int)at, T_);
        x.src = (const char *)(mine_q ? a.Q : a.P) + E * (mine_k ? at * ld64 + k0 : k0 * ld64 + at);
        return x;
    };
    // A lane's offset in a copy, with the copies of the other wave before it;
    // bits 0 and BIT of the copy's number permute the pieces of the rows.
    constexpr int BIT = T_ == 256 ? 2 : 1;
    unsigned o[4];
    int along[2];                // the lane's first element of k (rows along k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        constexpr int SEGS = T_ * E / 16, RPB = 64 / SEGS;
        const int ka = (16 / E) * ((lane & 7) ^ (4 * (i & 1) + (lane >> 4)));
        const int k = RPB * ((i & 1) + (i >> 1 << BIT)) + lane / SEGS, s = lane % SEGS;
        o[i] = (unsigned)((w & 1) * LPS) * copy_ld + (mine_k ? (unsigned)(lane >> 3) * ld + (unsigned)(E * ka)
                                                             : (unsigned)(lane / SEGS) * ld + 16u * (BF ? row_slot<T_>(k, s) : s));
        if (i < 2) along[i] = mine_k ? ka : 0;
    }
    // where copies go to and come from: step kt of a tile, stage S
    struct Copies {
        Buffer b;
        unsigned S;
        int k;                   // elements of k from the step on
    };
    auto copies = [&](const Tile &x, int kt, const char *S) {
        Copies z;
        z.k = x.k - kt * KE;
        const int kin = max(min(z.k, KE), 1);
        unsigned bytes = mine_k ? (unsigned)(x.left - 1) * ld + (unsigned)((kin * E + 15) & ~15)
                                : (unsigned)(kin - 1) * ld + (unsigned)((x.left * E + 15) & ~15);
        bytes *= (unsigned)(z.k > 0);      // what is past the end is zeros
        z.b = buffer(x.src + kt * step_bytes, bytes);
        z.S = lds_at(S) + w * (LPS * 1024);
        return z;
    };
    auto copy = [&](const Copies &z, int c) {
        copy_kb(z.b, along[c & 1] < z.k ? o[(c & 1) + 2 * ((c >> BIT) & 1)] + (unsigned)c * copy_ld : kPast, z.S + c * 1024);
    };
    // fp32 results are only as good as the order of their sum: runs of 256 k, each
    // summed by itself, are added to `total` (one run over 4096 k is 3.6 times as
    // far from the exact sum, and twice as far as the library's)
    constexpr int RUN = 256 / KE;
    f32x16 acc[WT][WT], total[WT][WT];
    Frag pa[WT], pb[WT], qa[WT], qb[WT];
    int lr = lane;               // formed anew for every tile: the addresses of its reads are not kept through the results
    // Part of a step: products of the operands a and b; those of the next part
    // (part ks of stage S) are read into na and nb behind the first half of the
    // products, so that they have landed when it begins, and copies C0 .. C1 - 1
    // leave between the products.  The order is the one written here.
    auto part = [&](const Frag *a, const Frag *b, const char *S, int ks, Frag *na, Frag *nb, const Copies &z, auto c0, auto c1) {
        constexpr int C0 = decltype(c0)::value, C = decltype(c1)::value - C0, H = MF > 1 ? MF / 2 : 1, R = 2 * WT;
        wait_reads();
        each<MF>([&](auto n) {
            constexpr int P = decltype(n)::value, i = P / WT % WT, j = P % WT, s = P / (WT * WT);
            if constexpr (BF) acc[i][j] = mfma32x32(__builtin_bit_cast(bf16x8, a[i].w), __builtin_bit_cast(bf16x8, b[j].w), acc[i][j]);
            else acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[i].w[s]), __uint_as_float(b[j].w[s]), acc[i][j], 0, 0, 0);
            constexpr int r0 = P < H ? P * R / H : R, r1 = P < H ? (P + 1) * R / H : R;
#pragma unroll
            for (int r = r0; r < r1; ++r) {
                if (r < WT) na[r < WT ? r : 0] = read_frag<BF, QK, T_>(S, wl + 32 * r, ks, lr);
                else nb[r < WT ? 0 : r - WT] = read_frag<BF, PK, T_>(S + T_ * KB, wb + 32 * (r - WT), ks, lr);
            }
#pragma unroll
            for (int c = P * C / MF; c < (P + 1) * C / MF; ++c) copy(z, C0 + c);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    constexpr int EARLY = FOUR ? LPS : LPS / 2;      // copies that leave in a step's last part; the others in the next one's first
    const std::integral_constant<int, 0> c0;
    const std::integral_constant<int, EARLY> ce;
    const std::integral_constant<int, LPS> c1;
    // what every wave has read and copied is everyone's
    auto meet = [&](auto in_flight) {
        wait_reads();
        wait_copies<decltype(in_flight)::value>();
        lds_barrier();
    };
    // Two stages: a step on stage S is four parts.  The second half of the next
    // step's copies (stage N, step kx of tile x) leaves in the first, and after
    // the third all of them have landed; then every wave has read all of S,
    // which the copies of step ky of tile y fill from the last part on.
    auto step = [&](char *S, char *N, const Tile &x, int kx, const Tile &y, int ky) {
        const Copies u = copies(x, kx, N);
        part(pa, pb, S, 1, qa, qb, u, ce, c1);
        part(qa, qb, S, 2, pa, pb, u, c0, c0);
        part(pa, pb, S, 3, qa, qb, u, c0, c0);
        meet(c0);
        const Copies v = copies(y, ky, S);
        part(qa, qb, N, 0, pa, pb, v, c0, ce);
    };
    // Four stages: a step is two parts, between them the copies of the next step
    // have landed; those of the two after it stay in flight.
    auto half_step = [&](char *S, char *N, const Tile &y, int ky) {
        const Copies v = copies(y, ky, S);
        part(pa, pb, S, 1, qa, qb, v, c0, c0);
        meet(std::integral_constant<int, 2 * LPS>{});
        part(qa, qb, N, 0, pa, pb, v, c0, c1);
    };
    auto fill = [&](const Tile &x, int kt, char *S, int n) {
        const Copies z = copies(x, kt, S);
#pragma unroll
        for (int c = 0; c < LPS; ++c)
            if (c < n) copy(z, c);
    };
    const int bias_shift = a.bias && a.bias_bf ? 16 : 0;      // bf16 copies lie in the low half of a word
    auto copy_bias = [&](int n0, int turn) {
        const unsigned e = a.bias_bf ? 2u : 4u, left = (unsigned)(a.N - n0);
        copy_elements(buffer((const char *)a.bias + (int64_t)n0 * e, left * e), min((unsigned)threadIdx.x, left - 1) * e,
                      lds_at((const char *)(sb[turn] + 64 * w)), a.bias_bf);
    };
    Tile src = place(t);         // the tile that is being copied
    if (a.bias) copy_bias(src.n0, 0);
    else if (BEGIN) sb[0][threadIdx.x] = sb[1][threadIdx.x] = 0.f;
    fill(src, 0, st0, LPS);
    if constexpr (FOUR) {
        fill(src, 1, st1, LPS);
        fill(src, 2, st2, LPS);
        fill(src, 3, st3, LPS);
        wait_copies<3 * LPS>();
    } else {
        fill(src, 1, st1, EARLY);
        wait_copies<EARLY>();
    }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < WT; ++i) {
        pa[i] = read_frag<BF, QK, T_>(st0, wl + 32 * i, 0, lane);
        pb[i] = read_frag<BF, PK, T_>(st0 + T_ * KB, wb + 32 * i, 0, lane);
    }
    int turn = 0;
    for (;;) {
        const int tn = t + stride, n0 = src.n0, m0 = src.m0, split = src.split;
        const int nk = (src.k + KE - 1) / KE;
        const float *bias = sb[turn];
        auto bias_at = [&](int i, int g, float *x) {      // of a lane's four columns from 8 g of MFMA tiles i
            const u32x4 b = *(const u32x4 *)(bias + wl + 32 * i + 8 * g + 4 * (lane >> 5));
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(b[e] << bias_shift);
        };
#pragma unroll
        for (int i = 0; i < WT; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float x[4] = {0.f, 0.f, 0.f, 0.f};
                if (BEGIN) bias_at(i, g, x);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int j = 0; j < WT; ++j) (BF ? acc : total)[i][j][4 * g + e] = x[e];
            }
        turn = turn + 1 < TURNS ? turn + 1 : 0;
        const Tile next = place(tn < tend ? tn : t);      // after the last tile: copies that nothing multiplies
        if (a.bias) copy_bias(next.n0, turn);
        lr = opaque(lane);
        int kt = 0;
        do {
            if constexpr (!BF) {
#pragma unroll
                for (int i = 0; i < WT; ++i)
#pragma unroll
                    for (int j = 0; j < WT; ++j)
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
            }
            const int end = BF ? nk : min(nk, kt + RUN);
            do {
                const bool last = kt + NS >= nk;
                const int kn = last ? 0 : kt + NS;
                const Tile now = src;
                if (last) src = next;
                if constexpr (FOUR) {
                    half_step(st0, st1, src, kn);
                    half_step(st1, st2, src, kn + 1);
                    half_step(st2, st3, src, kn + 2);
                    half_step(st3, st0, src, kn + 3);
                } else {
                    step(st0, st1, now, kt + 1, src, kn);
                    step(st1, st0, src, kn, src, kn + 1);
                }
                kt += NS;
            } while (kt < end);
            if constexpr (!BF) {
#pragma unroll
                for (int i = 0; i < WT; ++i)
#pragma unroll
                    for (int j = 0; j < WT; ++j) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) total[i][j][e] += acc[i][j][e];
                        asm volatile("" : "+v"(total[i][j]));
                    }
            }
        } while (!BF && kt < nk);
        // the sums stay in the matrix cores' registers until a tile of them is worked on
        if constexpr (BF) {
#pragma unroll
            for (int i = 0; i < WT; ++i)
#pragma unroll
                for (int j = 0; j < WT; ++j) asm volatile("" : "+a"(acc[i][j]));
        }

        // Activation and residual in registers, 64-byte pieces of rows from
        // them.  The residual's pieces are under way some MFMA tiles ahead.
        const bool whole = a.M - m0 >= T_ && a.N - n0 >= T_;
        const int le = opaque(lane);                     // addresses formed here, not kept through the steps
        const int col = n0 + wl + Unit::lane_column(le), row = wb + Unit::lane_row(le);      // row: of the tile
        auto at = [&](const void *to, int64_t ld, int i, int j, int k) {      // piece k of the unit at tile i, j
            return (char *)to + (((int64_t)m0 + row + 32 * j + Unit::row(k)) * ld + col + 32 * i) * (YB ? 2 : 4);
        };
        auto left = [&](int i, int j, int k) { return row + 32 * j + Unit::row(k) < a.M - m0 ? a.N - (col + 32 * i) : 0; };
        constexpr int PAIRS = WT / NT, UNITS = PAIRS * WT, AHEAD = UNITS < (YB ? 4 : 2) ? UNITS : YB ? 4 : 2;
        Unit r[AHEAD];
        auto fetch = [&](int x) {
            const int i = NT * (x % PAIRS), j = x / PAIRS;
            if (whole) {
#pragma unroll
                for (int k = 0; k < Unit::N; ++k) r[x % AHEAD].w[k] = get<YB>(at(a.res, a.ldr, i, j, k), PER);
            } else {
#pragma unroll
                for (int k = 0; k < Unit::N; ++k) r[x % AHEAD].w[k] = get<YB>(at(a.res, a.ldr, i, j, k), left(i, j, k));
            }
        };
        auto leave = [&](const f32x16 *v, void *to, int64_t ld, int i, int j) {
            Unit p;
            p.from(v);
            if (whole) {
#pragma unroll
                for (int k = 0; k < Unit::N; ++k) put<YB>(at(to, ld, i, j, k), p.w[k], PER);
            } else {
#pragma unroll
                for (int k = 0; k < Unit::N; ++k) put<YB>(at(to, ld, i, j, k), p.w[k], left(i, j, k));
            }
        };
        void *C = (char *)a.C + (int64_t)split * a.M * a.ldc * (YB ? 2 : 4);
        if (a.res) {
#pragma unroll
            for (int x = 0; x < AHEAD; ++x) fetch(x);
        }
        each<UNITS>([&](auto number) {
            constexpr int x = decltype(number)::value, i = NT * (x % PAIRS), j = x / PAIRS;
            __builtin_amdgcn_sched_barrier(0);
            f32x16 v[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                v[n] = (BF ? acc : total)[i + n][j];
                asm volatile("" : "+v"(v[n]));           // leaves the matrix cores' registers here
            }
            if (!BEGIN && a.bias) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        float x[4];
                        bias_at(i + n, g, x);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[n][4 * g + e] += x[e];
                    }
            }
            if (ACT) {
                if (a.Z) leave(v, a.Z, a.N, i, j);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[n][e] = activate<ACT>(v[n][e]);
            }
            if (a.res) {
                r[x % AHEAD].add_to(v);
                if constexpr (x + AHEAD < UNITS) fetch(x + AHEAD);
            }
            leave(v, C, a.ldc, i, j);
        });
        if (tn >= tend) break;
        t = tn;
    }
    wait_copies<0>();
}

}  // namespace haste
